"""Attention over the E4M3 cache against the 64-bit oracle, within the bound of
kv_util.attention_bounds."""
import numpy as np
import pytest
import torch

from column_scaled_gemm_amd import fp8sm
from kv_util import DT, attention_bounds, batch, dev_cache, random_cache, rng, to_dev
from oracle import kv as okv

pytestmark = pytest.mark.gpu


def check(out, lse, q, ref, cu, L, table, scale, causal, window, dtype):
    o, s, spread, qk = okv.attention(q.double().cpu().numpy(), ref, cu, L, table, scale, causal, window)
    to, tl = attention_bounds(o, s, spread, qk, scale, q.shape[2], max(int(max(L)), 1), dtype)
    g, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    mine = ~np.isnan(o)
    assert np.array_equal(np.isneginf(gl[~np.isnan(s)]), np.isneginf(s[~np.isnan(s)]))
    err = np.abs(g - o)[mine] / to[mine]
    fin = np.isfinite(s)
    err_l = (np.abs(gl[fin] - s[fin]) / tl[fin]) if fin.any() else np.zeros(1)
    print(f"[bound] out {err.max() if err.size else 0:.3f} lse {err_l.max():.3f}", flush=True)
    assert np.all(err <= 1) and np.all(err_l <= 1)
    return mine


def run(n, lens, Hq, H, D, block, dtype, window=0, causal=True, max_q=None, max_kv=None, gain=1.0, seed=0,
        scale=None, damage=None):
    print(f"[case] attn n={n} lens={lens} {Hq}/{H} D={D} block={block} {dtype} w={window} causal={causal} "
          f"max_q={max_q} max_kv={max_kv}", flush=True)
    r = rng(seed + sum(lens) + Hq)
    cu, L, table, blocks = batch(r, n, lens, block)
    ref = random_cache(r, blocks, H, block, D)
    # what lies behind a sequence's end may hold anything, NaN codes too
    for b, ln in enumerate(lens):
        if ln % block:
            for which in (0, 1):
                for s in range(ln % block, block):
                    for h in range(H):
                        ref.put(which, table[b, ln // block], s, h, 0x7F)
    if damage:
        damage(cu, L, table, ref)
    T = sum(n)
    qkv = torch.from_numpy((r.standard_normal((T, Hq * D + 64)) * gain).astype(np.float32)).to(DT[dtype]).cuda()
    q = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    wide = torch.full((T, Hq * D + 16), 9.0, dtype=DT[dtype], device="cuda")
    out = wide[:, :Hq * D].unflatten(1, (Hq, D))
    d = to_dev(cu, L, table)
    kw = dict(max_kv=max_kv, causal=causal, window=window, scale=scale)
    mq = max(max(n), 1) if max_q is None else max_q
    got, lse = fp8sm.attention_cache(q, dev_cache(ref), *d, mq, out=out, return_lse=True, **kw)
    assert torch.all(wide[:, Hq * D:] == 9)
    check(got, lse, q, ref, cu, L, table, D ** -0.5 if scale is None else scale, causal, window, dtype)
    again = fp8sm.attention_cache(q, dev_cache(ref), *d, mq, **kw)
    assert torch.equal(again, got)          # run to run the same bits, without lse too
    return got, lse, q, ref, d


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,lens,Hq,H,block", [
    ([1], [1], 1, 1, 16), ([1], [63], 4, 1, 16), ([1, 1, 1], [64, 65, 300], 8, 2, 32),
    ([2, 1, 3], [90, 1, 257], 5, 1, 64), ([9], [700], 4, 2, 128), ([4, 0, 4], [33, 20, 130], 16, 2, 16)])
def test_few_rows(n, lens, Hq, H, block, dtype, D):
    run(n, lens, Hq, H, D, block, dtype)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,lens,Hq,H,block", [
    ([65], [65], 1, 1, 16), ([128], [200], 2, 2, 32), ([70, 129], [70, 300], 4, 2, 64),
    ([43], [500], 7, 1, 128), ([100, 1, 0, 17, 90], [130, 77, 12, 140, 90], 6, 2, 16)])
def test_many_rows(n, lens, Hq, H, block, dtype, D):
    run(n, lens, Hq, H, D, block, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("window", [1, 7, 64, 100, 1000])
@pytest.mark.parametrize("n,lens", [([1, 2], [300, 129]), ([90, 3], [300, 129])])
def test_window(n, lens, window, dtype):
    run(n, lens, 2, 1, 64, 16, dtype, window=window)


@pytest.mark.parametrize("n,lens", [([1, 3], [200, 65]), ([150, 2], [200, 65])])
def test_without_causality(n, lens):
    run(n, lens, 2, 2, 128, 32, "bf16", causal=False)


@pytest.mark.parametrize("n,lens", [([5, 2], [3, 0]), ([140, 80], [100, 0]), ([20], [7])])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_before_the_first_token_see_nothing(n, lens, causal):
    got, lse, *_ = run(n, lens, 2, 1, 64, 16, "bf16", causal=causal)
    if causal:
        assert torch.all(got[:n[0] - lens[0]] == 0) and torch.all(torch.isneginf(lse[:n[0] - lens[0]]))


@pytest.mark.parametrize("n,lens,Hq", [([1, 1], [3000, 900], 4), ([2], [4100], 16), ([80, 1], [2500, 1700], 2)])
@pytest.mark.parametrize("max_kv", [None, 1, 5000, 1 << 30])
@pytest.mark.parametrize("window", [0, 1500])
def test_splits_whatever_the_hints(n, lens, Hq, max_kv, window):
    """max_kv and max_q steer, they do not bound."""
    run(n, lens, Hq, 1, 64, 64, "bf16", max_kv=max_kv, window=window)
    run(n, lens, Hq, 1, 64, 64, "bf16", max_kv=max_kv, window=window, max_q=1 if max(n) > 1 else 500)


@pytest.mark.parametrize("gain", [0.0, 8.0])
@pytest.mark.parametrize("n", [[1], [80]])
def test_flat_and_sharp_scores(n, gain):
    run(n, [900], 2, 1, 128, 16, "fp16", gain=gain)
    run(n, [900], 2, 1, 128, 16, "bf16", gain=gain, scale=0.3)


@pytest.mark.parametrize("n,max_q", [([1, 1], None), ([70, 5], None), ([1, 70], None)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_wide_scale_range_and_missing_blocks(n, max_q, dtype):
    def damage(cu, L, table, ref):
        for which in (0, 1):
            ref.exp[which][:] = rng(5).integers(105, 128, ref.exp[which].shape)
        ref.exp[0][:] = np.minimum(ref.exp[0], 121)
        table[0, 1], table[1, 2] = -1, ref.blocks
        # the first step of tokens is gone as a whole
        table[1, 0] = 2 ** 30

    run(n, [200, 170], 4, 2, 64, 64, dtype, damage=damage)


def test_rows_of_no_sequence_are_left():
    r = rng(9)
    cu, L, table, blocks = batch(r, [2, 90], [70, 100], 16)
    ref = random_cache(r, blocks, 1, 16, 64)
    T = 100
    cu = cu + 3
    q = torch.from_numpy(r.standard_normal((T, 2, 64)).astype(np.float32)).to(torch.bfloat16).cuda()
    out, lse = torch.full_like(q, 5.0), torch.full((T, 2), 5.0, device="cuda")
    fp8sm.attention_cache(q, dev_cache(ref), *to_dev(cu, L, table), 90, out=out, lse=lse)
    mine = check(out, lse, q, ref, cu, L, table, 0.125, True, 0, "bf16")
    rest = torch.from_numpy(~mine.all((1, 2)))
    assert rest.sum() == 8 and torch.all(out.cpu()[rest] == 5) and torch.all(lse.cpu()[rest] == 5)


def test_many_sequences():
    r = rng(10)
    n = [int(v) for v in r.integers(0, 3, 200)]
    lens = [a + int(v) for a, v in zip(n, r.integers(0, 50, 200))]
    run(n, lens, 4, 1, 64, 16, "bf16")


def test_a_row_does_not_depend_on_the_rest_of_the_batch():
    """Same kernel, same split: a sequence alone gives the bits it gives in a batch."""
    got, lse, q, ref, d = run([1, 1, 1], [300, 50, 129], 4, 2, 128, 16, "bf16", max_kv=300)
    for b in range(3):
        one = fp8sm.attention_cache(q[b:b + 1], dev_cache(ref), to_dev(np.int32([0, 1]))[0], d[1][b:b + 1],
                                    d[2][b:b + 1], 1, max_kv=300)
        assert torch.equal(one[0], got[b])


def test_captured_and_replayed_with_other_lengths():
    r = rng(11)
    B, H, D, block = 3, 2, 64, 16
    cu, L, table, blocks = batch(r, [1] * B, [600, 600, 600], block)
    ref = random_cache(r, blocks, H, block, D)
    cache, (dcu, dl, dt) = dev_cache(ref), to_dev(cu, L, table)
    rows = torch.zeros(B, 8 * D, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    cs = torch.from_numpy(np.concatenate([np.cos(np.outer(np.arange(700), 0.1 ** np.arange(32))),
                                          np.sin(np.outer(np.arange(700), 0.1 ** np.arange(32)))], 1).astype(np.float32)).cuda()

    def step(rows, cache):
        fp8sm.qk_norm_rope(rows, 4, 2, D, pos, cs, out=rows)
        fp8sm.kv_cache_write(rows[:, 4 * D:6 * D], rows[:, 6 * D:], cache, dcu, dl, dt)
        return fp8sm.attention_cache(rows[:, :4 * D].unflatten(1, (4, D)), cache, dcu, dl, dt, 1, max_kv=600)

    step(rows, cache)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(rows, cache)
    for lens in ([1, 30, 600], [2, 31, 17], [599, 600, 300], [2, 32, 18]):
        x = torch.from_numpy(r.standard_normal((B, 8 * D)).astype(np.float32)).to(torch.bfloat16).cuda()
        dl.copy_(torch.tensor(lens, dtype=torch.int32))
        pos.copy_(dl - 1)
        mine = fp8sm.KVCache(*(t.clone() for t in cache))
        want = step(x.clone(), mine)
        rows.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        for a, b in zip(cache, mine):
            assert torch.equal(a, b)


def test_two_streams_with_their_own_workspaces():
    jobs = [run([1, 1], [3000, 2000], 8, 2, 64, 32, "bf16", seed=s) for s in (1, 2)]
    caches = [dev_cache(j[3]) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    outs = [torch.empty_like(j[0]) for j in jobs]
    torch.cuda.synchronize()
    for _ in range(4):
        for j, c, st, o in zip(jobs, caches, streams, outs):
            with torch.cuda.stream(st):
                fp8sm.attention_cache(j[2], c, *j[4], 1, out=o)
        for j, c, st, o in zip(jobs, caches, streams, outs):   # from a stream that is not the current one
            fp8sm.attention_cache(j[2], c, *j[4], 1, out=o, stream=st)
    torch.cuda.synchronize()
    for j, o in zip(jobs, outs):
        assert torch.equal(o, j[0])


def test_the_run_from_the_projection_to_the_output_projection():
    """quant -> QKV product -> norm + rotation -> cache -> attention -> quant ->
    output product: a prompt in two pieces, then single tokens, against the same
    steps in 64 bits from the values that each step was given."""
    r = rng(12)
    hid, Hq, H, D, block = 256, 4, 2, 64, 16
    W = (Hq + 2 * H) * D
    wqkv, wo = (torch.from_numpy((r.standard_normal(s) * 0.06).astype(np.float32)).to(torch.bfloat16).cuda()
                for s in ((W, hid), (hid, Hq * D)))
    qw, sw = fp8sm.quant_group(wqkv, -1)
    qo, so = fp8sm.quant_group(wo, -1)
    nw = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    ang = np.outer(np.arange(200), 100.0 ** (-np.arange(32) / 32))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    dcs = to_dev(cs)[0]
    table = np.int32([[3, 0, 7, 1, 9, 2, 4], [5, 6, 8, 10, 11, 12, 13]])
    cache = fp8sm.kv_cache_empty(14, H, D, block)
    for t in cache:
        t.zero_()
    ref = okv.Cache(*(t.cpu().numpy() for t in cache))
    have = [0, 0]
    for n in ([70, 5], [0, 66], [1, 1], [1, 1], [2, 0]):
        have = [a + b for a, b in zip(have, n)]
        cu, L = np.int32([0, n[0], sum(n)]), np.int32(have)
        pos = np.concatenate([np.arange(a - b, a) for a, b in zip(have, n)]).astype(np.int32)
        d = to_dev(cu, L, table)
        x = torch.from_numpy(r.standard_normal((sum(n), hid)).astype(np.float32)).to(torch.bfloat16).cuda()
        qx, sx = fp8sm.quant_group(x, -1)
        qkv = fp8sm.scaled_mm(qx, qw, sx.reshape(-1), sw.reshape(-1), fp8sm.KIND_ROW, fp8sm.KIND_COL)
        before = qkv.double().cpu().numpy()
        fp8sm.qk_norm_rope(qkv, Hq, H, D, to_dev(pos)[0], dcs, nw, nw, out=qkv)
        rot, mag = okv.norm_rope(before, Hq, H, D, pos, cs, np.ones(D), np.ones(D))
        after = qkv.double().cpu().numpy()
        assert np.all(np.abs(after[:, :(Hq + H) * D].reshape(rot.shape) - rot) <=
                      1.01 * (np.abs(rot) * 2.0 ** -8 + mag * (D / 2 + 10) * 2.0 ** -24))
        k, v = qkv[:, Hq * D:(Hq + H) * D], qkv[:, (Hq + H) * D:]
        fp8sm.kv_cache_write(k, v, cache, *d)
        okv.write(ref, *(t.double().cpu().numpy().reshape(-1, H, D) for t in (k, v)), cu, L, table)
        for g, c in zip(cache, (*ref.codes, *ref.exp)):
            assert np.array_equal(g.cpu().numpy(), c)
        q = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        out, lse = fp8sm.attention_cache(q, cache, *d, max(n), max_kv=max(have), return_lse=True)
        check(out, lse, q, ref, cu, L, table, 0.125, True, 0, "bf16")
        qa, sa = fp8sm.quant_group(out.flatten(1), -1)
        y = fp8sm.scaled_mm(qa, qo, sa.reshape(-1), so.reshape(-1), fp8sm.KIND_ROW, fp8sm.KIND_COL)
        assert y.shape == (sum(n), hid) and bool(torch.isfinite(y).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,lens,Hq,wide", [([5], [70], 2, False), ([9], [300], 3, False), ([150], [190], 1, False),
                                            ([150], [190], 1, True)])
@pytest.mark.parametrize("window", [0, 60])
def test_nan_tokens_reach_only_the_rows_that_see_them(n, lens, Hq, wide, window, dtype, D):
    """A NaN key makes every output of a row that sees it NaN, a NaN value its
    channel; the other rows are as if it were not there."""
    print(f"[case] nan {n} {lens} {Hq} {wide} {window} {dtype} {D}", flush=True)
    r = rng(40 + D)
    cu, L, table, blocks = batch(r, n, lens, 16)
    ref = random_cache(r, blocks, 1, 16, D)
    if wide:
        ref.exp[1][:] = r.integers(100, 125, ref.exp[1].shape)
    T, ln = n[0], lens[0]
    q = torch.from_numpy(r.standard_normal((T, Hq, D)).astype(np.float32)).to(DT[dtype]).cuda()
    clean = okv.Cache(ref.codes[0], ref.codes[1], *ref.exp)
    # a NaN value in the last token but two of channel 3, one further back, a NaN key
    for which, pos, ch in ((1, ln - 3, 3), (1, ln - T + 1, 5), (1, 2, 7), (0, ln - 2, 1)):
        page, slot = table[0, pos // 16], pos % 16
        c = ref.get(which, page, slot, 0).copy()
        c[ch] = 0xFF
        ref.put(which, page, slot, 0, c)
    d = to_dev(cu, L, table)
    out, lse = fp8sm.attention_cache(q, dev_cache(ref), *d, T, window=window, return_lse=True)
    o, s, spread, qk = okv.attention(q.double().cpu().numpy(), clean, cu, L, table, D ** -0.5, True, window)
    to, tl = attention_bounds(o, s, spread, qk, D ** -0.5, D, ln, dtype)
    pos = np.arange(ln - T, ln)[:, None]

    def sees(p):
        return ((p <= pos) & (p > pos - window) if window else p <= pos)[:, 0]

    want = np.zeros((T, Hq, D), dtype=bool)
    want[sees(ln - 3), :, 3] = True
    want[sees(ln - T + 1), :, 5] = True
    want[sees(2), :, 7] = True
    want[sees(ln - 2)] = True
    g, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isnan(g), want)
    assert np.array_equal(np.isnan(gl), np.broadcast_to(sees(ln - 2)[:, None], gl.shape))
    # the clean cache differs in tokens that these rows see with other codes: compare rows that see none
    none = ~(sees(ln - 3) | sees(ln - T + 1) | sees(2) | sees(ln - 2))
    if none.any():
        assert np.all(np.abs(g - o)[none] <= to[none]) and np.all(np.abs(gl - s)[none] <= tl[none])


@pytest.mark.parametrize("n", [[1, 2], [70, 1]])
@pytest.mark.parametrize("scale", [0.0, -0.2])
def test_zero_and_negative_scale(n, scale):
    print(f"[case] scale {scale} {n}", flush=True)
    r = rng(50)
    cu, L, table, blocks = batch(r, n, [130, 70], 16)
    ref = random_cache(r, blocks, 2, 16, 64)
    q = torch.from_numpy(r.standard_normal((sum(n), 4, 64)).astype(np.float32)).to(torch.bfloat16).cuda()
    out, lse = fp8sm.attention_cache(q, dev_cache(ref), *to_dev(cu, L, table), max(n), scale=scale, return_lse=True)
    o, s, spread, qk = okv.attention(q.double().cpu().numpy(), ref, cu, L, table, scale)
    to, tl = attention_bounds(o, s, spread, qk, abs(scale), 64, 130, "bf16")
    assert np.all(np.abs(out.double().cpu().numpy() - o) <= to)
    assert np.all(np.abs(lse.double().cpu().numpy() - s) <= tl)


@pytest.mark.parametrize("n", [[1, 2], [70, 1]])
def test_largest_scale_of_scores_that_are_zero(n):
    got, lse, *_ = run(n, [130, 70], 4, 2, 64, 16, "bf16", gain=0.0, scale=3e38)
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("n,lens", [([6, 3], [2, 40]), ([140], [70])])
@pytest.mark.parametrize("window", [(1 << 30) - 1, 1 << 30, (1 << 31) - 1])
def test_largest_windows(n, lens, window):
    """Rows before the first token too: their position less the window."""
    run(n, lens, 2, 1, 64, 16, "bf16", window=window)


@pytest.mark.parametrize("n", [[3], [80]])
@pytest.mark.parametrize("ke,ve", [(85, 85), (100, 200), (85, 240)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_extreme_scales(n, ke, ve, dtype):
    """Tiny keys and values, and values beyond fp16's range (bf16 results)."""
    def damage(cu, L, table, ref):
        ref.exp[0][:] = ke
        ref.exp[1][:] = ve
    if dtype == "fp16" and ve > 130:
        return
    run(n, [200], 2, 1, 64, 32, dtype, damage=damage)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_short_sequences_with_long_caches_in_a_mixed_batch(dtype, D):
    """Both kernels run, each with splits of its own."""
    run([90, 1, 0, 2, 30, 1], [2300, 5000, 70, 3100, 2100, 40], 4, 2, D, 64, dtype, max_kv=5000)


def test_sequences_that_share_blocks():
    r = rng(51)
    cu, L, table, blocks = batch(r, [1, 70, 1], [100, 100, 33], 16)
    table[1, :2], table[2, :2] = table[0, :2], table[0, :2]
    ref = random_cache(r, blocks, 1, 16, 64)
    q = torch.from_numpy(r.standard_normal((72, 3, 64)).astype(np.float32)).to(torch.float16).cuda()
    out, lse = fp8sm.attention_cache(q, dev_cache(ref), *to_dev(cu, L, table), 70, return_lse=True)
    check(out, lse, q, ref, cu, L, table, 0.125, True, 0, "fp16")


def test_on_a_stream_that_is_not_the_current_one():
    """The outputs and the workspace allocated for such a call are that stream's, so
    memory that the current stream still works on is not handed to it."""
    got, lse, q, ref, d = run([1, 1, 2], [3000, 500, 2500], 8, 2, 128, 32, "bf16")
    cache, side = dev_cache(ref), torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device="cuda")
    for _ in range(3):
        torch.cuda.synchronize()
        for _ in range(4):
            busy = busy @ busy * 1e-4      # the current stream is behind, its freed memory in use
        out = fp8sm.attention_cache(q, cache, *d, 2, stream=side)
        k, v = fp8sm.kv_cache_read(cache, *d, 4, stream=side)
        side.synchronize()
        assert torch.equal(out.cpu(), got.cpu())
        w = okv.read(ref, d[0].cpu().numpy(), d[1].cpu().numpy(), d[2].cpu().numpy(), 4)
        assert torch.equal(k.cpu(), torch.from_numpy(w[0]).bfloat16())
        assert torch.equal(v.cpu(), torch.from_numpy(w[1]).bfloat16())
