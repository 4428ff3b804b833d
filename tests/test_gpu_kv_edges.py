"""Cache and attention calls at the edges of what their documentation allows:
rows far outside the sequences, sinks, huge scales, many sequences, long walks.
Against the 64-bit oracle, within the bounds of kv_util."""
import numpy as np
import pytest
import torch

from column_scaled_gemm_amd import fp8sm
from kv_util import DT, attention_bounds, batch, dev_cache, random_cache, rng, to_dev
from oracle import kv as okv
from test_gpu_attention import check, run
from test_gpu_kv_cache import check_cache

pytestmark = pytest.mark.gpu


def rows(r, T, H, D, dtype="bf16"):
    return torch.from_numpy(r.standard_normal((T, H, D)).astype(np.float32)).to(DT[dtype])


@pytest.mark.parametrize("before", [16, 200, 1000])
@pytest.mark.parametrize("block", [16, 128])
@pytest.mark.parametrize("n,lens", [([3, 90], [40, 90]), ([0, 5], [70, 300]), ([33], [33])])
def test_many_rows_before_the_first_sequence(n, lens, block, before):
    """More of them than a block or a tile of rows: they have work slots that no
    sequence owns.  Nothing is written there, to no cache block either."""
    print(f"[case] before {before} {n} {lens} {block}", flush=True)
    r = rng(before + block)
    H, D = 2, 64
    cu, L, table, blocks = batch(r, n, lens, block)
    cu = (cu + before).astype(np.int32)
    T = int(cu[-1]) + 40
    ref = random_cache(r, blocks, H, block, D)
    for e in ref.exp:
        e[:] = 40       # below what a write of nothing would set
    x = rows(r, T, H, D)
    dev, d = dev_cache(ref), to_dev(cu, L, table)
    fp8sm.kv_cache_write(x.cuda(), x.cuda(), dev, *d)
    okv.write(ref, x.double().numpy(), x.double().numpy(), cu, L, table)
    check_cache(dev, ref)
    got = [torch.full((T, H, D), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    fp8sm.kv_cache_read(dev, *d, T, k=got[0], v=got[1])
    for g, w in zip(got, okv.read(ref, cu, L, table, T)):
        assert torch.equal(g.cpu(), torch.from_numpy(np.where(np.isnan(w), 3.0, w)).to(torch.bfloat16))
    q = rows(r, T, 4, D).cuda()
    for max_q in (1, 16, T):        # the kernels for few and for many rows
        out, lse = torch.full_like(q, 5.0), torch.full((T, 4), 5.0, device="cuda")
        fp8sm.attention_cache(q, dev, *d, max_q, out=out, lse=lse)
        mine = check(out, lse, q, ref, cu, L, table, D ** -0.5, True, 0, "bf16")
        rest = torch.from_numpy(~mine.all((1, 2)))
        assert int(rest.sum()) == T - sum(n)
        assert torch.all(out.cpu()[rest] == 5) and torch.all(lse.cpu()[rest] == 5)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,ln", [(3, 200), (80, 200), (3, 2500), (80, 2500)])
@pytest.mark.parametrize("gap", [10, 13, 16, 18, 22, 25])
def test_a_sink_whose_value_is_zero(n, ln, gap, dtype, D):
    """The first token leads every row by `gap` nats and adds nothing: what is left is
    the tail.  A p may be off by half a step of fp16 or by 2^-32 of the row's largest p,
    whichever is more; the latter moves a result by at most 2^-32 of the sum of the
    values' magnitudes."""
    print(f"[case] sink {n} {ln} {gap} {dtype} {D}", flush=True)
    r = rng(gap + ln)
    cu, L, table, blocks = batch(r, [n], [ln], 16)
    ref = random_cache(r, blocks, 1, 16, D)
    ref.exp[0][:], ref.exp[1][:] = 127, 127 + 4
    # keys: channel 0 alone counts, 1 for the sink and up to 2^-6 for the others
    for p in range(ln):
        page, slot = table[0, p // 16], p % 16
        k = ref.get(0, page, slot, 0).copy()
        k[0] = 0x38 if p == 0 else int(r.integers(0, 9))
        ref.put(0, page, slot, 0, k)
        v = ref.get(1, page, slot, 0) & 0x7F      # of one sign: nothing cancels
        ref.put(1, page, slot, 0, np.zeros_like(v) if p == 0 else v)
    q = torch.zeros(n, 2, D, dtype=DT[dtype], device="cuda")
    q[:, :, 0] = 8.0 * gap
    d = to_dev(cu, L, table)
    out, lse = fp8sm.attention_cache(q, dev_cache(ref), *d, n, scale=0.125, return_lse=True)
    o, s, spread, qk = okv.attention(q.double().cpu().numpy(), ref, cu, L, table, 0.125)
    to, tl = attention_bounds(o, s, spread, qk, 0.125, D, ln, dtype)
    if dtype == "bf16":
        to -= 2.0 ** -24        # bf16 has no such floor
    total = np.abs(okv.read(ref, [0, ln], [ln], table, ln)[1]).sum(0)
    to += 2.0 ** -32 * total
    err = np.abs(out.double().cpu().numpy() - o) / to
    print(f"[bound] {err.max():.3f}", flush=True)
    assert np.all(err <= 1)
    assert np.all(np.abs(lse.double().cpu().numpy() - s) <= tl)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,ln", [(1, 2), (2, 3), (3, 5), (2, 40), (5, 9), (40, 40), (33, 70)])
def test_probabilities_of_bf16_calls_lose_no_more_than_fp16_keeps(n, ln, D):
    """Values that cancel: what P was rounded by shows beside a small result's own
    rounding.  The bound of an fp16 call, with a half step of bf16 for the result."""
    print(f"[case] cancel {n} {ln} {D}", flush=True)
    r = rng(n * 100 + ln)
    G = 4       # up to 8 tokens: the kernel for few rows, more: for many
    cu, L, table, blocks = batch(r, [n], [ln], 16)
    ref = random_cache(r, blocks, 1, 16, D, spread=1)
    q = (rows(r, n, G, D) * 0.05).to(torch.bfloat16).cuda()
    out, lse = fp8sm.attention_cache(q, dev_cache(ref), *to_dev(cu, L, table), n, return_lse=True)
    o, s, spread, qk = okv.attention(q.double().cpu().numpy(), ref, cu, L, table, D ** -0.5)
    to, tl = attention_bounds(o, s, spread, qk, D ** -0.5, D, ln, "fp16")
    to += 1.01 * np.abs(o) * (2.0 ** -8 - 2.0 ** -11)
    err = np.abs(out.double().cpu().numpy() - o) / to
    print(f"[bound] {err.max():.3f}", flush=True)
    assert np.all(err <= 1) and np.all(np.abs(lse.double().cpu().numpy() - s) <= tl)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,ln", [(3, 200), (80, 200), (3, 2500), (80, 2500)])
@pytest.mark.parametrize("scale", [3e4, 1e9, -1e9, 1e20, 3e38])
def test_huge_scales_pick_the_largest_score(n, ln, scale, dtype, D):
    """Scores are whole numbers, 28672 and a place in a permutation more: the softmax
    of such scales is the token with the largest, its value comes out as it is."""
    print(f"[case] huge {n} {ln} {scale} {dtype} {D}", flush=True)
    r = rng(ln + n)
    cu, L, table, blocks = batch(r, [n], [ln], 16)
    ref = random_cache(r, blocks, 1, 16, D, spread=1)
    ref.exp[0][:] = 127
    codes = torch.arange(16.0).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    order = r.permutation(ln)
    for p in range(ln):
        k = np.zeros(D, dtype=np.uint8)
        k[:3] = codes[order[p] % 16], codes[order[p] // 16 % 16], codes[order[p] // 256]
        k[3] = 0x7E                                   # 448
        ref.put(0, table[0, p // 16], p % 16, 0, k)
    q = torch.zeros(n, 2, D, dtype=DT[dtype], device="cuda")
    q[:, :, :4] = torch.tensor([1.0, 16.0, 256.0, 64.0])
    d = to_dev(cu, L, table)
    out, lse = fp8sm.attention_cache(q, dev_cache(ref), *d, n, scale=scale, return_lse=True)
    vals = okv.read(ref, [0, ln], [ln], table, ln)[1][:, 0]
    g, gl = out.cpu(), lse.double().cpu().numpy()
    for i in range(n):
        seen = order[:ln - n + 1 + i]
        best = int(np.argmax(seen) if scale > 0 else np.argmin(seen))
        want = torch.from_numpy(vals[best]).to(DT[dtype])
        assert torch.equal(g[i, 0], want) and torch.equal(g[i, 1], want), i
        top = (28672.0 + seen[best]) * scale
        if abs(top) < 3e38:
            # the scale, log2(e), their product, its product, ln(2) and the last one
            assert np.all(np.abs(gl[i] - top) <= 1.01 * 6 * 2.0 ** -24 * abs(top))
        else:
            assert np.all(np.isposinf(gl[i]))


def sampled(q, got, lse, cache, ref, L, table, picks, dtype="bf16", n=1, window=0):
    """Checks the sequences `picks` of a batch of n rows each against the oracle."""
    D = q.shape[2]
    for b in picks:
        sl = slice(b * n, (b + 1) * n)
        check(got[sl], lse[sl], q[sl], ref, np.int32([0, n]), L[b:b + 1], table[b:b + 1], D ** -0.5, True, window,
              dtype)


@pytest.mark.parametrize("max_q,G", [(1, 4), (100, 4)])
@pytest.mark.parametrize("long", [False, True])
def test_more_workgroups_than_a_grids_first_dimension(max_q, G, long):
    """70000 sequences of one row that share their blocks, for the kernels for few and
    for many rows; the long ones in the few splits that the workspace's bound leaves,
    with a join of more than 65536 workgroups."""
    print(f"[case] grid {max_q} {G} {long}", flush=True)
    r = rng(60)
    B, D, block = 70000, 64, 128
    top = 7000 if long else 60
    L = r.integers(1, top + 1, B).astype(np.int32)
    L[[0, 1, B - 2, B - 1]] = [1, top, top, 1]
    ref = random_cache(r, 60, 1, block, D)
    table = np.broadcast_to(r.permutation(60)[:-(-top // block)].astype(np.int32), (B, -(-top // block)))
    cache = dev_cache(ref)
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    dl, dt = to_dev(L, table)
    q = torch.randn(B, G, D, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    max_kv = 1 << 20 if max_q == 1 else 1000       # (beside long contexts few rows go to their own kernel)
    need = fp8sm.attention_cache_workspace(B, B, G, 1, D, max_q, max_kv)
    assert need == (3 * B * G * (D + 2) * 4 if max_q == 1 else 0)
    out, lse = fp8sm.attention_cache(q, cache, cu, dl, dt, max_q, max_kv=max_kv, return_lse=True)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    sampled(q, out, lse, cache, ref, L, table, [0, 1, 40000, 65535, 65536, B - 2, B - 1])


@pytest.mark.parametrize("T", [0, 1, 2])
@pytest.mark.parametrize("own", [False, True])
def test_rotation_in_place_of_few_rows(T, own):
    """out: x itself, or the view of its query and key heads (a decode batch may
    shrink to one row, whose stride says nothing)."""
    r = rng(70)
    Hq, Hk, D = 4, 2, 64
    x = rows(r, T, Hq + 2 * Hk, D).flatten(1).cuda()
    pos, cs = to_dev(np.arange(5, 5 + T, dtype=np.int32), np.ones((9, D), dtype=np.float32))
    want = fp8sm.qk_norm_rope(x, Hq, Hk, D, pos, cs)
    y = x.clone()
    out = y if own else y[:, :(Hq + Hk) * D]
    assert fp8sm.qk_norm_rope(y, Hq, Hk, D, pos, cs, out=out) is out
    assert torch.equal(y[:, :(Hq + Hk) * D], want) and torch.equal(y[:, (Hq + Hk) * D:], x[:, (Hq + Hk) * D:])


@pytest.mark.parametrize("n", [[3, 1], [80, 1]])
@pytest.mark.parametrize("window", [(1 << 31) + 2, (1 << 32) + 5])
def test_windows_beyond_32_bits(n, window):
    run(n, [130, 70], 2, 1, 64, 16, "bf16", window=window)


@pytest.mark.parametrize("T,B", [(0, 2), (0, 0), (3, 0)])
def test_empty_batches(T, B):
    """As a server's step may leave them: no rows, no sequences, and no longest one."""
    c = fp8sm.kv_cache_empty(3, 2, 64, 16)
    for t in c:
        t.fill_(7)
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, lens, table = torch.zeros(B + 1, **i32), torch.full((B,), 20, **i32), torch.zeros(B, 2, **i32)
    q = torch.full((T, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    k = q[:, :2].contiguous()
    out, lse = torch.full_like(q, 5.0), torch.full((T, 4), 5.0, device="cuda")
    fp8sm.kv_cache_write(k, k, c, cu, lens, table)
    fp8sm.attention_cache(q, c, cu, lens, table, 0, out=out, lse=lse)
    got = fp8sm.kv_cache_read(c, cu, lens, table, T, k=torch.full_like(k, 5.0), v=torch.full_like(k, 5.0))
    for t, v in [(t, 7) for t in c] + [(t, 5) for t in (out, lse, *got)]:
        assert bool(torch.all(t == v))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_reading_keys_or_values_alone(dtype):
    r = rng(71)
    cu, L, table, blocks = batch(r, [3, 20], [40, 33], 16)
    cache, d = dev_cache(random_cache(r, blocks, 2, 16, 64)), to_dev(cu, L, table)
    k, v = fp8sm.kv_cache_read(cache, *d, 23, dtype=dtype)
    k1, none = fp8sm.kv_cache_read(cache, *d, 23, dtype=dtype, values=False)
    assert none is None and torch.equal(k1, k)
    none, v1 = fp8sm.kv_cache_read(cache, *d, 23, dtype=dtype, keys=False)
    assert none is None and torch.equal(v1, v)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    none, v2 = fp8sm.kv_cache_read(cache, *d, 23, dtype=dtype, keys=False, v=torch.zeros_like(v), stream=side)
    side.synchronize()
    assert none is None and torch.equal(v2, v)
    assert fp8sm.kv_cache_read(cache, *d, 23, keys=False, values=False) == (None, None)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("kind", ["plain", "window", "full", "wide", "missing"])
def test_long_walks_of_one_workgroup(kind, dtype, D):
    """More steps than one gather of blocks and scales brings, thrice, unsplit: the
    hint says one token."""
    def damage(cu, L, table, ref):
        if kind == "wide":
            ref.exp[1][:] = rng(5).integers(100, 121, ref.exp[1].shape)
        if kind == "missing":
            table[0, 3], table[0, 200] = -1, ref.blocks

    for n in ([70], [3]):       # the kernels for many and for few rows
        run(n, [6500], 2, 1, D, 16, dtype, max_kv=1, window=5000 if kind == "window" else 0, causal=kind != "full",
            damage=damage)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,lens", [([1, 3], [200, 65]), ([150, 2], [200, 65]), ([140, 80], [100, 0])])
def test_without_causality_in_fp16(n, lens, D):
    run(n, lens, 4, 2, D, 32, "fp16", causal=False)


def test_long_contexts_without_causality_and_splits():
    run([1, 90], [9000, 3000], 4, 2, 64, 64, "fp16", causal=False)


def test_a_mixed_batch_captured_and_replayed_with_other_rows_and_lengths():
    """Both kernels, splits and the join; rows before, behind and of no sequence."""
    r = rng(80)
    H, D, block, T = 2, 64, 32, 130
    cu0, L0, table, blocks = batch(r, [60, 1, 5], [5000, 5000, 5000], block)
    cache = dev_cache(random_cache(r, blocks, H, block, D))
    cu, lens, tab = to_dev(cu0, L0, table)
    q = rows(r, T, 4, D).cuda()
    x = rows(r, T, H, D).cuda()
    out = torch.zeros_like(q)
    lse = torch.zeros(T, 4, device="cuda")

    def step(cache, out, lse):
        fp8sm.kv_cache_write(x, x, cache, cu, lens, tab)
        fp8sm.attention_cache(q, cache, cu, lens, tab, 100, max_kv=5000, out=out, lse=lse)

    step(cache, out, lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache, out, lse)
    for c, n in (([0, 60, 61, 66], [5000, 4000, 70]), ([30, 30, 130, 130], [9, 2600, 1]), ([0, 1, 2, 3], [4999, 17, 0]),
                 ([100, 101, 110, 110], [5000, 9, 5000]), ([0, 60, 61, 66], [5000, 4000, 70])):
        cu.copy_(torch.tensor(c, dtype=torch.int32))
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        mine = fp8sm.KVCache(*(t.clone() for t in cache))
        want, want_l = torch.full_like(out, 5.0), torch.full_like(lse, 5.0)
        step(mine, want, want_l)
        out.fill_(5.0)
        lse.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_l)
        rest = torch.ones(T, dtype=torch.bool)
        rest[c[0]:c[-1]] = False
        assert torch.all(out.cpu()[rest] == 5) and torch.all(lse.cpu()[rest] == 5)
        for a, b in zip(cache, mine):
            assert torch.equal(a, b)
