"""Packed attention and rotation on several axes against the 64-bit oracle, within
derived bounds, and a layer in 8-bit integers from end to end."""
import numpy as np
import pytest
import torch

from column_scaled_gemm_amd import fp8sm
from kv_util import DT, attention_bounds, rng
from oracle import int8 as oi, packed as op

pytestmark = pytest.mark.gpu


def ints(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def normal(r, *shape):
    return torch.from_numpy(r.standard_normal(shape).astype(np.float32)).cuda()


def check(out, lse, q, k, v, cu, scale, causal, window, dtype):
    o, s, spread, qk = op.attention(*(t.double().cpu().numpy() for t in (q, k, v)), cu, scale, causal, window)
    longest = max(max(b - a for a, b in zip(cu[:-1], cu[1:])), 1)
    to, tl = attention_bounds(o, s, spread, qk, abs(scale), q.shape[2], longest, dtype)
    g, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    mine = np.isfinite(o)
    err, err_l = np.abs(g - o)[mine] / to[mine], np.abs(gl - s)[np.isfinite(s)] / tl[np.isfinite(s)]
    print(f"[bound] out {err.max():.3f} lse {err_l.max():.3f}", flush=True)
    assert np.all(err <= 1) and np.all(err_l <= 1)
    return o


def run(n, Hq, H, D, dtype, causal=True, window=0, gain=1.0, scale=None, before=0, behind=2, seed=0):
    print(f"[case] packed n={n} {Hq}/{H} D={D} {dtype} causal={causal} w={window} gain={gain} scale={scale}", flush=True)
    r = rng(seed + sum(n) + Hq)
    cu = [before]
    for k in n:
        cu.append(cu[-1] + k)
    T = cu[-1] + behind
    rows = normal(r, T, (Hq + 2 * H) * D + 8) * gain
    rows[:before] = float("nan")
    rows[cu[-1]:] = float("nan")           # of no prompt: may hold anything
    rows = rows.to(DT[dtype])
    q, k, v = rows[:, 8:].split([Hq * D, H * D, H * D], 1)
    q, k, v = q.unflatten(1, (Hq, D)), k.unflatten(1, (H, D)), v.unflatten(1, (H, D))
    wide = torch.full((T, Hq * D + 16), 9.0, dtype=DT[dtype], device="cuda")
    out, lse = wide[:, :Hq * D].unflatten(1, (Hq, D)), torch.full((T, Hq), 5.0, device="cuda")
    kw = dict(causal=causal, window=window, scale=scale)
    fp8sm.attention_packed(q, k, v, ints(cu), out=out, lse=lse, **kw)
    check(out, lse, q, k, v, cu, D ** -0.5 if scale is None else scale, causal, window, dtype)
    for a, b in ((0, before), (cu[-1], T)):
        assert torch.all(out[a:b] == 9) and torch.all(lse[a:b] == 5)
    assert torch.all(wide[:, Hq * D:] == 9)
    again = fp8sm.attention_packed(q, k, v, ints(cu), **kw)
    assert torch.equal(again[before:cu[-1]], out[before:cu[-1]])
    return q, k, v, cu, out, lse


LENGTHS = [([1], 1, 1), ([2], 4, 1), ([63], 2, 2), ([64], 2, 1), ([65], 4, 4), ([127, 1, 0, 129], 4, 2),
           ([0, 33, 0, 0, 200], 7, 1), ([300, 5, 64, 128], 10, 2), ([1] * 70, 3, 3), ([520], 6, 6)]


@pytest.mark.parametrize("n,Hq,H", LENGTHS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("causal", [True, False])
def test_lengths_and_heads(n, Hq, H, D, dtype, causal):
    run(n, Hq, H, D, dtype, causal=causal)


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 200, 1000, 2 ** 31 - 1])
@pytest.mark.parametrize("D,dtype", [(64, "fp16"), (128, "bf16")])
def test_windows(window, D, dtype):
    run([300, 70, 1], 6, 2, D, dtype, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("causal", [True, False])
def test_long_prompts(dtype, causal):
    run([2500, 1100], 2, 1, 128, dtype, causal=causal)
    run([3000], 1, 1, 64, dtype, causal=causal)


@pytest.mark.parametrize("gain", [0.0, 6.0])
@pytest.mark.parametrize("scale", [None, -0.3, 0.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_flat_sharp_and_negative_scores(gain, scale, dtype):
    run([190, 40], 2, 1, 64, dtype, gain=gain, scale=scale)


@pytest.mark.parametrize("Hq,H", [(63, 63), (64, 64), (65, 65), (72, 72), (140, 70)])
@pytest.mark.parametrize("causal", [True, False])
def test_many_heads(Hq, H, causal):
    run([140, 0, 30, 1], Hq, H, 64, "bf16", causal=causal, before=3)


def test_more_threads_than_32_bits_count():
    """300000 prompts without tokens around one with some: 4.9e9 threads in one call."""
    print("[case] many empty prompts", flush=True)
    n, H, D = 40, 64, 64
    q, k, v = (normal(rng(5), n, H, D).bfloat16() for _ in range(3))
    want = fp8sm.attention_packed(q, k, v, ints([0, n]))
    for place in (1, 150000, 300000):
        cu = torch.full((300001,), n, dtype=torch.int32, device="cuda")
        cu[:place] = 0
        assert torch.equal(fp8sm.attention_packed(q, k, v, cu), want)


def test_rows_before_the_first_prompt():
    run([100, 30], 4, 2, 128, "bf16", before=5)
    run([100, 30], 4, 2, 64, "fp16", before=300)


@pytest.mark.parametrize("scale", [1e30, 1e36, 3e38])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_huge_scales_pick_the_largest_score(scale, dtype):
    """The softmax of scores a huge factor apart is one of the token with the largest."""
    print("[case] huge", scale, dtype, flush=True)
    r = rng(7)
    n, D = 150, 64
    q, k, v = (normal(r, n, 1, D).to(DT[dtype]) for _ in range(3))
    out = fp8sm.attention_packed(q, k, v, ints([0, n]), scale=scale)
    s = q[:, 0].double() @ k[:, 0].double().T.contiguous()
    s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), float("-inf"))
    top = s.topk(2, 1).values
    clear = top[:, 0] - top[:, 1] > 1e-3       # (fp32 scores: 64 products of size below 2^4 each)
    assert torch.equal(out[clear, 0], v[s.argmax(1), 0][clear])


def test_a_token_of_no_value_leaves_the_rest_its_weight():
    """A token whose value is 0 leads by 18 nats: the others make up the output."""
    for dtype in ("bf16", "fp16"):
        n, D = 200, 64
        q = torch.zeros(n, 1, D, dtype=DT[dtype], device="cuda")
        k, v = torch.zeros_like(q), torch.ones_like(q)
        q[:, :, 0] = 1
        k[0, 0, 0] = 18 * 8
        v[0] = 0
        out = fp8sm.attention_packed(q, k, v, ints([0, n]))
        i = torch.arange(n, device="cuda", dtype=torch.float64)
        want = i / (i + np.exp(18.0))
        err = (out[:, 0, 0].double() - want).abs()[1:] / want[1:]
        # p and the result rounded (half a step each), the sum and the exponential in
        # fp32; below 2^-14 fp16 results have the fixed step 2^-24.  The p of fp16 calls,
        # 2^7 times as large, have that step too: off by up to 2^-25 2^-7 = 2^-32 of the
        # row's largest, which is e^18 times theirs
        step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
        floor = 2.0 ** -25 / want[1:] + 2.0 ** -32 * np.exp(18.0) if dtype == "fp16" else 0
        assert torch.all(err <= 2 * step + 1e-5 + floor)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "fp16"), (128, "bf16")])
def test_what_a_row_does_not_see_does_not_reach_it(causal, D, dtype):
    """Infinities and NaN in keys and values: other prompts, and earlier rows of the
    same one, have the bits they have without; rows that see one say so."""
    print("[case] masked places", causal, D, dtype, flush=True)
    r = rng(3)
    n = [130, 200, 77]
    cu = [0, 130, 330, 407]
    q, k, v = normal(r, 407, 4, D), normal(r, 407, 2, D), normal(r, 407, 2, D)
    q, k, v = (t.to(DT[dtype]) for t in (q, k, v))
    clean, clean_lse = fp8sm.attention_packed(q, k, v, ints(cu), causal=causal, return_lse=True)
    for bad in (float("nan"), float("inf"), -float("inf")):
        v2, k2 = v.clone(), k.clone()
        v2[130 + 150, 1, 5] = bad          # heads 2, 3 of the second prompt, channel 5
        out, lse = fp8sm.attention_packed(q, k, v2, ints(cu), causal=causal, return_lse=True)
        hit = torch.zeros_like(out, dtype=torch.bool)
        hit[280 if causal else 130:330, 2:, 5] = True
        assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse, clean_lse)
        assert not torch.isfinite(out[hit]).any()
        k2[130 + 150, 0, 3] = bad          # heads 0, 1: those rows' scores
        out, lse = fp8sm.attention_packed(q, k2, v, ints(cu), causal=causal, return_lse=True)
        hit = torch.zeros_like(lse, dtype=torch.bool)
        hit[280 if causal else 130:330, :2] = True
        assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])
        if bad != bad:
            assert torch.isnan(out[hit]).all()
        q2 = q.clone()
        q2[140, 3, 0] = bad
        out = fp8sm.attention_packed(q2, k, v, ints(cu), causal=causal)
        rest = torch.ones(407, 4, dtype=torch.bool, device="cuda")
        rest[140, 3] = False
        assert torch.equal(out[rest], clean[rest])


def test_offsets_that_do_not_ascend_are_clamped():
    """cu is data: whatever it holds, only rows of [0, T) are touched."""
    r = rng(4)
    q, k, v = (normal(r, 50, 2, 64).bfloat16() for _ in range(3))
    for cu in ([-5, 20, 900], [0, 30, 10, 50], [60, 70, 80], [0, 0, 0]):
        print("[case] cu", cu, flush=True)
        out = torch.full((60, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
        fp8sm.attention_packed(q, k, v, ints(cu), out=out[:50])
        assert torch.all(out[50:] == 9)
    want = fp8sm.attention_packed(q[:20], k[:20], v[:20], ints([0, 20]))
    out = torch.full((50, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    fp8sm.attention_packed(q, k, v, ints([-5, 20]), out=out)
    assert torch.equal(out[:20], want) and torch.all(out[20:] == 9)


def test_in_place_streams_and_replayed_graphs():
    r = rng(5)
    Hq, H, D = 8, 2, 128
    rows = normal(r, 333, (Hq + 2 * H) * D).bfloat16()

    def parts(x):
        q, k, v = x.split([Hq * D, H * D, H * D], 1)
        return q.unflatten(1, (Hq, D)), k.unflatten(1, (H, D)), v.unflatten(1, (H, D))

    cu = ints([0, 100, 101, 300])
    want = fp8sm.attention_packed(*parts(rows), cu)
    x = rows.clone()
    q, k, v = parts(x)
    assert fp8sm.attention_packed(q, k, v, cu, out=q) is q
    assert torch.equal(q[:300], want[:300]) and torch.equal(x[:, Hq * D:], rows[:, Hq * D:])
    assert torch.equal(x[300:], rows[300:])
    outs = []
    for st in (torch.cuda.Stream(), torch.cuda.Stream()):
        st.wait_stream(torch.cuda.current_stream())
        outs.append(fp8sm.attention_packed(*parts(rows), cu, stream=st))
    torch.cuda.synchronize()
    assert all(torch.equal(o[:300], want[:300]) for o in outs)
    held, o = cu.clone(), torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fp8sm.attention_packed(*parts(rows), held, out=o)
    for lens in ([0, 100, 101, 300], [0, 1, 2, 3], [0, 0, 333, 333], [0, 150, 200, 280]):
        held.copy_(ints(lens))
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o[:lens[-1]], fp8sm.attention_packed(*parts(rows), ints(lens))[:lens[-1]])
        assert not o[lens[-1]:].any()


# ---------------------------------------------------------------- rotation on several axes

@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 64), (128, 16), (64, 48), (128, 112)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dtype,axes_n,mixed", [("bf16", 3, False), ("fp16", 2, True), ("bf16", 4, True), ("fp16", 1, False)])
def test_rotation_on_axes(D, rot, interleaved, norm, dtype, axes_n, mixed):
    print(f"[case] axes D={D} rot={rot} inter={interleaved} norm={norm} {dtype} {axes_n} {mixed}", flush=True)
    r = rng(rot + axes_n)
    T, Hq, Hk, far = 37, 5, 3, 500
    half = rot // 2
    x = normal(r, T, (Hq + Hk) * D + 8).to(DT[dtype])
    pos = r.integers(0, far, (axes_n, T)).astype(np.int32)
    pos[axes_n - 1, 3], pos[0, 7] = -1, far
    cut = sorted(r.integers(0, half + 1, axes_n - 1).tolist())
    sections = np.diff([0] + cut + [half]).tolist()
    axes = fp8sm.rope_axes(sections, mixed)
    ang = np.arange(far)[:, None] * 100.0 ** (-np.arange(half) / half)
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    w = [(1 + 0.2 * normal(r, D)).to(DT[dtype]) if norm else None for _ in range(2)]
    held = torch.zeros(axes_n, T + 3, dtype=torch.int32, device="cuda")
    held[:, :T] = torch.from_numpy(pos)
    y = torch.full((T, (Hq + Hk) * D + 16), 9.0, dtype=DT[dtype], device="cuda")
    fp8sm.qk_norm_rope_axes(x, Hq, Hk, D, held[:, :T], torch.from_numpy(table).cuda(), axes, *w,
                            interleaved=interleaved, out=y[:, :(Hq + Hk) * D])
    f = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    want, mag = op.norm_rope_axes(f(x), Hq, Hk, D, pos, table, axes, f(w[0]), f(w[1]), interleaved=interleaved)
    got = y[:, :(Hq + Hk) * D].double().cpu().numpy().reshape(want.shape)
    off = np.isnan(want[:, 0, 0])
    assert set(np.nonzero(off)[0]) == {3, 7}
    assert (got[off] == 9).all() and torch.all(y[:, (Hq + Hk) * D:] == 9)
    # fp32 steps: D squares summed, a root, a division, two products, then two products
    # and a sum: (D + 10) roundings of half a step at most; then the result's one
    bound = mag * (D + 10) * 2.0 ** -24 + np.abs(want) * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -11) + 2.0 ** -25
    err = (np.abs(got - want) / bound)[~off].max()
    print(f"[bound] {err:.3f}", flush=True)
    assert err <= 1


def test_equal_positions_are_the_one_axis_rotation_bit_for_bit():
    r = rng(8)
    for T in (0, 1, 300):
        x = torch.empty(T, 26 * 128, dtype=torch.bfloat16, device="cuda").copy_(normal(r, T, 26 * 128))
        pos = ints(r.integers(0, 90, T).tolist())
        ang = torch.rand(90, 64, device="cuda") * 6
        table = torch.cat([ang.cos(), ang.sin()], 1)
        w = normal(r, 128).bfloat16()
        one = fp8sm.qk_norm_rope(x, 22, 4, 128, pos, table, w, w)
        axes = fp8sm.rope_axes([16, 24, 24])
        assert torch.equal(fp8sm.qk_norm_rope_axes(x, 22, 4, 128, pos.expand(3, T), table, axes, w, w), one)
        y = x.clone()
        assert fp8sm.qk_norm_rope_axes(y, 22, 4, 128, pos[None], table, bytes(64), w, w, out=y) is y
        assert torch.equal(y, one)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("causal", [True, False])
def test_a_layer_in_8_bit_integers(causal):
    """Packed prompts from the layer's input to the output projection's output, on one
    stream and as a replayed graph; every step against the oracle on its own inputs."""
    print("[case] layer", causal, flush=True)
    r = rng(21)
    T, hidden, Hq, H, D, far = 210, 512, 8, 2, 64, 100
    cu = [0, 90, 91, 210]
    x = normal(r, T, hidden).bfloat16()
    w1, w2 = normal(r, (Hq + 2 * H) * D, hidden) * 0.05, normal(r, hidden, Hq * D) * 0.05
    qw1, sw1 = fp8sm.quant_int8(w1.bfloat16())
    qw2, sw2 = fp8sm.quant_int8(w2.bfloat16())
    pos = torch.from_numpy(r.integers(0, far, (3, T)).astype(np.int32)).cuda()
    ang = torch.arange(far, device="cuda", dtype=torch.float64)[:, None] * 50.0 ** (-torch.arange(32, device="cuda") / 32)
    table = torch.cat([ang.cos(), ang.sin()], 1).float()
    axes = fp8sm.rope_axes([8, 12, 12])
    one = torch.ones(D, device="cuda").bfloat16()
    starts = ints(cu)

    def layer(x, seen=lambda *a: None):
        qx, sx = fp8sm.quant_int8(x)
        qkv = fp8sm.scaled_mm_int8(qx, qw1, sx, sw1)
        seen("in", qx, sx, qkv.clone())
        fp8sm.qk_norm_rope_axes(qkv, Hq, H, D, pos, table, axes, one, one, out=qkv)
        q, k, v = qkv.split([Hq * D, H * D, H * D], 1)
        q, k, v = q.unflatten(1, (Hq, D)), k.unflatten(1, (H, D)), v.unflatten(1, (H, D))
        o, lse = fp8sm.attention_packed(q, k, v, starts, causal=causal, return_lse=True)
        seen("attn", q, k, v, o, lse)
        qo, so = fp8sm.quant_int8(o.flatten(1))
        y = fp8sm.scaled_mm_int8(qo, qw2, so, sw2)
        seen("out", qo, so, y)
        return y

    stages = {}
    layer(x, lambda name, *a: stages.setdefault(name, a))
    c = lambda t: t.cpu().numpy()  # noqa: E731
    bits = lambda t: c(t.contiguous().view(torch.int16)).view(np.uint16)  # noqa: E731

    def linear(inp, w, sw, codes, scales, out):
        want_q, want_s = oi.quant(c(inp.float()))
        assert np.array_equal(c(codes), want_q) and np.array_equal(c(scales), want_s)
        assert np.array_equal(bits(out), oi.scaled_mm(want_q, c(w), want_s, c(sw)))

    qx, sx, qkv = stages["in"]
    linear(x, qw1, sw1, qx, sx, qkv)
    q, k, v, o, lse = stages["attn"]
    turned, mag = op.norm_rope_axes(c(qkv.double()), Hq, H, D, c(pos), c(table), axes, np.ones(D), np.ones(D))
    got = c(torch.cat([q, k], 1).double())
    assert np.all(np.abs(got - turned) <= mag * (D + 10) * 2.0 ** -24 + np.abs(turned) * 2.0 ** -8 + 2.0 ** -25)
    assert torch.equal(v, qkv[:, (Hq + H) * D:].unflatten(1, (H, D)))
    check(o, lse, q, k, v, cu, D ** -0.5, causal, 0, "bf16")
    linear(o.flatten(1), qw2, sw2, *stages["out"])
    xs = x.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = layer(xs)
    for n in range(4):
        xs.copy_(x.roll(n, 0))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, layer(x.roll(n, 0)))
