"""Int8 quant and the scaled int8 product against the oracle, bit for bit: every
step of their definitions is a correctly rounded one, so nothing may differ."""
import numpy as np
import pytest
import torch

from column_scaled_gemm_amd import fp8sm, inputs
from oracle import int8 as oi, quant as oq

pytestmark = pytest.mark.gpu
F32 = np.float32
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
TEN, ROW, COL = fp8sm.KIND_TENSOR, fp8sm.KIND_ROW, fp8sm.KIND_COL
SENT8, SENT16 = 0x5A, 0x7FC1


def case(*what):
    print("[case]", *what, flush=True)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bits16(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def views(t, pad=8):
    """t inside a larger buffer: other row and batch strides than its shape's."""
    shape = list(t.shape)
    shape[-1] += pad
    if len(shape) == 3:
        shape[-2] += 1
    big = torch.zeros(shape, dtype=t.dtype, device="cuda")
    v = big[..., :t.shape[-1]]
    if len(shape) == 3:
        v = v[:, :-1]
    v.copy_(t)
    return v


# ---------------------------------------------------------------- quant

# K: one and two chunks a lane, four wavefronts a row with 1, 2, 3, 4, 6, 8 chunks, two passes
KS = [8, 504, 520, 1016, 1032, 2056, 4096, 4104, 5376, 8192, 8200, 14336, 16384, 16392]


@pytest.mark.parametrize("K", KS)
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_quant_is_the_oracle(K, fused, dtype):
    case("quant", K, fused, dtype)
    r = inputs.rng(K + fused)
    M = 7
    x = r.standard_normal((M, K * (1 + fused))).astype(F32)
    x[:, ::97] *= 20
    x[1] = 0
    x[2] *= F32(1e-6)
    t = inputs.to_dtype(x, DT[dtype])
    y = inputs.widen(t)
    want_q, want_s = oi.quant(oq.silu_mul_f32(y) if fused else y)
    q, s = fp8sm.quant_int8(t.cuda(), fuse_silu_mul=fused)
    assert q.dtype == torch.int8 and q.shape == (M, K) and s.shape == (M,)
    assert np.array_equal(q.cpu().numpy(), want_q) and np.array_equal(s.cpu().numpy(), want_s)
    # strided in and out, on a stream of its own
    out = views(torch.full((M, K), SENT8, dtype=torch.int8), 16)
    xs = views(t)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    q2, s2 = fp8sm.quant_int8(xs, fuse_silu_mul=fused, q=out, stream=stream)
    torch.cuda.synchronize()
    assert q2 is out and torch.equal(q2, q) and torch.equal(s2, s)


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("K", [64, 2048, 16400])
def test_quant_batches_leave_other_rows(K, fused, dtype):
    case("quant batched", K, fused, dtype)
    B, M = 6, 5
    rows = [0, 5, -3, 2, 99, 1]
    r = inputs.rng(K)
    t = inputs.to_dtype(r.standard_normal((B, M, K * (1 + fused))).astype(F32), DT[dtype])
    y = inputs.widen(t)
    q = torch.full((B, M, K), SENT8, dtype=torch.int8, device="cuda")
    s = torch.full((B, M), 7.0, device="cuda")
    fp8sm.quant_int8(views(t), fuse_silu_mul=fused, rows=torch.tensor(rows, dtype=torch.int32, device="cuda"),
                     q=q, scales=s)
    q, s = q.cpu().numpy(), s.cpu().numpy()
    for b in range(B):
        n = min(max(rows[b], 0), M)
        yb = y[b].reshape(M, -1)
        want_q, want_s = oi.quant(oq.silu_mul_f32(yb) if fused else yb)
        assert np.array_equal(q[b, :n], want_q[:n]) and np.array_equal(s[b, :n], want_s[:n])
        assert (q[b, n:] == SENT8).all() and (s[b, n:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_quant_of_every_gate(dtype):
    """silu of every finite 16-bit gate times 1, through rows whose scale shows it:
    each row pairs one gate with nothing, so the scale is |silu| / 127."""
    case("every gate", dtype)
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    g = torch.from_numpy(bits.view(np.int16).copy()).view(DT[dtype])
    g = g[torch.isfinite(g.float())]
    x = torch.zeros(g.numel(), 16, dtype=DT[dtype])
    x[:, 0] = g
    x[:, 8] = 1
    want_q, want_s = oi.quant(oq.silu_mul_f32(inputs.widen(x)))
    q, s = fp8sm.quant_int8(x.cuda(), fuse_silu_mul=True)
    assert np.array_equal(s.cpu().numpy(), want_s) and np.array_equal(q.cpu().numpy(), want_q)


@pytest.mark.parametrize("K", [64, 1024, 2048, 16400])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_quant_of_values_that_are_not_finite(K, dtype):
    case("not finite", K, dtype)
    r = inputs.rng(5)
    x = r.standard_normal((9, K)).astype(F32)
    for i, bad in enumerate(([np.inf], [-np.inf], [np.nan], [np.inf, np.nan], [-np.nan, -np.inf, np.inf])):
        for k, v in enumerate(bad):
            x[i, (i * 37 + k * 11) % K] = v
    x[5] = np.inf
    x[6] = np.nan
    x[7, -1] = -np.inf
    t = inputs.to_dtype(x, DT[dtype])
    want_q, want_s = oi.quant(inputs.widen(t))
    q, s = fp8sm.quant_int8(t.cuda())
    assert np.array_equal(s.cpu().numpy(), want_s) and np.array_equal(q.cpu().numpy(), want_q)
    g = inputs.to_dtype(np.concatenate([x, np.ones_like(x)], 1), DT[dtype])
    with np.errstate(invalid="ignore"):
        want_q, want_s = oi.quant(oq.silu_mul_f32(inputs.widen(g)))
    q, s = fp8sm.quant_int8(g.cuda(), fuse_silu_mul=True)
    assert np.array_equal(s.cpu().numpy(), want_s) and np.array_equal(q.cpu().numpy(), want_q)


# ---------------------------------------------------------------- product

def codes(r, *shape):
    c = np.clip(np.rint(r.standard_normal(shape) * 50), -128, 127).astype(np.int8)
    c.reshape(-1)[::41] = -128
    return c


def scales(r, n, unit):
    return ((0.5 + r.random(n)) * unit).astype(F32)


MNK = [(1, 8, 16), (1, 4096, 4096), (3, 40, 272), (15, 136, 528), (16, 256, 2048), (17, 72, 1008),
       (31, 264, 4112), (33, 96, 512), (48, 48, 2064), (64, 200, 14336), (65, 64, 64), (65, 136, 80),
       (100, 264, 1040), (128, 128, 16), (129, 384, 2000), (257, 520, 336), (300, 1000, 4096)]


@pytest.mark.parametrize("M,N,K", MNK)
@pytest.mark.parametrize("out", ["bf16", "fp16"])
def test_product_is_the_oracle(M, N, K, out):
    case("product", M, N, K, out)
    r = inputs.rng(M + N + K)
    a, b = codes(r, M, K), codes(r, N, K)
    sa, sb = scales(r, M, 0.02), scales(r, N, 0.003)
    bias = inputs.to_dtype(r.standard_normal(N).astype(F32), DT[out])
    c = fp8sm.scaled_mm_int8(dev(a), dev(b), dev(sa), dev(sb), out_dtype=DT[out])
    assert np.array_equal(bits16(c), oi.scaled_mm(a, b, sa, sb, out=out))
    # strided operands, a bias, scalar scales, an output with room beside the rows
    big = torch.full((M, N + 8), 3.0, dtype=DT[out], device="cuda")
    c = fp8sm.scaled_mm_int8(views(dev(a), 16), views(dev(b), 48), dev(sa[:1]), dev(sb[:1]), TEN, TEN,
                             c=big[:, :N], bias=bias.cuda())
    assert np.array_equal(bits16(c), oi.scaled_mm(a, b, sa[:1], sb[:1], inputs.widen(bias), out))
    assert (big[:, N:] == 3).all()


@pytest.mark.parametrize("M,N", [(5, 64), (200, 256)])
def test_largest_sums_are_exact(M, N):
    case("largest sums", M, N)
    K = 65536
    a = np.full((M, K), -128, dtype=np.int8)
    b = np.full((N, K), -128, dtype=np.int8)
    b[1::2] = 127
    b[3, :99] = 1
    one = np.ones(1, dtype=F32)
    c = fp8sm.scaled_mm_int8(dev(a), dev(b), dev(one * F32(2.0 ** -20)), dev(one), TEN, TEN)
    assert np.array_equal(bits16(c), oi.scaled_mm(a[:1], b, one * F32(2.0 ** -20), one).repeat(M, 0))


@pytest.mark.parametrize("M,N,K", [(3, 64, 272), (40, 136, 512), (130, 264, 2048), (128, 512, 64)])
@pytest.mark.parametrize("shared", [False, True])
def test_batches_with_live_rows(M, N, K, shared):
    case("batches", M, N, K, shared)
    B = 5
    rows = [M, 0, -1, M // 2 + 1, 10 ** 6]
    r = inputs.rng(M)
    a = codes(r, B, M, K)
    b = codes(r, N, K) if shared else codes(r, B, N, K)
    sa, sb = scales(r, (B, M), 0.02), scales(r, N if shared else (B, N), 0.003)
    c = torch.full((B, M, N), 1, dtype=torch.int16, device="cuda").fill_(SENT16).view(torch.bfloat16)
    fp8sm.scaled_mm_int8(views(dev(a), 16), dev(b), dev(sa), dev(sb),
                         rows=torch.tensor(rows, dtype=torch.int32, device="cuda"), c=c)
    got = bits16(c)
    for e in range(B):
        n = min(max(rows[e], 0), M)
        want = oi.scaled_mm(a[e], b if shared else b[e], sa[e], sb if shared else sb[e])
        assert np.array_equal(got[e, :n], want[:n]) and (got[e, n:] == SENT16).all()


def test_no_k_and_no_rows():
    bias = torch.randn(24, device="cuda").half()
    one = torch.ones(1, device="cuda")
    e = lambda *s: torch.empty(*s, dtype=torch.int8, device="cuda")  # noqa: E731
    c = fp8sm.scaled_mm_int8(e(5, 0), e(24, 0), one, one, TEN, TEN, bias=bias, out_dtype=torch.float16)
    assert torch.equal(c, bias.expand(5, 24))
    assert fp8sm.scaled_mm_int8(e(0, 32), e(24, 32), one[:0], one.expand(24).contiguous()).shape == (0, 24)
    assert fp8sm.scaled_mm_int8(e(4, 32), e(0, 32), one.expand(4).contiguous(), one[:0]).shape == (4, 0)
    q, s = fp8sm.quant_int8(torch.empty(0, 64, device="cuda").half())
    assert q.shape == (0, 64) and s.shape == (0,)


def test_rows_do_not_depend_on_the_batch_they_are_in():
    """A row alone, in a small batch and in a large one goes through different kernels."""
    r = inputs.rng(9)
    a, b = codes(r, 700, 1040), codes(r, 9000, 1040)
    sa, sb = scales(r, 700, 0.02), scales(r, 9000, 0.003)
    a, b, sa, sb = dev(a), dev(b), dev(sa), dev(sb)
    every = fp8sm.scaled_mm_int8(a, b, sa, sb)
    for n in (1, 16, 17, 40, 64, 65, 200, 600):
        case("rows", n)
        assert torch.equal(fp8sm.scaled_mm_int8(a[:n], b, sa[:n].contiguous(), sb), every[:n])
    for cols in (8, 40, 1000):
        assert torch.equal(fp8sm.scaled_mm_int8(a, b[:cols], sa, sb[:cols].contiguous()), every[:, :cols])


def test_two_streams_and_a_replayed_graph():
    r = inputs.rng(13)
    x = inputs.to_dtype(r.standard_normal((20, 1024)).astype(F32)).cuda()
    w = dev(codes(r, 512, 1024))
    sw = dev(scales(r, 512, 0.003))

    def step(x, q, s, c):
        fp8sm.quant_int8(x, q=q, scales=s)
        return fp8sm.scaled_mm_int8(q, w, s, sw, c=c)

    def room():
        return (torch.empty(20, 1024, dtype=torch.int8, device="cuda"), torch.empty(20, device="cuda"),
                torch.empty(20, 512, dtype=torch.bfloat16, device="cuda"))

    want = step(x, *room()).clone()
    torch.cuda.synchronize()
    outs, streams = [room(), room()], [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for o, st in zip(outs, streams):
            with torch.cuda.stream(st):
                step(x, *o)
    torch.cuda.synchronize()
    assert all(torch.equal(o[2], want) for o in outs)
    xs, o = x.clone(), room()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(xs, *o)
    for k in range(4):
        xs.copy_(x * (k + 1))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o[2], step(xs.clone(), *room()))
