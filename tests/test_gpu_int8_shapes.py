"""Seeded random shapes of the scaled int8 product through every kernel variant, bit for
bit, with K tails, strides, batches and live rows; sums in exact integers on the GPU."""
import random

import pytest
import torch

from column_scaled_gemm_amd import fp8sm

pytestmark = pytest.mark.gpu


def exact(a, b, sa, sb, bias, out):
    """The definition in torch: exact sums (products of 2^14 in float64), then fp32 steps
    that are each rounded, then one rounding to `out`."""
    y = (a.double() @ b.double().T.contiguous()).float()
    y = (y * sa[:, None]) * sb
    if bias is not None:
        y = y + bias.float()
    return y.to(out)


# rows and columns that lead to each tile of the dispatch, and to its edges
KINDS = {"few16": ((1, 16), (8, 9000)), "few32": ((17, 32), (8, 4096)), "64x32": ((33, 128), (8, 4096)),
         "64x64": ((33, 64), (5000, 16000)), "64x128": ((65, 400), (4000, 9000)), "128x64": ((257, 384), (4600, 5376)),
         "128x128": ((200, 900), (1000, 6000)), "128x128 many": ((1500, 2500), (2000, 4200)),
         "256x256": ((2500, 3500), (5000, 9000))}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("seed", range(4))
def test_random_shapes(kind, seed):
    r = random.Random(f"{kind} {seed}")
    (m0, m1), (n0, n1) = KINDS[kind]
    M, N = r.randint(m0, m1), 8 * r.randint(n0 // 8, n1 // 8)
    K = 16 * r.randint(1, 40 if kind == "256x256" else 160)
    out = r.choice([torch.bfloat16, torch.float16])
    print(f"[case] {kind} {M}x{N}x{K} {out}", flush=True)
    g = torch.Generator("cuda").manual_seed(seed)

    def codes(rows):
        pad = r.choice([0, 16, 64])
        return torch.randint(-128, 128, (rows, K + pad), generator=g, device="cuda", dtype=torch.int8)[:, :K]

    a, b = codes(M), codes(N)
    sa = torch.rand(M, generator=g, device="cuda") * 1e-3
    sb = torch.rand(N, generator=g, device="cuda")
    bias = torch.randn(N, generator=g, device="cuda").to(out) if r.random() < 0.5 else None
    c = torch.full((M, N + 8), 3.0, dtype=out, device="cuda")
    fp8sm.scaled_mm_int8(a, b, sa, sb, c=c[:, :N], bias=bias)
    assert torch.equal(c[:, :N], exact(a, b, sa, sb, bias, out))
    assert (c[:, N:] == 3).all()


@pytest.mark.parametrize("M,N,E", [(16, 256, 7), (32, 128, 5), (60, 512, 9), (128, 1024, 32), (200, 640, 3), (300, 2048, 20)])
def test_random_batches(M, N, E):
    r = random.Random(M + N)
    K = 16 * r.randint(3, 70)
    print(f"[case] {E} x {M}x{N}x{K}", flush=True)
    g = torch.Generator("cuda").manual_seed(M)
    a = torch.randint(-128, 128, (E, M, K), generator=g, device="cuda", dtype=torch.int8)
    b = torch.randint(-128, 128, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
    sa, sb = (torch.rand(E, n, generator=g, device="cuda") * 0.01 for n in (M, N))
    live = [r.choice([0, 1, M, r.randint(0, M)]) for _ in range(E)]
    c = torch.full((E, M, N), 3.0, dtype=torch.bfloat16, device="cuda")
    fp8sm.scaled_mm_int8(a, b, sa, sb, rows=torch.tensor(live, dtype=torch.int32, device="cuda"), c=c)
    for e, n in enumerate(live):
        assert torch.equal(c[e, :n], exact(a[e], b[e], sa[e], sb[e], None, torch.bfloat16)[:n])
        assert (c[e, n:] == 3).all()
