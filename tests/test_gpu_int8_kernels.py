"""Every kernel of the int8 product by name, bit for bit: its ring filled once, walked in
the steady loop, and ended by a tail of K; odd rows and columns, strides, batches with live rows."""
import random

import pytest
import torch

from column_scaled_gemm_amd import fp8sm
from test_gpu_int8_shapes import exact
from test_int8_kernels import SIZES, lengths

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [0, 1])
@pytest.mark.parametrize("name", SIZES)
def test_every_kernel(name, size):
    B, M, N = SIZES[name][size]
    assert fp8sm.int8_kernel(B, M, N) == name
    r = random.Random(f"{name} {size}")
    g = torch.Generator("cuda").manual_seed(size)
    for K in lengths(name):
        out = r.choice([torch.bfloat16, torch.float16])
        print(f"[case] {name} {B} x {M}x{N}x{K} {out}", flush=True)

        def codes(rows):
            pad = r.choice([0, 16, 64])
            return torch.randint(-128, 128, (B, rows, K + pad), generator=g, device="cuda", dtype=torch.int8)[..., :K]

        a, b = codes(M), codes(N)
        sa = torch.rand(B, M, generator=g, device="cuda") * 1e-3
        sb = torch.rand(B, N, generator=g, device="cuda")
        bias = torch.randn(N, generator=g, device="cuda").to(out) if r.random() < 0.5 else None
        live = [r.choice([0, 1, M, r.randint(0, M)]) for _ in range(B - 1)] + [M]
        rows = torch.tensor(live, dtype=torch.int32, device="cuda") if B > 1 else None
        c = torch.full((B, M, N + 8), 3.0, dtype=out, device="cuda")
        fp8sm.scaled_mm_int8(a, b, sa, sb, rows=rows, c=c[..., :N], bias=bias)
        for e, n in enumerate(live):
            assert torch.equal(c[e, :n, :N], exact(a[e, :n], b[e], sa[e, :n], sb[e], bias, out))
            assert (c[e, n:] == 3).all()
        assert (c[..., N:] == 3).all()
