"""Packed attention of so many heads that their keys outgrow the caches, which orders the
workgroups another way: the bits of the same heads in smaller calls."""
import pytest
import torch

from column_scaled_gemm_amd import fp8sm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,G,n,D,causal", [(1024, 1, [700], 128, True), (1000, 1, [1500, 20], 128, True),
                                            (240, 3, [3000, 2500], 128, False), (1000, 1, [1500], 64, True)])
def test_many_heads_of_many_tokens(H, G, n, D, causal):
    print("[case] heads", H, G, n, D, causal, flush=True)
    T = sum(n) + 3
    assert T // len(n) * H * D * 4 > 5 << 26
    g = torch.Generator("cuda").manual_seed(H)
    q, k, v = (torch.randn(T, h, D, generator=g, device="cuda", dtype=torch.float32).bfloat16() for h in (H * G, H, H))
    cu = torch.tensor([0] + n, device="cuda").cumsum(0).int()
    out = torch.full_like(q, 9.0)
    _, lse = fp8sm.attention_packed(q, k, v, cu, causal=causal, out=out, return_lse=True)
    assert (out[-3:] == 9).all()
    for h in range(0, H, 64):
        e = min(h + 64, H)
        part = [t.contiguous() for t in (q[:, h * G:e * G], k[:, h:e], v[:, h:e])]
        o, l = fp8sm.attention_packed(*part, cu, causal=causal, return_lse=True)
        assert torch.equal(out[:-3, h * G:e * G], o[:-3]) and torch.equal(lse[:-3, h * G:e * G], l[:-3])
