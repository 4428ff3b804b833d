"""Refusals of packed attention and of rotation on several axes, on the host before
any launch (no GPU needed)."""
import ctypes
import os

import pytest
import torch

from conftest import ROOT

LIB = os.path.join(ROOT, "column_scaled_gemm_amd", "libfp8sm.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libfp8sm.so not built")
P = ctypes.c_void_p


def _codes():
    from column_scaled_gemm_amd import fp8sm
    return fp8sm.lib(), {v: k for k, v in fp8sm.STATUS.items()}


def _attn(lib, **kw):
    a = dict(q=16, ldq=256, k=16, ldk=128, v=16, ldv=128, dt=0, T=4, B=2, Hq=4, H=2, D=64, cu=4, scale=0.125,
             flags=1, window=0, o=16, ldo=256, lse=0)
    a.update(kw)
    return lib.fp8sm_attention_packed(P(a["q"]), a["ldq"], P(a["k"]), a["ldk"], P(a["v"]), a["ldv"], a["dt"], a["T"],
                                      a["B"], a["Hq"], a["H"], a["D"], P(a["cu"]), a["scale"], a["flags"],
                                      a["window"], P(a["o"]), a["ldo"], P(a["lse"]), P(0))


@pytest.mark.parametrize("kw,err", [
    (dict(dt=2), "UNSUPPORTED"), (dict(flags=2), "UNSUPPORTED"), (dict(D=96), "UNSUPPORTED"),
    (dict(window=4, flags=0), "UNSUPPORTED"), (dict(T=-1), "SHAPE"), (dict(B=-1), "SHAPE"), (dict(H=0), "SHAPE"),
    (dict(Hq=0), "SHAPE"), (dict(Hq=3), "SHAPE"), (dict(window=-1), "SHAPE"), (dict(scale=float("nan")), "SHAPE"),
    (dict(scale=float("inf")), "SHAPE"), (dict(ldq=248), "SHAPE"), (dict(ldk=120), "SHAPE"),
    (dict(ldv=120), "SHAPE"), (dict(ldo=248), "SHAPE"), (dict(T=(1 << 23) + 1), "RANGE"),
    (dict(B=(1 << 20) + 1), "RANGE"), (dict(Hq=1026, ldq=1 << 17, ldo=1 << 17), "RANGE"),
    (dict(T=1 << 23, Hq=256, ldq=1 << 15, ldo=1 << 15), "RANGE"), (dict(ldk=(1 << 23) + 8), "RANGE"),
    (dict(ldv=(1 << 23) + 8), "RANGE"), (dict(ldq=260), "ALIGN"), (dict(ldk=132), "ALIGN"),
    (dict(ldv=132), "ALIGN"), (dict(ldo=260), "ALIGN"), (dict(q=0), "NULL"), (dict(k=0), "NULL"),
    (dict(v=0), "NULL"), (dict(cu=0), "NULL"), (dict(o=0), "NULL"), (dict(q=8), "ALIGN"), (dict(k=8), "ALIGN"),
    (dict(v=8), "ALIGN"), (dict(o=8), "ALIGN"), (dict(cu=2), "ALIGN"), (dict(lse=2), "ALIGN")])
def test_attention_refusals(kw, err):
    lib, E = _codes()
    assert _attn(lib, **kw) == E["ERR_" + err]


def test_attention_of_nothing_is_ok():
    lib, E = _codes()
    assert _attn(lib, T=0, q=0) == _attn(lib, B=0, cu=0) == E["OK"]


def _rope(lib, axes=bytes([0, 1] * 16), **kw):
    a = dict(x=16, dt=0, T=4, Hq=2, Hk=1, D=64, ldx=192, wq=16, wk=16, cs=16, mp=8, pos=4, ldp=4, n=2, rot=64,
             flags=0, y=4096, ldy=192)
    a.update(kw)
    return lib.fp8sm_qk_norm_rope_axes(P(a["x"]), a["dt"], a["T"], a["Hq"], a["Hk"], a["D"], a["ldx"], P(a["wq"]),
                                       P(a["wk"]), 1e-6, P(a["cs"]), a["mp"], P(a["pos"]), a["ldp"], a["n"], axes,
                                       a["rot"], a["flags"], P(a["y"]), a["ldy"], P(0))


@pytest.mark.parametrize("kw,err", [
    (dict(n=0), "SHAPE"), (dict(n=5), "RANGE"), (dict(ldp=3), "SHAPE"), (dict(axes=bytes([0, 2] * 16)), "SHAPE"),
    (dict(axes=None), "NULL"), (dict(rot=-16), "SHAPE"), (dict(rot=80, axes=bytes(40)), "SHAPE"),
    (dict(rot=24, axes=bytes(12)), "SHAPE"), (dict(rot=1 << 20), "SHAPE"), (dict(dt=2), "UNSUPPORTED"),
    (dict(flags=2), "UNSUPPORTED"), (dict(D=96), "UNSUPPORTED"), (dict(T=-1), "SHAPE"), (dict(ldx=184), "SHAPE"),
    (dict(y=16, ldy=256), "SHAPE"), (dict(ldx=196), "ALIGN"), (dict(pos=2), "ALIGN"), (dict(cs=8), "ALIGN"),
    (dict(pos=0), "NULL"), (dict(cs=0), "NULL"), (dict(wk=0), "NULL"), (dict(T=(1 << 24) + 1, ldp=1 << 25), "RANGE")])
def test_rope_refusals(kw, err):
    lib, E = _codes()
    assert _rope(lib, **kw) == E["ERR_" + err]


def test_rope_of_nothing_is_ok():
    lib, E = _codes()
    assert _rope(lib, T=0, x=0) == E["OK"]


def test_sections():
    from column_scaled_gemm_amd import fp8sm
    assert fp8sm.rope_axes([2, 3, 1]) == [0, 0, 1, 1, 1, 2]
    assert fp8sm.rope_axes([3, 2, 1], mixed=True) == [0, 1, 2, 0, 1, 0]
    assert fp8sm.rope_axes([0, 2], mixed=True) == [1, 1] and fp8sm.rope_axes([]) == []


def test_binding_refuses_what_the_abi_cannot_see():
    from column_scaled_gemm_amd import fp8sm
    i32 = torch.int32
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    k = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    cu = torch.zeros(3, dtype=i32)
    with pytest.raises(fp8sm.DeviceTensorError):
        fp8sm.attention_packed(q, k, k, cu)
    for args, kw in (((q.flatten(1), k, k, cu), {}), ((q, k[:4], k, cu), {}), ((q, k, k[:4], cu), {}),
                     ((q, k.half(), k, cu), {}), ((q, k, k[:, :1], cu), {}), ((q, k, k, cu[:0]), {}),
                     ((q, k, k, cu[None]), {}), ((q.transpose(0, 1), k, k, cu), {}), ((q, k, k, cu), dict(out=q[:4])),
                     ((q, k, k, cu), dict(out=q.half())), ((q, k, k, cu), dict(lse=torch.zeros(5, 3)))):
        with pytest.raises(ValueError):
            fp8sm.attention_packed(*args, **kw)
    with pytest.raises(TypeError):
        fp8sm.attention_packed(q, k, k, cu.long())
    with pytest.raises(TypeError):
        fp8sm.attention_packed(q, k, k, cu, lse=torch.zeros(5, 4).double())
    x, t = torch.zeros(5, 192, dtype=torch.bfloat16), torch.zeros(8, 64)
    pos, axes = torch.zeros(2, 5, dtype=i32), [0, 1] * 16
    with pytest.raises(fp8sm.DeviceTensorError):
        fp8sm.qk_norm_rope_axes(x, 2, 1, 64, pos, t, axes)
    for args in ((pos[:, :4], t, axes), (pos[0], t, axes), (pos, t, axes[:31]), (pos, t[0], axes),
                 (pos.T.contiguous().T, t, axes), (pos, t, [0, 256] * 16)):
        with pytest.raises(ValueError):
            fp8sm.qk_norm_rope_axes(x, 2, 1, 64, *args)
    with pytest.raises(ValueError):
        fp8sm.qk_norm_rope_axes(x, 3, 1, 64, pos, t, axes)
    for args in ((pos.long(), t, axes), (pos, t.double(), axes)):
        with pytest.raises(TypeError):
            fp8sm.qk_norm_rope_axes(x, 2, 1, 64, *args)
