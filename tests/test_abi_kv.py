"""Refusals of the cache and attention calls, on the host before any launch (no
GPU needed), and the workspace query."""
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


def _rope(lib, **kw):
    a = dict(x=16, dt=0, T=4, Hq=2, Hk=1, D=64, ldx=192, wq=16, wk=16, cs=16, mp=8, pos=4, rot=64,
             flags=0, y=4096, ldy=192)
    a.update(kw)
    return lib.fp8sm_qk_norm_rope(P(a["x"]), a["dt"], a["T"], a["Hq"], a["Hk"], a["D"], a["ldx"],
                                  P(a["wq"]), P(a["wk"]), 1e-6, P(a["cs"]), a["mp"], P(a["pos"]),
                                  a["rot"], a["flags"], P(a["y"]), a["ldy"], P(0))


@pytest.mark.parametrize("kw,err", [
    (dict(dt=2), "UNSUPPORTED"), (dict(flags=2), "UNSUPPORTED"), (dict(D=96), "UNSUPPORTED"),
    (dict(T=-1), "SHAPE"), (dict(Hq=0, Hk=0), "SHAPE"), (dict(Hq=-1), "SHAPE"),
    (dict(rot=80), "SHAPE"), (dict(rot=24), "SHAPE"), (dict(rot=-16), "SHAPE"),
    (dict(mp=-1), "SHAPE"), (dict(ldx=184), "SHAPE"), (dict(ldy=184), "SHAPE"),
    (dict(y=16, ldy=256), "SHAPE"), (dict(ldx=196), "ALIGN"), (dict(x=8), "ALIGN"),
    (dict(y=4104), "ALIGN"), (dict(wq=8), "ALIGN"), (dict(cs=8), "ALIGN"), (dict(pos=2), "ALIGN"),
    (dict(x=0), "NULL"), (dict(y=0), "NULL"), (dict(wq=0), "NULL"), (dict(wk=0), "NULL"),
    (dict(cs=0), "NULL"), (dict(pos=0), "NULL"), (dict(T=(1 << 24) + 1), "RANGE"),
    (dict(Hq=1025, ldx=1 << 17, ldy=1 << 17), "RANGE"), (dict(mp=(1 << 30) + 1), "RANGE")])
def test_rope_refusals(kw, err):
    lib, E = _codes()
    assert _rope(lib, **kw) == E["ERR_" + err]


def test_rope_of_nothing_is_ok():
    lib, E = _codes()
    assert _rope(lib, T=0, x=0, y=0) == E["OK"]


KV = dict(T=4, B=2, cu=4, lens=4, table=4, ldt=8, nb=8, P=32, H=2, D=64, block=16, k=16, v=16, ke=1,
          ve=1)
COMMON = [
    (dict(T=-1), "SHAPE"), (dict(B=-1), "SHAPE"), (dict(H=0), "SHAPE"), (dict(P=0), "SHAPE"),
    (dict(nb=0), "SHAPE"), (dict(ldt=7), "SHAPE"), (dict(D=96), "UNSUPPORTED"),
    (dict(block=48), "UNSUPPORTED"), (dict(block=8), "UNSUPPORTED"), (dict(block=256), "UNSUPPORTED"),
    (dict(T=(1 << 24) + 1), "RANGE"), (dict(B=(1 << 20) + 1), "RANGE"), (dict(P=1 << 31), "RANGE"),
    (dict(H=1025), "RANGE"), (dict(nb=(1 << 26) + 1, ldt=1 << 27), "RANGE"), (dict(cu=0), "NULL"), (dict(lens=0), "NULL"),
    (dict(table=0), "NULL"), (dict(k=0), "NULL"), (dict(v=0), "NULL"), (dict(ke=0), "NULL"),
    (dict(ve=0), "NULL"), (dict(cu=2), "ALIGN"), (dict(lens=6), "ALIGN"), (dict(table=5), "ALIGN"),
    (dict(k=8), "ALIGN"), (dict(v=24), "ALIGN")]


def _write(lib, **kw):
    a = dict(KV, x=16, y=16, ldx=128, ldy=128, dt=0)
    a.update(kw)
    return lib.fp8sm_kv_cache_write(P(a["x"]), a["ldx"], P(a["y"]), a["ldy"], a["dt"], a["T"], a["B"],
                                    P(a["cu"]), P(a["lens"]), P(a["table"]), a["ldt"], a["nb"], a["P"],
                                    a["H"], a["D"], a["block"], P(a["k"]), P(a["v"]), P(a["ke"]),
                                    P(a["ve"]), P(0))


def _read(lib, **kw):
    a = dict(KV, x=16, y=16, ldx=128, ldy=128, dt=0)
    a.update(kw)
    return lib.fp8sm_kv_cache_read(P(a["k"]), P(a["v"]), P(a["ke"]), P(a["ve"]), a["P"], a["H"], a["D"],
                                   a["block"], a["T"], a["B"], P(a["cu"]), P(a["lens"]), P(a["table"]),
                                   a["ldt"], a["nb"], a["dt"], P(a["x"]), a["ldx"], P(a["y"]), a["ldy"],
                                   P(0))


def _attn(lib, **kw):
    a = dict(KV, q=16, ldq=256, dt=0, Hq=4, mq=2, mkv=64, flags=1, window=0, o=16, ldo=256, lse=0, ws=0,
             wsb=0)
    a.update(kw)
    return lib.fp8sm_attention_cache(P(a["q"]), a["ldq"], a["dt"], a["T"], a["B"], a["Hq"], P(a["cu"]),
                                     P(a["lens"]), P(a["table"]), a["ldt"], a["nb"], P(a["k"]), P(a["v"]),
                                     P(a["ke"]), P(a["ve"]), a["P"], a["H"], a["D"], a["block"], a["mq"],
                                     a["mkv"], 0.125, a["flags"], a["window"], P(a["o"]), a["ldo"],
                                     P(a["lse"]), P(a["ws"]), a["wsb"], P(0))


@pytest.mark.parametrize("call", [_write, _read, _attn])
@pytest.mark.parametrize("kw,err", COMMON)
def test_common_refusals(call, kw, err):
    lib, E = _codes()
    assert call(lib, **kw) == E["ERR_" + err]


@pytest.mark.parametrize("call", [_write, _read, _attn])
def test_empty_batches_are_ok(call):
    lib, E = _codes()
    assert call(lib, T=0) == E["OK"] and call(lib, B=0) == E["OK"]


@pytest.mark.parametrize("call", [_write, _read])
@pytest.mark.parametrize("kw,err", [
    (dict(dt=2), "UNSUPPORTED"), (dict(ldx=120), "SHAPE"), (dict(ldy=120), "SHAPE"),
    (dict(ldx=132), "ALIGN"), (dict(ldy=132), "ALIGN"), (dict(x=8), "ALIGN"), (dict(y=8), "ALIGN")])
def test_row_refusals(call, kw, err):
    lib, E = _codes()
    assert call(lib, **kw) == E["ERR_" + err]


def test_write_needs_both_and_read_takes_either():
    lib, E = _codes()
    assert _write(lib, x=0) == _write(lib, y=0) == E["ERR_NULL"]
    assert _read(lib, x=0, y=0) == E["OK"]


@pytest.mark.parametrize("kw,err", [
    (dict(dt=2), "UNSUPPORTED"), (dict(flags=2), "UNSUPPORTED"), (dict(Hq=3), "SHAPE"),
    (dict(Hq=0), "SHAPE"), (dict(window=-1), "SHAPE"), (dict(window=4, flags=0), "UNSUPPORTED"),
    (dict(mq=0), "SHAPE"), (dict(mkv=-1), "SHAPE"), (dict(ldq=248), "SHAPE"), (dict(ldo=248), "SHAPE"),
    (dict(ldq=260), "ALIGN"), (dict(ldo=260), "ALIGN"), (dict(q=8), "ALIGN"), (dict(o=8), "ALIGN"),
    (dict(lse=2), "ALIGN"), (dict(q=0), "NULL"), (dict(o=0), "NULL"),
    (dict(T=1 << 24, Hq=128, ldq=1 << 14, ldo=1 << 14), "RANGE"), (dict(Hq=1026, ldq=1 << 17, ldo=1 << 17), "RANGE")])
def test_attention_refusals(kw, err):
    lib, E = _codes()
    assert _attn(lib, **kw) == E["ERR_" + err]


def test_attention_workspace():
    from column_scaled_gemm_amd import fp8sm
    lib, E = _codes()
    need = fp8sm.attention_cache_workspace(4, 2, 4, 2, 64, 2, 100000)
    assert need > 0 and need % (4 * 4 * (64 + 2) * 4) == 0   # splits x rows x heads x (D + 2) floats
    big = dict(mkv=100000)
    assert _attn(lib, **big) == E["ERR_NULL"]
    assert _attn(lib, ws=16, wsb=need - 1, **big) == E["ERR_SHAPE"]
    assert _attn(lib, ws=8, wsb=need, **big) == E["ERR_ALIGN"]
    assert fp8sm.attention_cache_workspace(4, 2, 4, 2, 64, 2, 64) == 0
    for bad in [(0, 2, 4, 2, 64, 2, 64), (4, 2, 3, 2, 64, 2, 64), (4, 2, 4, 2, 96, 2, 64),
                (4, 2, 4, 2, 64, 0, 64), (4, 2, 4, 2, 64, 1, -1)]:
        assert fp8sm.attention_cache_workspace(*bad) == 0
    # no sizes overflow the plan
    assert fp8sm.attention_cache_workspace(1, 1, 1, 1, 64, 1 << 62, 1 << 62) > 0


@pytest.mark.parametrize("T,B,H", [(1, 1 << 20, 1), (1, 1 << 20, 1024), (1000, 1 << 17, 8), (64, 4096, 8)])
def test_splits_fit_a_grid_with_more_sequences_than_rows(T, B, H):
    """Every sequence has a slot for each head and split; a grid has 65536 x 65535."""
    from column_scaled_gemm_amd import fp8sm
    need = fp8sm.attention_cache_workspace(T, B, H, H, 64, 1, 1 << 30)
    splits = max(1, need // (T * H * (64 + 2) * 4))
    assert (T // 16 + B) * (H * splits + 1) <= 65536 * 65535


def test_binding_refuses_what_the_abi_cannot_see():
    from column_scaled_gemm_amd import fp8sm
    c = fp8sm.kv_cache_empty(3, 2, 64, 16, device="cpu")
    i32 = torch.int32
    cu, lens, table = torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(2, 4, dtype=i32)
    k = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)

    def write(k=k, v=k, c=c, cu=cu, lens=lens, table=table):
        fp8sm.kv_cache_write(k, v, c, cu, lens, table)

    with pytest.raises(fp8sm.DeviceTensorError):
        write()
    for bad in (dict(cu=cu[:2]), dict(table=table[:1]), dict(table=table.T.contiguous().T), dict(k=k[:, :1]),
                dict(v=k[:4]), dict(v=k.half()), dict(k=k.transpose(0, 1)),
                dict(c=c._replace(v=c.v[:, :1])), dict(c=c._replace(k_exp=c.k_exp[:1])),
                dict(c=c._replace(k=c.k.view(torch.int8)))):
        with pytest.raises(ValueError):
            write(**bad)
    with pytest.raises(TypeError):
        write(cu=cu.long())
    with pytest.raises(ValueError):
        fp8sm.attention_cache(q.flatten(1), c, cu, lens, table, 5)
    with pytest.raises(ValueError):
        fp8sm.attention_cache(q, c, cu, lens, table, 5, out=q[:4])
    with pytest.raises(ValueError):
        fp8sm.attention_cache(q, c, cu, lens, table, 5, lse=torch.zeros(5, 3))
    with pytest.raises(ValueError):
        fp8sm.attention_cache(q, c, cu, lens, table, 1, max_kv=1 << 20, workspace=torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError):
        fp8sm.kv_cache_read(c, cu, lens, table, 6, k=k)
    x = torch.zeros(5, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fp8sm.qk_norm_rope(x, 4, 1, 64)
    with pytest.raises(ValueError):
        fp8sm.qk_norm_rope(x, 2, 1, 64, cos_sin=torch.zeros(4, 64))
    with pytest.raises(ValueError):
        fp8sm.qk_norm_rope(x, 2, 1, 64, torch.zeros(4, dtype=i32), torch.zeros(4, 64))
    with pytest.raises(TypeError):
        fp8sm.qk_norm_rope(x, 2, 1, 64, torch.zeros(5, dtype=i32), torch.zeros(4, 64, dtype=torch.float64))
    with pytest.raises(TypeError):
        fp8sm.qk_norm_rope(x, 2, 1, 64, q_weight=torch.zeros(64), k_weight=torch.zeros(64))
