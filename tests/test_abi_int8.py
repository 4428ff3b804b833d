"""Refusals of the int8 calls, on the host before any launch (no GPU needed), the
instruction forms of the copies that headers hold, and the binding's own checks."""
import ctypes
import glob
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


def _quant(lib, **kw):
    a = dict(x=16, dt=0, nb=1, M=4, K=64, bsx=0, ldx=128, rows=0, flags=0, q=16, bsq=0, ldq=64, s=16)
    a.update(kw)
    return lib.fp8sm_quant_int8(P(a["x"]), a["dt"], a["nb"], a["M"], a["K"], a["bsx"], a["ldx"], P(a["rows"]),
                                a["flags"], P(a["q"]), a["bsq"], a["ldq"], P(a["s"]), P(0))


@pytest.mark.parametrize("kw,err", [
    (dict(dt=2), "UNSUPPORTED"), (dict(flags=2), "UNSUPPORTED"), (dict(M=-1), "SHAPE"), (dict(K=0), "SHAPE"),
    (dict(nb=-1), "SHAPE"), (dict(nb=65536), "RANGE"), (dict(bsx=-8), "SHAPE"), (dict(bsq=-8), "SHAPE"),
    (dict(M=1 << 24), "RANGE"), (dict(K=(1 << 30) + 8, ldx=1 << 31, ldq=1 << 31), "RANGE"),
    (dict(ldx=56), "SHAPE"), (dict(flags=1, ldx=120), "SHAPE"), (dict(ldq=56), "SHAPE"),
    (dict(K=60), "ALIGN"), (dict(ldx=132), "ALIGN"), (dict(ldq=68), "ALIGN"), (dict(nb=2, bsq=260), "ALIGN"),
    (dict(nb=2, bsx=4, bsq=256), "ALIGN"), (dict(nb=2, bsq=248), "SHAPE"), (dict(rows=2), "ALIGN"),
    (dict(x=0), "NULL"), (dict(q=0), "NULL"), (dict(s=0), "NULL"), (dict(x=8), "ALIGN"), (dict(q=4), "ALIGN"),
    (dict(s=2), "ALIGN")])
def test_quant_refusals(kw, err):
    lib, E = _codes()
    assert _quant(lib, **kw) == E["ERR_" + err]


def _mm(lib, **kw):
    a = dict(nb=1, rows=0, A=16, bsa=0, lda=64, B=16, bsb=0, ldb=64, C=16, bsc=0, ldc=64, M=4, N=64, K=64, ka=1,
             sa=16, bssa=0, kb=2, sb=16, bssb=0, bias=0, out=0)
    a.update(kw)
    return lib.fp8sm_scaled_mm_int8(a["nb"], P(a["rows"]), P(a["A"]), a["bsa"], a["lda"], P(a["B"]), a["bsb"],
                                    a["ldb"], P(a["C"]), a["bsc"], a["ldc"], a["M"], a["N"], a["K"], a["ka"],
                                    P(a["sa"]), a["bssa"], a["kb"], P(a["sb"]), a["bssb"], P(a["bias"]), a["out"],
                                    P(0))


@pytest.mark.parametrize("kw,err", [
    (dict(ka=2), "UNSUPPORTED"), (dict(kb=1), "UNSUPPORTED"), (dict(ka=4, kb=5), "UNSUPPORTED"),
    (dict(ka=3, kb=5), "UNSUPPORTED"), (dict(out=2), "UNSUPPORTED"), (dict(M=-1), "SHAPE"), (dict(N=-8), "SHAPE"),
    (dict(K=-16), "SHAPE"), (dict(lda=48), "SHAPE"), (dict(ldb=48), "SHAPE"), (dict(ldc=56), "SHAPE"),
    (dict(K=56), "ALIGN"), (dict(lda=72), "ALIGN"), (dict(ldb=72), "ALIGN"), (dict(N=60), "ALIGN"),
    (dict(ldc=68), "ALIGN"), (dict(K=65552, lda=65552, ldb=65552), "RANGE"), (dict(lda=(1 << 24) + 16), "RANGE"),
    (dict(M=(1 << 30) + 1), "RANGE"), (dict(M=1 << 20, N=1 << 18, ldc=1 << 18), "RANGE"), (dict(nb=-1), "SHAPE"),
    (dict(nb=65536), "RANGE"), (dict(nb=2, bsc=248), "SHAPE"), (dict(nb=2, bsc=256, bsa=8), "ALIGN"),
    (dict(nb=2, bsc=256, bssa=-1), "SHAPE"), (dict(rows=2), "ALIGN"), (dict(A=0), "NULL"), (dict(B=0), "NULL"),
    (dict(C=0), "NULL"), (dict(sa=0), "NULL"), (dict(sb=0), "NULL"), (dict(A=8), "ALIGN"), (dict(B=8), "ALIGN"),
    (dict(C=8), "ALIGN"), (dict(sa=2), "ALIGN"), (dict(sb=2), "ALIGN"), (dict(bias=1), "ALIGN")])
def test_product_refusals(kw, err):
    lib, E = _codes()
    assert _mm(lib, **kw) == E["ERR_" + err]


def test_nothing_to_do_is_ok():
    lib, E = _codes()
    assert _quant(lib, M=0, x=0) == _quant(lib, nb=0, q=0) == E["OK"]
    assert _mm(lib, M=0, A=0) == _mm(lib, N=0, ldc=0) == _mm(lib, nb=0) == E["OK"]


def test_binding_refuses_what_the_abi_cannot_see():
    from column_scaled_gemm_amd import fp8sm
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    i8 = torch.int8
    a, b = torch.zeros(4, 64, dtype=i8), torch.zeros(8, 64, dtype=i8)
    sa, sb = torch.ones(4), torch.ones(8)
    with pytest.raises(fp8sm.DeviceTensorError):
        fp8sm.quant_int8(x)
    with pytest.raises(fp8sm.DeviceTensorError):
        fp8sm.scaled_mm_int8(a, b, sa, sb)
    for kw in (dict(q=torch.zeros(3, 64, dtype=i8)), dict(q=torch.zeros(4, 56, dtype=i8)), dict(scales=sa[:3]),
               dict(q=torch.zeros(64, 4, dtype=i8).T), dict(rows=torch.zeros(1, dtype=torch.int32))):
        with pytest.raises(ValueError):
            fp8sm.quant_int8(x, **kw)
    for kw in (dict(q=torch.zeros(4, 64, dtype=torch.uint8)), dict(scales=sa.double())):
        with pytest.raises(TypeError):
            fp8sm.quant_int8(x, **kw)
    with pytest.raises(ValueError):
        fp8sm.quant_int8(x[0])
    with pytest.raises(ValueError):
        fp8sm.quant_int8(x[:, :63], fuse_silu_mul=True)
    with pytest.raises(ValueError):
        fp8sm.quant_int8(x.T)
    for args, kw in (((a, b[:, :48], sa, sb), {}), ((a, b[None], sa, sb), {}), ((a, b, sa[:3], sb), {}),
                     ((a, b, sa, sb[:7]), {}), ((a, b, sa, sb), dict(c=torch.zeros(4, 4).bfloat16())),
                     ((a, b, sa, sb), dict(bias=sb[:4].bfloat16())), ((a[None].expand(2, 4, 64), b[None], sa, sb), {}),
                     ((a, b, sa, sb), dict(kind_a=fp8sm.KIND_GROUP128_FP32)),
                     ((a, b, sa, sb, fp8sm.KIND_TENSOR), {})):
        with pytest.raises(ValueError):
            fp8sm.scaled_mm_int8(*args, **kw)
    for args, kw in (((a.byte(), b, sa, sb), {}), ((a, b, sa.double(), sb), {}),
                     ((a, b, sa, sb), dict(bias=sb.half())),
                     ((a, b, sa, sb), dict(c=torch.zeros(4, 8).half(), out_dtype=torch.bfloat16))):
        with pytest.raises(TypeError):
            fp8sm.scaled_mm_int8(*args, **kw)


def test_copies_in_headers_wait_after_their_write_of_m0():
    from test_lds_copy_wait import asm_blocks, is_lds_copy, writes_m0
    seen = 0
    for path in glob.glob(os.path.join(ROOT, "column_scaled_gemm_amd", "csrc", "*.h")):
        for block in asm_blocks(open(path).read()):
            for i, op in enumerate(block):
                if is_lds_copy(op):
                    seen += 1
                    assert i >= 2 and block[i - 1] == "s_nop 0" and writes_m0(block[i - 2])
    assert seen >= 1
