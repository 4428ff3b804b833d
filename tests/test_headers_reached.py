"""Nothing stays in the kernels' shared headers that no kernel calls (CPU only)."""
import glob
import os
import re

import pytest

from column_scaled_gemm_amd import build

HEADERS = sorted(os.path.join(build.CSRC, n) for n in
                 ("attn_common.h", "device_common.h", "gemm_common.h", "kv_common.h", "lds_copy.h", "packed_rows.h"))


@pytest.mark.parametrize("path", HEADERS, ids=os.path.basename)
def test_every_function_has_a_caller(path):
    code = "".join(re.sub(r"//[^\n]*", "", open(p).read())
                   for p in glob.glob(os.path.join(build.CSRC, "*")) if p.endswith((".h", ".hip", ".cpp")))
    names = re.findall(r"(?:__device__|__host__|static|inline)[^;{}()]*?\b(\w+)\((?!\()[^;{}]*\{",
                       re.sub(r"__attribute__\(\(\w+\)\)", "", re.sub(r"//[^\n]*", "", open(path).read())))
    assert names
    unused = [n for n in names if n != "explicit" and len(re.findall(rf"\b{n}\b", code)) < 2]
    assert not unused, unused
