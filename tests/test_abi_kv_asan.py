"""The refusals of the head norm, cache and attention calls and their workspace
query, against a build of the library's host part with AddressSanitizer: as
test_abi_asan.py does for the others, and with its parts.  Host code only; nothing
here launches a kernel."""
import os
import subprocess
import sys

import pytest

from conftest import ROOT

asan = pytest.importorskip("test_abi_asan")
pytestmark = asan.pytestmark


def test_kv_rejection_paths_are_clean_under_address_sanitizer(tmp_path):
    obj, lib = str(tmp_path / "api_asan.o"), str(tmp_path / "libfp8sm_asan.so")
    host = ["-O1", "-g", "-std=c++17", "-fPIC", "-fno-omit-frame-pointer", "-ffp-contract=off",
            "-I", os.path.join(ROOT, "include"), "-I", asan.BUILD, "-D__HIP_PLATFORM_AMD__",
            "-I", "/opt/rocm/include"]
    for cmd in ([*host, "-Xarch_host", "-fsanitize=address", "-x", "c++", "-c",
                 os.path.join(asan.CSRC, "api.cpp"), "-o", obj],
                ["--offload-arch=gfx950", "-shared", "-fPIC", "-shared-libsan",
                 "-Xarch_host", "-fsanitize=address", "-o", lib, *asan.OBJS, obj]):
        r = subprocess.run([asan._hipcc(), *cmd], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
    tests = [os.path.join(ROOT, "tests", n) for n in ("test_abi_kv.py", "test_abi_kv_edges.py")]
    runner = ("import sys; sys.path.insert(0, %r); sys.path.insert(0, %r)\n"
              "from column_scaled_gemm_amd import fp8sm\n"
              "fp8sm.LIB_PATH = %r\n"
              "import pytest\n"
              "sys.exit(pytest.main(['-q', '-x', '-m', 'not gpu', '-p', 'no:cacheprovider', *%r]))\n"
              ) % (ROOT, os.path.join(ROOT, "tests"), lib, tests)
    env = dict(os.environ, LD_PRELOAD=asan.RUNTIME[-1],
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0")
    r = subprocess.run([sys.executable, "-c", runner], capture_output=True, text=True, env=env,
                       cwd=str(tmp_path), timeout=600)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out, out[-4000:]
    assert r.returncode == 0, out[-4000:]
    assert " passed" in out
