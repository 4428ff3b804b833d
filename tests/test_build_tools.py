"""What building the library runs (CPU only)."""
import os
import subprocess

import pytest

from column_scaled_gemm_amd import build


def test_joining_objects_takes_the_compiler_driver_only(tmp_path, monkeypatch):
    """A family of kernels in several sources is one relocatable object, joined by
    the linker that the compiler brings, not by one that may not be there."""
    try:
        hipcc = build._hipcc()
    except RuntimeError:
        pytest.skip("hipcc not found")
    parts = []
    for n in "ab":
        src = tmp_path / f"{n}.cpp"
        src.write_text(f"int {n}() {{ return 1; }}\n")
        parts.append(str(tmp_path / f"{n}.o"))
        subprocess.run([hipcc, "-x", "c++", "-fPIC", "-c", str(src), "-o", parts[-1]], check=True)
    ran = []
    real = subprocess.run

    def run(cmd, *args, **kw):
        ran.append(cmd[0])
        return real(cmd, *args, **kw)

    monkeypatch.setattr(build.subprocess, "run", run)
    out = str(tmp_path / "ab.o")
    build._join(parts, out)
    assert ran == [hipcc] and os.path.getsize(out) > 0
    build._join(parts[:1], out)     # one part: a copy
    assert ran == [hipcc]
    assert open(out, "rb").read() == open(parts[0], "rb").read()
