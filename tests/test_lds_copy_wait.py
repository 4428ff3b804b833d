"""Copies from memory straight into LDS take their destination from m0, and the
hardware wants one wait state between a scalar write of m0 and such a copy.  The
compiler puts it in around its own instructions but does not look into inline
asm, so there the source has to hold it (CPU only)."""
import glob
import os
import re

import pytest

from conftest import ROOT

SOURCES = sorted(glob.glob(os.path.join(ROOT, "column_scaled_gemm_amd", "csrc", "*.hip")))


def asm_blocks(text):
    """The instructions of every inline asm statement, one list each."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"\basm\s+volatile\s*\(\s*((?:\"(?:[^\"\\]|\\.)*\"\s*)+)", text):
        code = "".join(re.findall(r"\"((?:[^\"\\]|\\.)*)\"", m.group(1)))
        yield [i.strip() for i in re.split(r"\\n|;", code.replace("\\t", " ")) if i.strip()]


def is_lds_copy(instruction):
    op = instruction.split()[0]
    return "_load_lds_" in op or (op.startswith("buffer_load") and re.search(r"\blds\b", instruction))


def writes_m0(instruction):
    return re.match(r"s_\w+\s+m0\b", instruction) is not None


@pytest.mark.parametrize("path", SOURCES, ids=[os.path.basename(p) for p in SOURCES])
def test_a_copy_never_directly_follows_its_write_of_m0(path):
    with open(path) as f:
        for block in asm_blocks(f.read()):
            for a, b in zip([""] + block, block):
                assert not (writes_m0(a) and is_lds_copy(b)), block
            # m0's writer outside the statement would be out of sight: each copy brings its own
            if any(is_lds_copy(i) for i in block):
                assert any(writes_m0(i) for i in block), block


def test_the_copies_are_seen():
    blocks = [b for p in SOURCES for b in asm_blocks(open(p).read()) if any(map(is_lds_copy, b))]
    assert len(blocks) == 3 and all("s_nop 0" in b for b in blocks)
