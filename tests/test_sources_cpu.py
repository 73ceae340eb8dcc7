"""What the kernels' sources may not hold: the library is one file that every process of
a run on several GPUs loads too."""
import glob
import os
import re

import pytest

from mixture_experts_layer_mm_gb300 import buildlib

# (In pieces: this file is a source too.)
COPY, MANY = "cp.async." + "bulk", "multi" + "cast"
SOURCES = sorted(glob.glob(os.path.join(buildlib.CSRC, "*.cu*")))


def _assembly(text):
    """The inline assembly of a source, each statement's literals joined."""
    for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(", text):
        end, out = m.end(), []
        while literal := re.match(r"\s*(?:\"((?:[^\"\\]|\\.)*)\"|//[^\n]*\n)", text[end:]):
            out.append(literal.group(1) or "")
            end += literal.end()
        yield "".join(out)


def test_assembly_is_found():
    found = [a for p in SOURCES for a in _assembly(open(p).read())]
    assert sum(COPY + ".tensor" in a for a in found) > 5
    assert any(MANY in a for a in found)          # (of the MMAs' completion signals)
    assert list(_assembly('asm volatile("a.b" // note\n ".c %0;" : "=r"(x)); asm("d;")')) == \
        ["a.b.c %0;", "d;"]


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_copy_goes_to_several_blocks(path):
    """A copy into the shared memory of several blocks at once is allowed only in code that
    runs on one GPU alone."""
    for a in _assembly(open(path).read()):
        assert not (COPY in a and MANY in a), a


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_shared_arrays_read_16_bytes_at_a_time_are_aligned_to_them(path):
    """An array of ints in shared memory is aligned to 4 bytes unless it says otherwise."""
    text = open(path).read()
    wide = set(re.findall(r"reinterpret_cast<(?:const )?u?(?:int|float)4\s*\*>\(&?(\w+)", text))
    for align, name in re.findall(r"__shared__\s+(__align__\(\d+\)\s+)?\w+\s+(\w+)\s*\[", text):
        assert name not in wide or align.strip() in ("__align__(16)", "__align__(1024)"), name
