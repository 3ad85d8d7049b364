"""Rules of the device sources that no run can show: what a compiler may do between two statements."""
import glob
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "calibration_free_bit_b200", "csrc")
SOURCES = sorted(f for e in ("cu", "cuh") for f in glob.glob(os.path.join(CSRC, "*." + e)))


def statements(path):
    """The asm statements of a file, comments removed."""
    text = re.sub(r"//[^\n]*", "", open(path).read())
    for m in re.finditer(r"\basm\b", text):
        depth, i = 0, text.index("(", m.end())
        for j in range(i, len(text)):
            depth += {"(": 1, ")": -1}.get(text[j], 0)
            if depth == 0:
                yield text[i:j]
                break


def test_the_sources_are_found():
    names = {os.path.basename(f) for f in SOURCES}
    assert {"sm100_common.cuh", "kv_wide.cuh", "kv_tc.cu", "k1_tc.cu"} <= names
    assert sum(1 for f in SOURCES for s in statements(f) if "tcgen05.ld" in s) >= 3


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_a_load_of_tensor_memory_waits_in_its_own_statement(path):
    """tcgen05.ld fills its registers later; a copy or a spill of one of them before the wait would
    take what was there."""
    for s in statements(path):
        if "tcgen05.ld" in s:
            assert "tcgen05.wait::ld" in s, s[:80]
            assert '"memory"' in s, s[:80]


# what a handle uploads before its first launch: tables, matrices, boundaries
CONSTANT = ("reinterpret_cast<const uint2 *>(src) + (i >> 3)", "src + (i >> 3)", "r_img + ",
            "reinterpret_cast<const uint4 *>(p.tbl) + ", "p.bounds + ", "p.wdec_tab + ")


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_only_constant_tables_take_the_non_coherent_path(path):
    """Kernels start while the one before them still runs, so codes, norms and page tables may
    change during the life of a kernel that reads them (after its wait): plain loads."""
    text = re.sub(r"//[^\n]*", "", open(path).read())
    for m in re.finditer(r"__ldg\(\s*", text):
        assert text[m.end():].startswith(CONSTANT), text[m.start():m.start() + 60]
    assert not re.search(r"ld\.global(\.\w+)*\.nc|__restrict__|ldlu|__ldcv", text)
