"""Every store of the serving kernels whose index is computed is guarded in the
bounds-checked build (VT_CHECKED): each of their sources has a guard of its own
or stores through a function of its header that has one."""
import os
import re

import pytest

import frequency_ranked_drafter_gb300 as vt

CSRC = os.path.join(os.path.dirname(vt.__file__), "csrc")


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", ["quantize.cu", "sample.cu", "verify.cu"])
def test_own_guard(name):
    assert "VT_CHECKED(" in source(name)


@pytest.mark.parametrize("name", ["matmul_i8_gemv.cu", "matmul_i8_mma.cu", "matmul_i8_tc.cu"])
def test_products_store_through_a_guarded_function(name):
    header = source("matmul_i8.cuh")
    store = header[header.index("void i8_store("):]
    store = store[:store.index("\n}")]
    guard, write = store.index("VT_CHECKED("), store.index("[i] =")
    assert guard < write
    text = source(name)
    assert "i8_store(" in text
    # nothing else there writes to the output
    assert not re.search(r"\b(g|a|p)\.out\s*\)?\s*\[", text)
