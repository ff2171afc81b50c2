"""What the serving kernels' sources may not hold (no GPU)."""
import os
import re

import pytest

from block_wise_int8_amd import build

KERNELS = [s for s in build.SOURCES if s.endswith(".hip") and "_mfma_" in open(s).read()]


def test_there_are_such_kernels():
    assert {os.path.basename(s) for s in KERNELS} >= {"qar_kv8.hip", "qar_mx4.hip"}


@pytest.mark.parametrize("source", KERNELS, ids=os.path.basename)
def test_no_vector_instructions_in_inline_assembly_beside_products(source):
    """A vector instruction may read a matrix instruction's result only after a number of wait states that the compiler counts
    for its own instructions, not for inline assembly."""
    text = re.sub(r"//[^\n]*", "", open(source).read())
    statements = re.findall(r"\basm\b\s*(?:volatile)?\s*\(((?:[^;\"]|\"[^\"]*\")*)\)\s*;", text)
    assert len(statements) == len(re.findall(r"\basm\b", text))
    for s in statements:
        code = " ".join(re.findall(r'"([^"]*)"', s.split(":")[0]))
        assert not re.search(r"\bv_\w+", code), s
