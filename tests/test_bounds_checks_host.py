"""The debug build's checks cover the mixture-of-experts kernels: their units reach global memory only
through the checked loads and stores (bounds_check.cuh).  Read from the sources, since no call of a
correct kernel can show a check that is missing."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "nvfp4_bit_quantized_03_b200", "csrc")
# the arrays that the kernels of these units are given
ARRAYS = "logits|bias|experts|weights|dweights|dlogits|offsets|pair_row|row_token|counts|out|dout|dy|y"


def _code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


@pytest.mark.parametrize("unit", ["route.cu", "combine.cu"])
def test_units_use_checked_accesses_only(unit):
    code = _code(unit)
    assert "__ldg(" not in code
    assert not re.findall(rf"\ba\.(?:map\.)?(?:{ARRAYS})\s*\[", code)        # a.weights[...]
    assert not re.findall(rf"\*\s*a\.(?:{ARRAYS})\b(?!\s*\w)", code)         # *a.weights
    assert not re.findall(r"\b(?:drow|column|o)\s*\[", code)               # pointers into them
    assert not re.findall(r"reinterpret_cast<(?:const )?uint[24]\*>\([^;]*?\)\s*\[", code)


def test_row_maps_use_checked_accesses_only():
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh", ".h")):
            assert not re.findall(r"\b(?:row_token|pair_row)\s*\[", _code(name)), name
