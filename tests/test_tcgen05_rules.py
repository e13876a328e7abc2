"""Static rule of the tcgen05 sources, checked on the CPU: a wait for loads from tensor memory has the loaded registers as
operands, so that the compiler cannot move their use before it."""
import glob
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "decode_packed_bit_b200", "csrc")


def waits(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return re.findall(r'asm volatile\(\s*"tcgen05\.wait::ld[^;]*;"(.*?)\);', f.read(), re.S)


@pytest.mark.parametrize("name", ["kv8_attn_tc.cu", "int4_gemm_tc.cu"])
def test_waits_for_tensor_memory_loads_tie_their_values(name):
    found = waits(name)
    assert found
    for operands in found:
        assert operands.count('"+r"') >= 16, operands
