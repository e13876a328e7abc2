"""Sizes of the decode-side calls beyond what their kernels' 32-bit indices hold are refused before anything else.  CPU
only: every call here fails validation."""
import ctypes

import pytest

from decode_packed_bit_b200 import build as lb_build

FAKE = ctypes.c_void_p(0x10000)


@pytest.fixture(scope="module")
def lb():
    lb_build.build()
    from decode_packed_bit_b200 import lowbit
    lowbit.lib()
    return lowbit


def test_lora_depth(lb):
    """K near 2^31 made the slices' ends wrap, and a loop over k that steps past 2^31 - 1 does not end."""
    for K in ((1 << 28) + 64, (1 << 31) - 64):
        assert lb.lowbit_lora_workspace_bytes(1, 1, 64, K, 8) == 0
        # (a workspace of no bytes: refused in any case)
        assert lb.lib().lowbit_lora_add(FAKE, FAKE, FAKE, FAKE, None, None, FAKE, FAKE, 1, 64, K, 8, 1, FAKE, 0, None) == 3
    assert lb.lowbit_lora_workspace_bytes(1, 1, 64, 1 << 28, 8) > 0
    assert lb.lib().lowbit_lora_add(FAKE, FAKE, FAKE, FAKE, None, None, FAKE, FAKE, 1, 64, 1 << 28, 8, 1, FAKE, 0, None) == 1
