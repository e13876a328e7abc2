"""Sizes of the decode-side calls beyond what their kernels' 32-bit indices hold are refused before anything else.  CPU
only: every call here fails validation."""
import ctypes
import itertools

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


# The words of each block: a size that 32 bits do not hold is a refusal, not the size that its low half names.  Each call
# has an address that is refused otherwise (its last one in the list), so that none can be launched.
AT = 0x10000
BLOCKS = {
    "lora_add_group": [AT, AT, 0, 0, "R", "M", "N", "K", "rank", "L", 0, 1 << 40, 0, AT, AT, AT, AT],
    "rope": [AT, 256, 2 * AT, 256, "qh", AT, 128, 2 * AT, 128, "kh", "ti", "to", AT, 0, "M", "D", "rot", "inter", 1.0, 0],
    "kv8_append": ["cache", AT, AT, AT, "B", "width", "rows", 0, 128, "kt", AT, 128, "vt", 0],
    "kv8_read": ["cache", 0, AT, AT, "B", "width", "rows", AT, AT, "to", 0],
    "kv8_attention": ["cache", AT, AT, AT, "B", "width", "rows", AT, 256, "heads", 0.1, AT, 256, 0, 1 << 40, 0],
}
SIZES = dict(R=1, M=4, N=64, K=128, rank=16, L=2, qh=2, kh=1, ti=0, to=1, D=128, rot=64, inter=0, B=2, width=4, rows=3, kt=0, vt=0, heads=4)


@pytest.mark.parametrize("name", BLOCKS)
def test_words_beyond_32_bits(lb, name):
    pytest.importorskip("torch")
    from decode_packed_bit_b200 import _marshal as m
    cache = lb._KV8CacheC(AT, AT, AT, AT, 8, 2, 32, 64)
    f = ctypes.cast(getattr(lb.lib(), f"lowbit_{name}_args"), ctypes.c_void_p).value

    def call(**sizes):
        sizes = {**SIZES, "cache": ctypes.addressof(cache), **sizes}
        return m.call(f, *[sizes.get(w, w) if isinstance(w, str) else w for w in BLOCKS[name]])

    assert call() == 1
    for word, by in itertools.product([w for w in BLOCKS[name] if isinstance(w, str) and w != "cache"], (1 << 32, 1 << 40, -(1 << 32))):
        assert call(**{word: SIZES[word] + by}) == 3, (word, by)
