"""The fault flags wait for every stream, those that do not block with the legacy one among them."""
import pytest
import torch

from test_gpu_kv8 import i32, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lb(cuda_device):
    from decode_packed_bit_b200 import build
    build.build()
    from decode_packed_bit_b200 import lowbit
    return lowbit


def test_flags_of_a_call_under_way_on_another_stream(lb):
    cache = make_cache(lb, 1, 4, 1, 32, 64)
    table, lens = i32([[99]]), i32([5])  # a page that the cache does not have
    out = torch.empty((1, 1, 64), device="cuda")
    w = torch.randn((8192, 8192), device="cuda")
    assert lb.lowbit_fault_flags() == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(side):
            for _ in range(8):  # a few milliseconds that the read comes after
                w @ w
            lb.lowbit_kv8_read(cache, table, lens, out, None)
        assert lb.lowbit_fault_flags() == 16
        assert side.query()
        assert lb.lowbit_fault_flags() == 0
    assert (out == 0).all()
