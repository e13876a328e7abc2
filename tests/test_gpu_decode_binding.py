"""Refusals of the decode-side binding that need a GPU's tensors: operands left out, of another rank, too many."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lb(cuda_device):
    from decode_packed_bit_b200 import build
    build.build()
    from decode_packed_bit_b200 import lowbit
    return lowbit


def zeros(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def test_rope_operands_left_out(lb):
    q, pos, phases = zeros(2, 4, 64), zeros(2, dtype=torch.int32), zeros(32, dtype=torch.int64)
    for args in ((None, None, None, None), (q, None, None, None), (None, q, None, None), (q, q, q, None), (None, None, None, q),
                 (q, None, q, q)):
        with pytest.raises(ValueError, match="lowbit_rope"):
            lb.lowbit_rope(*args, pos, phases)
    lb.lowbit_rope(q, q, None, None, pos, phases)
    lb.lowbit_rope(None, None, q, q, pos, phases)


def test_read_of_nothing(lb):
    cache = lb.KV8Cache.empty(2, 1, 32, 64)
    table, lens = zeros(1, 1, dtype=torch.int32), zeros(1, dtype=torch.int32)
    lb.lowbit_kv8_read(cache, table, lens, None, None)
    assert lb.lowbit_fault_flags() == 0


def test_lora_lists(lb):
    M, N, K, r, L = 2, 64, 64, 8, 1
    x, ids, y = zeros(M, K, dtype=torch.bfloat16), zeros(M, dtype=torch.int32), zeros(M, N)
    a, b = zeros(L, r, K, dtype=torch.bfloat16), zeros(L, N, r, dtype=torch.bfloat16)
    ws = zeros(1 << 16, dtype=torch.uint8)
    for n in (0, 17, 40):
        with pytest.raises(ValueError, match="1 to 16"):
            lb.lowbit_lora_add_group(x, ids, [a] * n, [b] * n, [y] * n, [y] * n, workspace=ws)
    for bad in (dict(a=[a[0]]), dict(b=[b[0]]), dict(b=[b[0, 0]]), dict(x=x[0]), dict(ys=[y[0]]), dict(ids=ids[None])):
        with pytest.raises(ValueError):
            lb.lowbit_lora_add_group(**{**dict(x=x, ids=ids, a=[a], b=[b], base=[y], ys=[y]), **bad}, workspace=ws)
    lb.lowbit_lora_add_group(x, ids, [a], [b], [y], [y], workspace=ws)
