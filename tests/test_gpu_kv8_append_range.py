"""Append and read at the ends of fp32's range, bit for bit against the definition: pages whose scale is subnormal, where
it is rounded by up to a half of itself and the quotients have to be held to 127."""
import numpy as np
import pytest
import torch

import decode_reference as ref
from parity_util import host
from test_gpu_kv8 import i32, make_batch, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lb(cuda_device):
    from decode_packed_bit_b200 import build
    build.build()
    from decode_packed_bit_b200 import lowbit
    return lowbit


UNITS = [1, 62, 63, 64, 126, 127, 190, 191, 254, 318, 1000, 8128, 16256, 1 << 20, 1 << 21, 1 << 22, 1 << 23, 3 << 22, 1 << 27, 1 << 30]


def values(g, rows, H, D, most):
    """float32 of at most `most` units of 2^-149, both signs of the largest among them."""
    x = np.rint(g.uniform(-1, 1, (rows, H, D)) * most) * 2.0 ** -149
    x[0, :, 0], x[-1, :, 1] = most * 2.0 ** -149, -most * 2.0 ** -149
    return x.astype(np.float32)


@pytest.mark.parametrize("rows", [1, 3, 40])
@pytest.mark.parametrize("D,P", [(64, 32), (128, 64), (128, 128)])
def test_subnormal_pages(lb, D, P, rows):
    """Fresh pages, and the same pages grown by a second write, which rounds the older codes again."""
    H, B = 2, len(UNITS)
    g = np.random.default_rng(rows + D)
    lens = [rows] * B
    n_pages, table = make_batch(P, [rows * 2] * B, P)
    cache = lb.KV8Cache.empty(n_pages, H, P, D)
    codes, scales = host(cache.k).copy(), host(cache.k_scales).copy()
    for step in (1, 2):
        lens = [rows * step] * B
        x = np.concatenate([values(g, rows, H, D, u * step * step + step) for u in UNITS])
        xd = torch.from_numpy(x).cuda()
        lb.lowbit_kv8_append(cache, i32(table), i32(lens), xd, xd, row_start=None if rows == 1 else i32(starts([rows] * B)))
        codes, scales = ref.append(codes, scales, x, lens, table, starts([rows] * B))
        for c, s in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
            assert np.array_equal(host(s), scales)
            assert np.array_equal(host(c), codes)
    back = torch.empty((rows * B, H, D), device="cuda")
    lb.lowbit_kv8_read(cache, i32(table), i32(lens), back, None, row_start=i32(starts([rows] * B)))
    for r, _, pos, page, slot in ref.places(lens, table, starts([rows] * B), rows * B, P, n_pages):
        want = torch.from_numpy(codes[page, :, slot].astype(np.float64) * scales[page].astype(np.float64)[:, None]).float()
        assert torch.equal(back[r].cpu(), want)


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_largest_values(lb, kind):
    """Values up to the largest that the type holds, and infinities, which count as the largest float."""
    H, D, P = 1, 64, 32
    cache = lb.KV8Cache.empty(3, H, P, D)
    g = np.random.default_rng(1)
    x = (g.uniform(-1, 1, (5, H, D)) * 3.3e38).astype(np.float32)
    x[2, 0, 3], x[4, 0, 7] = np.inf, -np.inf
    xd = torch.from_numpy(x).to(kind).cuda()
    table, lens = np.array([[2]], np.int32), [5]
    lb.lowbit_kv8_append(cache, i32(table), i32(lens), xd, xd, row_start=i32([0, 5]))
    codes, scales = ref.append(np.zeros((3, H, P, D), np.int8), np.zeros((3, H), np.float32), xd.float().cpu().numpy(), lens, table, np.array([0, 5]))
    assert np.array_equal(host(cache.k), codes) and np.array_equal(host(cache.k_scales), scales)
    assert np.array_equal(host(cache.v), codes) and np.array_equal(host(cache.v_scales), scales)
