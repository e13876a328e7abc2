"""The adapters' kernels for blocks of rows (more than 256, or 16 for each adapter of the pool) at every rank class, those
above 64 among them, for widths that are multiples of 4 and not; tests of the gathered form are beside them."""
import numpy as np
import pytest
import torch

from test_gpu_lora import check, make, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lb(cuda_device):
    from decode_packed_bit_b200 import build
    build.build()
    from decode_packed_bit_b200 import lowbit
    return lowbit


def blocks(M, L):
    """Whether a call goes in blocks of the caller's order."""
    return M > 256 or M >= 16 * L


@pytest.mark.parametrize("order", ["any", "runs", "one"])
@pytest.mark.parametrize("M,L", [(257, 40), (300, 3), (64, 4), (33, 2), (1030, 5)])
@pytest.mark.parametrize("rank,N", [(8, 200), (24, 133), (40, 132), (64, 77), (72, 200), (72, 131), (128, 256), (128, 390)])
def test_blocks(lb, M, L, rank, N, order):
    K = 192
    assert blocks(M, L)
    x, ids, a, b, base, ranks, scales = make(M + L + rank, M, N, K, rank, L)
    if order == "runs":
        ids = torch.sort(ids.roll(7)).values
    elif order == "one":
        ids[:] = L - 1
    ranks[0], ranks[L - 1] = rank, max(1, rank - 3)
    y = torch.full((M, N), float("nan"), device="cuda")
    ws = workspace(lb, 1, M, N, K, rank)
    lb.lowbit_lora_add(x, ids, a[0], b[0], base[0], y, ranks, scales, ws)
    check(y, x, ids, a[0], b[0], base[0], ranks, scales, f"M={M} L={L} rank={rank} N={N} {order}")
    z = base[0].clone()
    lb.lowbit_lora_add(x, ids, a[0], b[0], z, z, ranks, scales, ws)
    assert torch.equal(y, z)  # in place, the same bits


@pytest.mark.parametrize("rank", [72, 128])
@pytest.mark.parametrize("M,L,N", [(300, 4, 96), (64, 4, 131)])
def test_padding_and_other_adapters_cannot_reach_a_row(lb, M, L, N, rank):
    K = 256
    assert blocks(M, L)
    x, _, a, b, base, _, scales = make(rank, M, N, K, rank, L)
    ranks = torch.tensor([1, 65, rank - 1, rank], dtype=torch.int32, device="cuda")
    ids = torch.arange(M, device="cuda", dtype=torch.int32) % L
    clean_a, clean_b = a[0].clone(), b[0].clone()
    for i, r in enumerate(ranks.tolist()):
        a[0][i, r:] = float("nan")
        b[0][i, :, r:] = float("inf")
    y, z = torch.empty((M, N), device="cuda"), torch.empty((M, N), device="cuda")
    ws = workspace(lb, 1, M, N, K, rank)
    lb.lowbit_lora_add(x, ids, a[0], b[0], base[0], y, ranks, scales, ws)
    check(y, x, ids, clean_a, clean_b, base[0], ranks, scales, "padding holds NaN and infinities")
    a[0][3] = float("nan")
    lb.lowbit_lora_add(x, ids, a[0], b[0], base[0], z, ranks, scales, ws)
    assert torch.equal(y[ids != 3], z[ids != 3]) and torch.isnan(z[ids == 3]).all()


@pytest.mark.parametrize("R,M,L,rank", [(3, 300, 6, 128), (2, 40, 2, 72), (16, 260, 4, 16)])
def test_groups_captured(lb, R, M, L, rank):
    """Several projections in blocks, captured, replayed with other ids."""
    N, K = 136, 320
    assert blocks(M, L)
    x, ids, a, b, base, ranks, scales = make(R, M, N, K, rank, L, R)
    ys = [torch.empty((M, N), device="cuda") for _ in range(R)]
    ws = workspace(lb, R, M, N, K, rank)
    lb.lowbit_lora_add_group(x, ids, a, b, base, ys, ranks, scales, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lb.lowbit_lora_add_group(x, ids, a, b, base, ys, ranks, scales, ws)
    g = np.random.default_rng(R)
    for _ in range(2):
        ids.copy_(torch.from_numpy(g.integers(-1, L, M).astype(np.int32)))
        graph.replay()
        for r in range(R):
            check(ys[r], x, ids, a[r], b[r], base[r], ranks, scales, f"projection {r}")
