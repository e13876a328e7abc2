"""GPU parity of the per-request adapters (lowbit_lora_add, _group) against the definition in 64 bits, within the float
bar of the products (relative L2 <= 1e-5, per element <= 2e-3 of the sum of magnitudes): every rank class, ragged
ranks, rows without an adapter, odd row counts and widths, in place, groups, padding that holds NaN, a captured graph."""
import numpy as np
import pytest
import torch

import decode_reference as ref
from parity_util import check_float, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lb(cuda_device):
    from decode_packed_bit_b200 import build
    build.build()
    from decode_packed_bit_b200 import lowbit
    return lowbit


def make(seed, M, N, K, rank, L, R=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    a = [(torch.randn((L, rank, K), generator=g, device="cuda") / K ** 0.5).bfloat16() for _ in range(R)]
    b = [(torch.randn((L, N, rank), generator=g, device="cuda") / rank ** 0.5).bfloat16() for _ in range(R)]
    base = [torch.randn((M, N), generator=g, device="cuda") for _ in range(R)]
    ids = torch.randint(-1, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    ranks = torch.randint(1, rank + 1, (L,), generator=g, device="cuda", dtype=torch.int32)
    scales = torch.rand(L, generator=g, device="cuda") * 4 - 2
    return x, ids, a, b, base, ranks, scales


def workspace(lb, R, M, N, K, rank):
    n = lb.lowbit_lora_workspace_bytes(R, M, N, K, rank)
    assert n > 0
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN wherever it is read unwritten


def check(y, x, ids, a, b, base, ranks, scales, what):
    want, ab = ref.lora(ref.bf16_to_f64(x), host(ids), ref.bf16_to_f64(a), ref.bf16_to_f64(b),
                        host(base).astype(np.float64), None if ranks is None else host(ranks),
                        None if scales is None else host(scales))
    check_float(host(y), want, ab, what)


@pytest.mark.parametrize("M,N,K,rank,L", [
    (1, 64, 64, 8, 1), (1, 4096, 4096, 16, 5), (2, 1, 128, 8, 3), (3, 77, 192, 24, 4), (16, 512, 1024, 16, 16),
    (17, 130, 320, 32, 2), (33, 1000, 640, 40, 50), (61, 96, 2048, 64, 7), (100, 257, 512, 128, 9),
    (300, 344, 1024, 32, 3), (1025, 520, 256, 8, 6)])
def test_matches_definition(lb, M, N, K, rank, L):
    x, ids, a, b, base, ranks, scales = make(M + N + rank, M, N, K, rank, L)
    if M == 1:
        ids[0] = L - 1
    y = torch.full((M, N), float("nan"), device="cuda")
    lb.lowbit_lora_add(x, ids, a[0], b[0], base[0], y, ranks, scales, workspace(lb, 1, M, N, K, rank))
    check(y, x, ids, a[0], b[0], base[0], ranks, scales, f"M={M} N={N} K={K} rank={rank}")
    skip = (ids < 0)
    assert torch.equal(y[skip], base[0][skip])
    # whole ranks, no scales
    lb.lowbit_lora_add(x, ids, a[0], b[0], base[0], y, workspace=workspace(lb, 1, M, N, K, rank))
    check(y, x, ids, a[0], b[0], base[0], None, None, "no ranks, no scales")


@pytest.mark.parametrize("R,M,N,K,rank", [(2, 5, 300, 512, 16), (3, 40, 256, 256, 64), (16, 1, 64, 128, 8)])
def test_group_equals_single_calls(lb, R, M, N, K, rank):
    x, ids, a, b, base, ranks, scales = make(R * M, M, N, K, rank, 6, R)
    ys = [torch.full((M, N), float("nan"), device="cuda") for _ in range(R)]
    lb.lowbit_lora_add_group(x, ids, a, b, base, ys, ranks, scales, workspace(lb, R, M, N, K, rank))
    for r in range(R):
        check(ys[r], x, ids, a[r], b[r], base[r], ranks, scales, f"projection {r}")


def test_in_place_and_repeatable(lb):
    M, N, K, rank = 37, 200, 512, 32
    x, ids, a, b, base, ranks, scales = make(5, M, N, K, rank, 4)
    ws = workspace(lb, 1, M, N, K, rank)
    y = torch.empty((M, N), device="cuda")
    lb.lowbit_lora_add(x, ids, a[0], b[0], base[0], y, ranks, scales, ws)
    z = base[0].clone()
    lb.lowbit_lora_add(x, ids, a[0], b[0], z, z, ranks, scales, ws)
    assert torch.equal(y, z)  # the same bits again, in place


def test_ids_outside_the_pool_and_ranks_out_of_range(lb):
    M, N, K, rank, L = 20, 96, 128, 16, 3
    x, ids, a, b, base, ranks, scales = make(6, M, N, K, rank, L)
    ids[:4] = torch.tensor([L, -7, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    ranks[:3] = torch.tensor([-5, 99, 0], dtype=torch.int32, device="cuda")
    y = torch.empty((M, N), device="cuda")
    lb.lowbit_lora_add(x, ids, a[0], b[0], base[0], y, ranks, scales, workspace(lb, 1, M, N, K, rank))
    assert torch.equal(y[:4], base[0][:4])
    check(y, x, ids, a[0], b[0], base[0], ranks, scales, "clamped ranks")


def test_padding_and_other_adapters_cannot_reach_a_row(lb):
    M, N, K, rank, L = 24, 80, 256, 32, 4
    x, ids, a, b, base, _, scales = make(7, M, N, K, rank, L)
    ranks = torch.tensor([1, 13, 22, 32], dtype=torch.int32, device="cuda")
    ids = torch.arange(M, device="cuda", dtype=torch.int32) % L
    clean_a, clean_b = a[0].clone(), b[0].clone()
    for i, r in enumerate(ranks.tolist()):
        a[0][i, r:] = float("nan")
        b[0][i, :, r:] = float("inf")
    y = torch.empty((M, N), device="cuda")
    ws = workspace(lb, 1, M, N, K, rank)
    lb.lowbit_lora_add(x, ids, a[0], b[0], base[0], y, ranks, scales, ws)
    check(y, x, ids, clean_a, clean_b, base[0], ranks, scales, "padding holds NaN and infinities")
    # one adapter broken: only its rows are
    a[0][3] = float("nan")
    z = torch.empty((M, N), device="cuda")
    lb.lowbit_lora_add(x, ids, a[0], b[0], base[0], z, ranks, scales, ws)
    assert torch.equal(y[ids != 3], z[ids != 3])
    assert torch.isnan(z[ids == 3]).all()
    # and a row of x that is not finite
    x[5] = float("inf")
    lb.lowbit_lora_add(x, ids, clean_a, clean_b, base[0], z, ranks, scales, ws)
    keep = torch.arange(M, device="cuda") != 5
    assert torch.equal(y[keep], z[keep])


@pytest.mark.parametrize("M,L,used", [(40, 4, [1]), (250, 20, [3, 17]), (250, 20, [-1, 0, 5, 6, 7]), (33, 3, [2]), (64, 2, [0, 1]),
                                      (256, 16, [9]), (256, 17, [9]), (16, 1, [0]), (15, 1, [0]), (20, 30, [4, 4, 4, 5])])
@pytest.mark.parametrize("rank", [8, 40])
def test_many_rows_of_an_adapter(lb, M, L, used, rank):
    """More rows of one adapter than a tile holds, gathered or in blocks; exactly 16, and one more."""
    N, K = 200, 128
    x, _, a, b, base, ranks, scales = make(M + L, M, N, K, rank, L)
    g = torch.Generator().manual_seed(M)
    ids = torch.tensor(used, dtype=torch.int32)[torch.randint(0, len(used), (M,), generator=g)].cuda()
    y = torch.full((M, N), float("nan"), device="cuda")
    ws = workspace(lb, 1, M, N, K, rank)
    lb.lowbit_lora_add(x, ids, a[0], b[0], base[0], y, ranks, scales, ws)
    check(y, x, ids, a[0], b[0], base[0], ranks, scales, f"M={M} L={L} used={used} rank={rank}")
    z = base[0].clone()
    lb.lowbit_lora_add(x, ids, a[0], b[0], z, z, ranks, scales, ws)
    assert torch.equal(y, z)


def test_graph_follows_ids(lb):
    M, N, K, rank, L = 9, 128, 256, 16, 5
    x, ids, a, b, base, ranks, scales = make(8, M, N, K, rank, L)
    y = torch.empty((M, N), device="cuda")
    ws = workspace(lb, 1, M, N, K, rank)
    lb.lowbit_lora_add(x, ids, a[0], b[0], base[0], y, ranks, scales, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lb.lowbit_lora_add(x, ids, a[0], b[0], base[0], y, ranks, scales, ws)
    for seed in (1, 2):
        ids.copy_(torch.randint(-1, L, (M,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32))
        graph.replay()
        check(y, x, ids, a[0], b[0], base[0], ranks, scales, "replayed")


def test_beside_a_packed_projection(lb):
    """The projection's output as base, in place, as a decoder runs it."""
    M, N, K, rank, L = 6, 256, 1024, 16, 3
    x, ids, a, b, _, ranks, scales = make(9, M, N, K, rank, L)
    w = torch.randn((N, K), device="cuda") * 0.05
    q, s = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda"), torch.empty((N, K // 64), dtype=torch.int16, device="cuda")
    lb.lowbit_quantize("int4", w, q, s)
    y = torch.empty((M, N), device="cuda")
    lb.lowbit_int4g64_gemm(q, s, x, y)
    shared = y.clone()
    lb.lowbit_lora_add(x, ids, a[0], b[0], y, y, ranks, scales, workspace(lb, 1, M, N, K, rank))
    check(y, x, ids, a[0], b[0], shared, ranks, scales, "beside int4")


def test_binding_refusals(lb):
    M, N, K, rank, L = 4, 64, 128, 16, 2
    x, ids, a, b, base, ranks, scales = make(10, M, N, K, rank, L)
    y = torch.empty((M, N), device="cuda")
    ws = workspace(lb, 1, M, N, K, rank)
    with pytest.raises(ValueError):
        lb.lowbit_lora_add(x, ids.long(), a[0], b[0], base[0], y, workspace=ws)
    with pytest.raises(ValueError):
        lb.lowbit_lora_add(x, ids, a[0], b[0].transpose(1, 2), base[0], y, workspace=ws)
    with pytest.raises(ValueError):
        lb.lowbit_lora_add(x, ids, a[0], b[0], base[0].cpu(), y, workspace=ws)
    with pytest.raises(lb.LowbitError):
        lb.lowbit_lora_add(x, ids, a[0], b[0], base[0], y, workspace=ws[:16])
    with pytest.raises(lb.LowbitError):
        lb.lowbit_lora_add(x, ids, a[0], b[0], base[0], y)
