"""Attention over the KV8 cache within each kernel's own bound (attention_bounds derives them), which has to stay below a
twentieth of the largest value so that it can fail: scores of any size, sinks, rows without a place, on both kernels."""
import numpy as np
import pytest
import torch

import attention_bounds as ab
import decode_reference as ref
from parity_util import host
from test_gpu_kv8 import attend, i32, make_batch, make_cache, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lb(cuda_device):
    from decode_packed_bit_b200 import build
    build.build()
    from decode_packed_bit_b200 import lowbit
    return lowbit


def check(cache, table, lens, q, scale, row_start, out, **kw):
    arrays = [host(t) for t in (cache.k, cache.k_scales, cache.v, cache.v_scales)]
    return ab.check(arrays, table, lens, ref.bf16_to_f64(q), scale, row_start, ref.bf16_to_f64(out), **kw)


def queries(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def largest_score(cache, table, lens, q, row_start):
    """Of scale 1, over what each sequence holds."""
    most, H = 0.0, cache.n_heads
    for b, n in enumerate(lens):
        lo, hi = (b, b + 1) if row_start is None else (int(row_start[b]), int(row_start[b + 1]))
        if hi == lo or n == 0:
            continue
        ids = torch.tensor(table[b, : -(-n // cache.page_tokens)].astype(np.int64), device="cuda")
        k = (cache.k[ids].float() * cache.k_scales[ids][..., None, None]).transpose(0, 1).reshape(H, -1, cache.head_dim)[:, :n]
        s = torch.einsum("rhgd,hnd->rhgn", q[lo:hi].float().reshape(hi - lo, H, -1, cache.head_dim), k)
        most = max(most, float(s.abs().max()))
    return most


# single rows, several of them, sixteen to a tile, prompts: (H, G, D, P, lens, rows)
SHAPES = [(2, 4, 128, 64, [300, 1000, 77, 1], [1, 1, 1, 1]), (1, 8, 64, 32, [5000], [1]), (2, 5, 128, 128, [700, 90], [6, 3]),
          (4, 4, 64, 32, [140] * 48, [4] * 48), (4, 16, 128, 32, [200] * 24, [2] * 24), (8, 8, 128, 64, [400], [130]),
          (4, 8, 64, 128, [900, 300], [250, 20])]


@pytest.mark.parametrize("largest", [3.0, 1e3, 1e5, 1e6, 1e7])
@pytest.mark.parametrize("H,G,D,P,lens,rows", SHAPES)
def test_scores_of_any_size(lb, H, G, D, P, lens, rows, largest):
    n_pages, table = make_batch(sum(rows), lens, P)
    cache = make_cache(lb, D + G, n_pages, H, P, D)
    rs = starts(rows)
    q = queries(G + D, sum(rows), H * G, D)
    scale = largest / largest_score(cache, table, lens, q, rs)
    # Where the bound says nothing: a row's two largest scores lie nearer to each other than the scores' own rounding.
    # fp32 rounds scores of 10^5 to steps of 2^-7; the sums of the prompts' kernel may be off by 2 * 17 * 8 * 2^-23 of
    # sum |q k|, about 1.8 times the largest score here: 0.06 for scores of 10^3, which is 0.06 of the largest value
    # for two equal weights, and 6 for 10^5, where a row's two largest lie some thousands apart.
    loose = (0.0 if largest < 1e3 else 0.01 if largest < 1e4 else 0.08) if ab.prompts(H, G, len(lens), sum(rows)) else 0.0 if largest < 1e4 else 0.03
    for sign in (1, -1):
        out = attend(lb, cache, table, lens, q, sign * scale, rs)
        check(cache, table, lens, q, sign * scale, rs, out, loose=loose)
    assert lb.lowbit_fault_flags() == 0


@pytest.mark.parametrize("largest", [1.0, 1e5, 1e6, 1e7])
@pytest.mark.parametrize("rows,H,G", [(1, 2, 4), (9, 2, 3), (600, 2, 8)])
def test_equal_largest_scores(lb, rows, H, G, largest):
    """Four equal keys, far ahead of the others, in one tile and in two: the mean of their values, whatever their score."""
    D, P, n = 128, 32, 1000
    n_pages, table = make_batch(3, [n], P)
    cache = make_cache(lb, 2, n_pages, H, P, D)
    cache.k_scales[:] = 0.01
    cache.v_scales[:] = 0.01
    cache.k[:] = cache.k // 8
    best = torch.randint(64, 128, (D,), device="cuda", dtype=torch.int8)
    tokens = [3, 5, 350, 351]
    for t in tokens:
        cache.k[int(table[0, t // P]), :, t % P] = best
    q = (1 + torch.rand((rows, H * G, D), device="cuda")).bfloat16()
    scale = largest / float((q[0, 0].double() @ best.double()) * 0.01)
    out = attend(lb, cache, table, [n], q, scale, starts([rows])).double()
    if largest == 1.0:
        check(cache, table, [n], q, scale, starts([rows]), out)
        return
    v = torch.stack([cache.v[int(table[0, t // P]), :, t % P] for t in tokens]).double().mean(0) * 0.01  # [H][D]
    want = v.repeat_interleave(G, 0)[None]
    # each weight within 2^-11 (f16) or 2^-17, fp32 sums, bf16
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -10 * 1.27
    assert ((out - want).abs() <= tol).all()


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan"), 3e38])
@pytest.mark.parametrize("H,G,D,lens,rows", [(2, 4, 64, [2, 20, 100], [5, 30, 4]), (1, 8, 128, [1, 3], [2, 4]), (2, 4, 128, [1, 0, 33], [8, 1, 2]),
                                             (4, 8, 128, [40, 150, 90], [200, 160, 91])])
def test_rows_without_a_place_hold_anything(lb, H, G, D, lens, rows, bad):
    """Rows before the first token share tiles with rows that have one: zeros, and the others as they were."""
    n_pages, table = make_batch(D, lens, 32)
    cache = make_cache(lb, D + 1, n_pages, H, 32, D)
    rs = starts(rows)
    q = queries(D + G, sum(rows), H * G, D)
    clean = attend(lb, cache, table, lens, q, 0.1, rs)
    check(cache, table, lens, q, 0.1, rs, clean)
    for b, (n, r) in enumerate(zip(lens, rows)):
        without = int(rs[b]) + max(r - n, 0)
        q[int(rs[b]):without, :, 3] = bad
        q[int(rs[b]):without, 0, :] = bad
    for scale in (0.1, -0.1):
        out = attend(lb, cache, table, lens, q, scale, rs)
        check(cache, table, lens, q, scale, rs, out)
        if scale > 0:
            assert torch.equal(out, clean)


@pytest.mark.parametrize("lead", [8.0, 14.0, 16.4, 18.0])
@pytest.mark.parametrize("rows,H,G,D", [(1, 2, 4, 128), (9, 1, 8, 64), (600, 2, 8, 128), (1100, 8, 1, 64)])
def test_a_leading_token_without_value(lb, rows, H, G, D, lead):
    """One token leads all others by `lead` and has values of zero, so that what is left is the others' part, which
    weights of few bits would lose: the others have equal scores, and their roundings the same sign."""
    P, n = 32, 4000
    n_pages, table = make_batch(17, [n], P)
    cache = make_cache(lb, 18, n_pages, H, P, D)
    cache.k_scales[:] = 0.01
    cache.k[:] = 0
    first = int(table[0, 0])
    cache.k[first, :, 0] = 100
    cache.v[first, :, 0] = 0
    q = torch.ones((rows, H * G, D), device="cuda").bfloat16()
    out = attend(lb, cache, table, [n], q, lead / D, starts([rows]))
    check(cache, table, [n], q, lead / D, starts([rows]), out)


@pytest.mark.parametrize("power", [-50, -20, 0, 20, 45])
@pytest.mark.parametrize("rows,H,G", [(1, 2, 4), (9, 1, 8), (600, 2, 8)])
def test_pages_of_zero_values(lb, rows, H, G, power):
    """Pages whose values' scale is 0 (the first, some within, most of them) beside others of any usual magnitude."""
    D, P, n = 64, 32, 1000
    n_pages, table = make_batch(21, [n], P)
    for zero in ([0], [0, 1, 2, 3, 7, 20], list(range(0, 30)), [31]):
        cache = make_cache(lb, 22, n_pages, H, P, D)
        cache.v_scales *= 2.0 ** power
        cache.v_scales[table[0][zero].tolist()] = 0
        q = queries(23, rows, H * G, D) * 2
        out = attend(lb, cache, table, [n], q, 0.125, starts([rows]))
        check(cache, table, [n], q, 0.125, starts([rows]), out)
        assert out.any()
