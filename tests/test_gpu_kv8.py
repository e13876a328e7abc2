"""GPU parity of the KV8 cache: append and read bit for bit against the definition, attention within the bound that
its fixed-point steps allow (decode_reference.attention derives it), at the lengths where tiles and pages end, with
idle slots, rows without a place, absent pages, strides, captured graphs, several streams and a cache beyond 4 GB."""
import numpy as np
import pytest
import torch

import decode_reference as ref
from parity_util import host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lb(cuda_device):
    from decode_packed_bit_b200 import build
    build.build()
    from decode_packed_bit_b200 import lowbit
    return lowbit


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def make_batch(seed, lens, page, spare=3):
    """A page table with pages in random order; entries past a sequence's pages are out of range."""
    g = np.random.default_rng(seed)
    need = [-(-max(n, 0) // page) for n in lens]
    n_pages = sum(need) + spare
    order = g.permutation(n_pages)
    table = np.full((len(lens), max(need + [1]) + 1), 1 << 30, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return n_pages, table


def make_cache(lb, seed, n_pages, H, P, D):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    codes = [torch.randint(-127, 128, (n_pages, H, P, D), generator=g, device="cuda", dtype=torch.int8) for _ in range(2)]
    scales = [torch.rand((n_pages, H), generator=g, device="cuda") * 0.02 + 0.005 for _ in range(2)]
    return lb.KV8Cache(codes[0], scales[0], codes[1], scales[1])


def starts(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)


# -- append and read ----------------------------------------------------------------

@pytest.mark.parametrize("kt,vt", [(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("H,D,P,lens,rows", [
    (1, 64, 32, [1], [1]), (2, 128, 64, [64, 65, 1, 63], [1, 1, 1, 1]), (8, 128, 32, [33, 500, 7], [33, 1, 0]),
    (3, 64, 128, [300, 0, 129, 128], [260, 0, 2, 128]), (2, 128, 128, [1000, 40], [1000, 39]),
    (5, 64, 64, [70, 70, 70, 70, 70, 70], [5, 6, 7, 64, 65, 70])])
def test_append_and_read(lb, H, D, P, lens, rows, kt, vt):
    n_pages, table = make_batch(len(lens) + P, lens, P)
    cache = make_cache(lb, P + D, n_pages, H, P, D)
    T = sum(rows)
    k = (torch.randn((T, H, D), device="cuda") * torch.rand((T, 1, 1), device="cuda") * 5).to(kt)
    v = torch.randn((T, H, D), device="cuda").to(vt)
    one = all(r == 1 for r in rows)
    rs = starts(rows)
    want = [ref.append(host(c), host(s), x.float().cpu().numpy(), lens, table, rs)
            for c, s, x in ((cache.k, cache.k_scales, k), (cache.v, cache.v_scales, v))]
    for row_start in ([None] if one else []) + [i32(rs)]:
        lb.lowbit_kv8_append(cache, i32(table), i32(lens), k, v, row_start=row_start)
        for (codes, scales), c, s in zip(want, (cache.k, cache.v), (cache.k_scales, cache.v_scales)):
            assert np.array_equal(host(s), scales)
            assert np.array_equal(host(c), codes)  # a second write of the same tokens changes nothing
    # everything back, dense
    back = starts(lens)
    for dtype in (torch.float32, torch.bfloat16):
        ko, vo = (torch.full((sum(lens), H, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
        lb.lowbit_kv8_read(cache, i32(table), i32(lens), ko, vo, row_start=i32(back))
        for got, (codes, scales) in zip((ko, vo), want):
            exp = np.zeros((sum(lens), H, D), np.float32)
            for r, _, pos, page, slot in ref.places(lens, table, back, sum(lens), P, n_pages):
                exp[r] = codes[page, :, slot].astype(np.float32) * scales[page][:, None]
            assert torch.equal(got.cpu(), torch.from_numpy(exp).to(dtype))
    only = torch.empty((sum(lens), H, D), device="cuda")
    lb.lowbit_kv8_read(cache, i32(table), i32(lens), None, only, row_start=i32(back))
    assert torch.equal(only.bfloat16(), vo)
    assert lb.lowbit_fault_flags() == 0


def test_append_rounds_exactly_and_grows(lb):
    """Ties, values one unit beside them, growth over a page token by token, NaN, infinities, zeros, subnormals."""
    H, D, P = 1, 64, 32
    cache = lb.KV8Cache.empty(2, H, P, D)
    g = np.random.default_rng(3)
    codes, scales = host(cache.k).copy(), host(cache.k_scales).copy()
    table = np.array([[1]], np.int32)
    for t in range(P):
        x = np.zeros((1, H, D), np.float32)
        step = np.float32(0.37) * np.float32(1.1) ** (t // 3)
        x[0, 0, 0] = step * 127
        half = (np.arange(1, D, dtype=np.float64) - 31.5).astype(np.float32) * step
        x[0, 0, 1:] = np.where(g.random(D - 1) < 0.5, half, np.nextafter(half, np.float32(g.choice([-1e9, 1e9]))))
        if t == 20:
            x[0, 0, 5], x[0, 0, 6] = np.nan, 0.0
        if t == 25:
            x[:] = 0
        if t == 26:
            x[0, 0, :] = 1e-42
        xd = torch.from_numpy(x).cuda()
        lb.lowbit_kv8_append(cache, i32(table), i32([t + 1]), xd, xd)
        codes, scales = ref.append(codes, scales, x, [t + 1], table, None)
        assert np.array_equal(host(cache.k_scales), scales) and np.array_equal(host(cache.k), codes), f"token {t}"
        assert np.array_equal(host(cache.v), codes)
    x[0, 0, 3] = -np.inf
    xd = torch.from_numpy(x).cuda()
    lb.lowbit_kv8_append(cache, i32(table), i32([1]), xd, xd)
    codes, scales = ref.append(codes, scales, x, [1], table, None)
    assert np.isfinite(host(cache.k_scales)).all()
    assert np.array_equal(host(cache.k_scales), scales) and np.array_equal(host(cache.k), codes)
    # all-subnormal page: the scale may round to zero, the codes then are zero
    x[:] = 1e-45
    xd = torch.from_numpy(x).cuda()
    lb.lowbit_kv8_append(cache, i32([[0]]), i32([1]), xd, xd)
    codes, scales = ref.append(codes, scales, x, [1], np.array([[0]]), None)
    assert np.array_equal(host(cache.k_scales), scales) and np.array_equal(host(cache.k), codes)


def test_append_strided_from_one_buffer_and_rows_behind(lb):
    H, D, P = 2, 64, 32
    lens, rows = [40, 9], [3, 4]
    n_pages, table = make_batch(1, lens, P)
    cache = make_cache(lb, 1, n_pages, H, P, D)
    T = 12  # five rows behind the last sequence
    kv = torch.randn((T, 2 * H * D), device="cuda").bfloat16()
    kv[7:] = float("nan")
    k, v = kv[:, : H * D].view(T, H, D), kv[:, H * D:].view(T, H, D)
    want = [ref.append(host(c), host(s), x.float().cpu().numpy(), lens, table, starts(rows))
            for c, s, x in ((cache.k, cache.k_scales, k), (cache.v, cache.v_scales, v))]
    lb.lowbit_kv8_append(cache, i32(table), i32(lens), k, v, row_start=i32(starts(rows)))
    for (codes, scales), c, s in zip(want, (cache.k, cache.v), (cache.k_scales, cache.v_scales)):
        assert np.array_equal(host(s), scales) and np.array_equal(host(c), codes)
    out = torch.full((T, H, D), -3.0, device="cuda")
    lb.lowbit_kv8_read(cache, i32(table), i32(lens), out, None, row_start=i32(starts(rows)))
    assert (out[7:] == -3.0).all() and not (out[:7] == -3.0).any()


# -- attention ----------------------------------------------------------------------

def attend(lb, cache, table, lens, q, scale, row_start, ws=None, out=None):
    T, Q, _ = q.shape
    if ws is None:
        n = lb.lowbit_kv8_attention_workspace_bytes(cache, len(lens), T, Q)
        assert n > 0
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    if out is None:
        out = torch.full_like(q, -7.0)
    lb.lowbit_kv8_attention(cache, i32(table), i32(lens), q, out, scale,
                            row_start=None if row_start is None else i32(row_start), workspace=ws)
    return out


def check_attention(cache, table, lens, q, scale, row_start, out, untouched=-7.0):
    want, tol = ref.attention(host(cache.k), host(cache.k_scales), host(cache.v), host(cache.v_scales),
                              ref.bf16_to_f64(q), scale, lens, table, row_start)
    got = ref.bf16_to_f64(out)
    for r, (w, t) in enumerate(zip(want, tol)):
        if w is None:
            assert (got[r] == untouched).all(), f"row {r} behind the last sequence was written"
            continue
        diff = np.abs(got[r] - w)
        assert (diff <= t).all(), f"row {r}: {(diff > t).sum()} of {diff.size} off, worst {(diff - t).max():.3e}"


LENGTHS = [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 0, 255, 257]


@pytest.mark.parametrize("D,P", [(64, 32), (64, 64), (64, 128), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("H,G", [(1, 1), (2, 5), (1, 8), (2, 12), (1, 64)])
def test_attention_single_rows(lb, D, P, H, G):
    n_pages, table = make_batch(D + P + G, LENGTHS, P)
    cache = make_cache(lb, G, n_pages, H, P, D)
    q = torch.randn((len(LENGTHS), H * G, D), device="cuda").bfloat16()
    scale = D ** -0.5
    out = attend(lb, cache, table, LENGTHS, q, scale, None)
    check_attention(cache, table, LENGTHS, q, scale, None, out)
    assert (out[LENGTHS.index(0)] == 0).all()
    assert lb.lowbit_fault_flags() == 0


@pytest.mark.parametrize("H,G,D,P,lens,rows", [
    (2, 4, 128, 64, [100, 5, 300, 64], [3, 5, 0, 64]), (1, 5, 64, 32, [700, 90], [33, 90]),
    (3, 1, 128, 32, [40, 257, 1], [40, 17, 1]), (1, 16, 64, 128, [200], [150]),
    (2, 3, 128, 128, [600, 129], [450, 129]), (1, 8, 128, 64, [1100], [513])])
def test_attention_several_rows(lb, H, G, D, P, lens, rows):
    n_pages, table = make_batch(sum(rows), lens, P)
    cache = make_cache(lb, D, n_pages, H, P, D)
    rs = starts(rows)
    q = torch.randn((sum(rows) + 4, H * G, D), device="cuda").bfloat16() * 2
    out = attend(lb, cache, table, lens, q, 0.1, rs)
    check_attention(cache, table, lens, q, 0.1, rs, out)


# Calls that take the tcgen05 kernel: many rows.  Its steps fit the same bound: q as f16 is nearer than q's fixed
# point there, and a probability's f16 rounding, 2^-12 of itself, adds 2^-12 of the largest value, half of what the
# bound allows the fixed-point ones.
PROMPTS = [(2, 4, 128, 64, [700, 650], [600, 640]), (4, 5, 64, 32, [333, 128, 900], [200, 128, 130]),
           (8, 1, 128, 128, [1500], [1100]), (1, 64, 64, 128, [300], [150]), (3, 12, 128, 32, [400, 0, 100], [300, 5, 20]),
           (2, 3, 64, 64, [129, 1000, 128], [129, 1000, 250]), (8, 8, 128, 64, [257], [129])]


@pytest.mark.parametrize("H,G,D,P,lens,rows", PROMPTS)
def test_attention_prompts(lb, H, G, D, P, lens, rows):
    assert sum(rows) * G * H >= 8192 and sum(rows) * G >= 64 * len(rows)
    n_pages, table = make_batch(sum(rows) + D, lens, P)
    cache = make_cache(lb, D + G, n_pages, H, P, D)
    rs = starts(rows)
    q = torch.randn((sum(rows) + 3, H * G, D), device="cuda").bfloat16() * 1.5
    out = attend(lb, cache, table, lens, q, 0.1, rs)
    check_attention(cache, table, lens, q, 0.1, rs, out)
    assert lb.lowbit_fault_flags() == 0
    for _ in range(3):
        assert torch.equal(out, attend(lb, cache, table, lens, q, 0.1, rs))


def test_attention_prompts_extremes(lb):
    """Growing and falling scores, scales far apart between pages (zero among them), huge, tiny and non-finite rows of
    q, an absent page, stale codes behind the end."""
    H, G, D, P, lens, rows = 4, 4, 128, 32, [900, 300], [700, 300]
    n_pages, table = make_batch(16, lens, P)
    cache = make_cache(lb, 16, n_pages, H, P, D)
    order = table[0, :29]
    grow = torch.linspace(-3, 3, 29, device="cuda")
    cache.k_scales[order.tolist()] *= torch.exp(grow)[:, None]
    cache.v_scales[order.tolist()] *= torch.exp(-2 * grow)[:, None]
    cache.v_scales[int(order[3])] = 0
    cache.k_scales[int(order[5])] = 0
    table[1, 2] = -1
    cache.v[int(table[1, 9]), :, 12:] = 127
    rs = starts(rows)
    q = torch.randn((sum(rows), H * G, D), device="cuda").bfloat16()
    q[10, 0] *= 50
    q[11, 1] = 0
    q[12, 2] = 1e-37
    q[13, 3, 5] = 1e5
    for scale in (0.05, -0.05):
        out = attend(lb, cache, table, lens, q, scale, rs)
        check_attention(cache, table, lens, q, scale, rs, out)
    assert lb.lowbit_fault_flags() == 16
    z = q.clone()
    z[500, 7, 100], z[800, 3, 0] = float("nan"), float("-inf")
    got = attend(lb, cache, table, lens, z, -0.05, rs)
    assert torch.isnan(got[500, 7]).all() and torch.isnan(got[800, 3]).all()
    keep = torch.ones(got.shape[:2], dtype=torch.bool, device="cuda")
    keep[500, 7] = keep[800, 3] = False
    assert torch.equal(got[keep], out[keep])
    assert lb.lowbit_fault_flags() == 16


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("scale", [-0.1, 0.0])
def test_attention_scale_of_any_sign(lb, n, scale):
    lens = [100, 70]
    n_pages, table = make_batch(15, lens, 32)
    cache = make_cache(lb, 15, n_pages, 2, 32, 64)
    q = torch.randn((2 * n, 8, 64), device="cuda").bfloat16()
    out = attend(lb, cache, table, lens, q, scale, starts([n, n]))
    check_attention(cache, table, lens, q, scale, starts([n, n]), out)


@pytest.mark.parametrize("rows", [[1, 1, 1], [300, 200, 90]])
def test_attention_rows_without_a_place(lb, rows):
    """More rows than tokens: those before the first token see nothing and give zeros."""
    lens = [0, 20, 100]
    n_pages, table = make_batch(9, lens, 32)
    cache = make_cache(lb, 9, n_pages, 2, 32, 64)
    q = torch.randn((sum(rows), 4, 64), device="cuda").bfloat16()
    q[0] = float("nan")  # a row that sees nothing: zeros, whatever it holds
    out = attend(lb, cache, table, lens, q, 0.125, starts(rows))
    assert (out[0] == 0).all()
    q[0] = 0
    check_attention(cache, table, lens, q, 0.125, starts(rows), out)


@pytest.mark.parametrize("n", [1, 70])
def test_attention_extreme_values(lb, n):
    """One token outweighs the rest by far; all weights equal; tiny and huge q; a NaN row stays by itself."""
    H, G, D, P, lens = 1, 4, 128, 64, [500, 500]
    n_pages, table = make_batch(4, lens, P)
    cache = make_cache(lb, 4, n_pages, H, P, D)
    q = torch.randn((2 * n, G, D), device="cuda").bfloat16()
    q[0, 0] *= 40
    q[0, 1] = 0
    q[0, 2] = 1e-38
    q[0, 3, 7] = 3e4
    rs = starts([n, n])
    out = attend(lb, cache, table, lens, q, 0.1, rs)
    check_attention(cache, table, lens, q, 0.1, rs, out)
    for bad in (float("nan"), float("inf")):
        z = q.clone()
        z[n, 1, 3] = bad
        got = attend(lb, cache, table, lens, z, 0.1, rs)
        assert torch.isnan(got[n, 1]).all()
        keep = torch.ones(got.shape[:2], dtype=torch.bool)
        keep[n, 1] = False
        assert torch.equal(got[keep.cuda()], out[keep.cuda()])


def test_attention_does_not_read_past_the_length(lb):
    """Stale codes of the last page and scales of other pages cannot reach the result."""
    lens, P = [37, 90], 64
    n_pages, table = make_batch(5, lens, P)
    cache = make_cache(lb, 5, n_pages, 2, P, 128)
    q = torch.randn((2, 6, 128), device="cuda").bfloat16()
    out = attend(lb, cache, table, lens, q, 0.1, None)
    used = set()
    for b, n in enumerate(lens):
        last = int(table[b, (n - 1) // P])
        cache.k[last, :, (n - 1) % P + 1:] = 127
        cache.v[last, :, (n - 1) % P + 1:] = -127
        used |= set(table[b, : -(-n // P)].tolist())
    for p in set(range(n_pages)) - used:
        cache.k_scales[p] = cache.v_scales[p] = float("nan")
    assert torch.equal(out, attend(lb, cache, table, lens, q, 0.1, None))


@pytest.mark.parametrize("n", [1, 100])
def test_out_of_range_pages_and_lengths_are_counted_out(lb, n):
    lens, P, H, D = [200, 130, 150], 32, 2, 64
    n_pages, table = make_batch(6, lens, P)
    cache = make_cache(lb, 6, n_pages, H, P, D)
    table = table[:, :7].copy()
    table[0, 2], table[0, 3], table[1, 0] = -1, n_pages, -(1 << 31)
    table[2, :] = 1 << 30
    rs = starts([n] * 3)
    q = torch.randn((3 * n, H * 3, D), device="cuda").bfloat16()
    assert lb.lowbit_fault_flags() == 0
    out = attend(lb, cache, table, lens, q, 0.1, rs)
    assert lb.lowbit_fault_flags() == 16
    check_attention(cache, table, lens, q, 0.1, rs, out)
    assert (out[2 * n:] == 0).all()
    # a length beyond the table is clamped, a negative one is zero
    table[2, :] = table[1, :]
    long = [10 ** 6, -3, 150]
    out = attend(lb, cache, table, long, q, 0.1, rs)
    check_attention(cache, table, long, q, 0.1, rs, out)
    assert lb.lowbit_fault_flags() == 16
    # append and read: absent pages are not written and read as zeros
    x = torch.randn((3 * n, H, D), device="cuda")
    want = ref.append(host(cache.k), host(cache.k_scales), host(x), lens, table, rs) if n == 1 else None
    if n == 1:
        table[2, 4] = -5  # page of the last sequence's new token
        want = ref.append(host(cache.k), host(cache.k_scales), host(x), lens, table, rs)
        lb.lowbit_kv8_append(cache, i32(table), i32(lens), x, x, row_start=i32(rs))
        assert np.array_equal(host(cache.k), want[0]) and np.array_equal(host(cache.k_scales), want[1])
        back = torch.full_like(x, 9.0)
        lb.lowbit_kv8_read(cache, i32(table), i32(lens), back, None, row_start=i32(rs))
        assert (back[2] == 0).all()
        assert lb.lowbit_fault_flags() == 16
    assert lb.lowbit_fault_flags() == 0


def test_rows_out_of_range_are_skipped(lb):
    lens, P, H, D = [60, 60, 60], 32, 1, 64
    n_pages, table = make_batch(7, lens, P)
    cache = make_cache(lb, 7, n_pages, H, P, D)
    q = torch.randn((10, 2, D), device="cuda").bfloat16()
    for rs in ([0, 4, 8, 1000], [-5, 3, 2, 10], [12, 13, 14, 15]):
        rs = np.array(rs, np.int32)
        out = attend(lb, cache, table, lens, q, 0.1, rs)
        covered = {r for r, *_ in ref.places(lens, table, rs, 10, P, n_pages)}
        assert all((out[r] == -7.0).all() for r in range(10) if r not in covered)
        x = torch.randn((10, H, D), device="cuda")
        lb.lowbit_kv8_read(cache, i32(table), i32(lens), x, None, row_start=i32(rs))
        assert lb.lowbit_fault_flags() == 16


@pytest.mark.parametrize("D", [64, 128])
def test_attention_sixteen_rows_a_tile(lb, D):
    """So many units that tiles of sixteen query rows are taken: ragged rows and lengths, an idle slot, a row too many."""
    g = np.random.default_rng(D)
    H, G, P, B = 4, 4, 32, 48
    rows = [int(x) for x in g.integers(3, 6, B)]
    lens = [int(x) for x in g.integers(1, 150, B)]
    rows[5], lens[5], lens[6], rows[6] = 0, 0, 3, 5
    assert sum(rows) * G > 8 * B and -(-sum(rows) * G // (8 * B)) * B * H > 2 * 148
    n_pages, table = make_batch(D + 1, lens, P)
    cache = make_cache(lb, D + 2, n_pages, H, P, D)
    q = torch.randn((sum(rows) + 2, H * G, D), device="cuda").bfloat16()
    rs = starts(rows)
    out = attend(lb, cache, table, lens, q, D ** -0.5, rs)
    check_attention(cache, table, lens, q, D ** -0.5, rs, out)
    assert torch.equal(out, attend(lb, cache, table, lens, q, D ** -0.5, rs))
    assert lb.lowbit_fault_flags() == 0


@pytest.mark.parametrize("rs", [[0, 500, 90, 600], [0, 500, 0, 500], [300, 600, 10, 20], [600, 500, 400, 0]])
@pytest.mark.parametrize("G", [4, 8])  # on the integer tensor cores, on tcgen05
def test_falling_row_starts_stay_inside(lb, G, rs):
    """Not allowed, and read on the device: what comes out is not defined, but nothing outside is touched."""
    P, H, D = 32, 2, 64
    lens = [600, 600, 600]
    n_pages, table = make_batch(9, lens, P)
    rs, T = np.array(rs, np.int32), 600
    cache = make_cache(lb, 9, n_pages, H, P, D)
    used = {int(p) for p in table.ravel() if p < n_pages}
    spare = [p for p in range(n_pages) if p not in used]
    before = cache.k[spare].clone()
    x = torch.randn((T, H, D), device="cuda")
    lb.lowbit_kv8_append(cache, i32(table), i32(lens), x, x, row_start=i32(rs))
    assert torch.equal(cache.k[spare], before)
    y = torch.empty_like(x)
    lb.lowbit_kv8_read(cache, i32(table), i32(lens), y, None, row_start=i32(rs))
    q = torch.randn((T, H * G, D), device="cuda").bfloat16()
    attend(lb, cache, table, lens, q, 0.1, rs)
    assert lb.lowbit_fault_flags() == 16
    assert lb.lowbit_fault_flags() == 0


def test_attention_strides(lb):
    lens, P, H, G, D = [77, 200], 32, 2, 2, 64
    n_pages, table = make_batch(8, lens, P)
    cache = make_cache(lb, 8, n_pages, H, P, D)
    buf = torch.randn((2, H * G * D + 72), device="cuda").bfloat16()
    q = buf[:, 8: 8 + H * G * D].view(2, H * G, D)
    res = torch.full((2, H * G * D + 40), -7.0, device="cuda", dtype=torch.bfloat16)
    out = res[:, 16: 16 + H * G * D].view(2, H * G, D)
    attend(lb, cache, table, lens, q, 0.2, None, out=out)
    check_attention(cache, table, lens, q, 0.2, None, out)
    assert (res[:, :16] == -7.0).all() and (res[:, 16 + H * G * D:] == -7.0).all()


@pytest.mark.parametrize("rows_each", [1, 90])
def test_attention_split_over_the_gpu_is_repeatable(lb, rows_each):
    """Long contexts cut between many CTAs: the definition, the same bits again, the workspace left zeroed."""
    lens, P, H, G, D = [9000, 33, 4100], 64, 2, 4, 128
    rows = [rows_each, 1, rows_each]
    n_pages, table = make_batch(10, lens, P)
    cache = make_cache(lb, 10, n_pages, H, P, D)
    T = sum(rows)
    q = torch.randn((T, H * G, D), device="cuda").bfloat16()
    n = lb.lowbit_kv8_attention_workspace_bytes(cache, 3, T, H * G)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    out = attend(lb, cache, table, lens, q, 0.08, starts(rows), ws=ws)
    check_attention(cache, table, lens, q, 0.08, starts(rows), out)
    for _ in range(20):
        assert torch.equal(out, attend(lb, cache, table, lens, q, 0.08, starts(rows), ws=ws))


def test_attention_many_small_sequences(lb):
    g = np.random.default_rng(11)
    lens = g.integers(0, 40, 700).tolist()
    n_pages, table = make_batch(11, lens, 32)
    cache = make_cache(lb, 11, n_pages, 2, 32, 64)
    q = torch.randn((700, 4, 64), device="cuda").bfloat16()
    out = attend(lb, cache, table, lens, q, 0.125, None)
    check_attention(cache, table, lens, q, 0.125, None, out)


def test_no_sequences_or_rows(lb):
    cache = make_cache(lb, 12, 2, 1, 32, 64)
    q = torch.zeros((0, 2, 64), device="cuda", dtype=torch.bfloat16)
    x = torch.zeros((0, 1, 64), device="cuda")
    table, lens, rs = i32([[0]]), i32([5]), i32([0, 0])
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    lb.lowbit_kv8_attention(cache, table, lens, q, q, 0.1, row_start=rs, workspace=ws)
    lb.lowbit_kv8_append(cache, table, lens, x, x, row_start=rs)
    lb.lowbit_kv8_read(cache, table, lens, x, x, row_start=rs)


@pytest.mark.parametrize("rows", [1, 80])
def test_graph_follows_lengths_and_two_streams(lb, rows):
    P, H, G, D, B = 32, 2, 4, 128, 3
    lens = [2000, 900, 400]
    n_pages, table = make_batch(13, lens, P)
    cache = make_cache(lb, 13, n_pages, H, P, D)
    q = torch.randn((B * rows, H * G, D), device="cuda").bfloat16()
    rs = starts([rows] * B)
    n = lb.lowbit_kv8_attention_workspace_bytes(cache, B, B * rows, H * G)
    t, ln, st = i32(table), i32(lens), i32(rs)
    outs, graphs, streams = [], [], []
    for s in range(2):  # two graphs on two streams, a workspace each
        out, ws = torch.full_like(q, -7.0), torch.zeros(n, dtype=torch.uint8, device="cuda")
        lb.lowbit_kv8_attention(cache, t, ln, q, out, 0.1, row_start=st, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lb.lowbit_kv8_attention(cache, t, ln, q, out, 0.1, row_start=st, workspace=ws)
        outs.append(out)
        graphs.append((graph, ws))
        streams.append(torch.cuda.Stream())
    for step in ([1500, 64, 90], [100, 900, 85], lens):
        ln.copy_(i32(step))
        torch.cuda.synchronize()
        for out in outs:
            out.fill_(-7.0)
        torch.cuda.synchronize()
        for (graph, _), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                for _ in range(3):
                    graph.replay()
        torch.cuda.synchronize()
        check_attention(cache, table, step, q, 0.1, rs, outs[0])
        assert torch.equal(outs[0], outs[1])


def test_cache_beyond_4_gigabytes(lb):
    """Pages whose byte offset does not fit in 32 bits."""
    H, P, D = 8, 128, 128
    n_pages = (1 << 32) // (H * P * D) + 40
    k = torch.empty((n_pages, H, P, D), dtype=torch.int8, device="cuda")
    v = torch.empty_like(k)
    ks, vs = (torch.empty((n_pages, H), device="cuda") for _ in range(2))
    cache = lb.KV8Cache(k, ks, v, vs)
    lens = [300, 200]
    table = np.array([[n_pages - 1, 3, n_pages - 7], [n_pages - 2, n_pages - 30, 0]], np.int32)
    T = sum(lens)
    x, y = torch.randn((T, H, D), device="cuda"), torch.randn((T, H, D), device="cuda")
    lb.lowbit_kv8_append(cache, i32(table), i32(lens), x, y, row_start=i32(starts(lens)))
    back = torch.empty_like(x)
    lb.lowbit_kv8_read(cache, i32(table), i32(lens), back, None, row_start=i32(starts(lens)))
    assert float((back - x).abs().max()) <= float(x.abs().max()) / 254 * 1.0001
    # the same pages in a small cache give the same attention, bit for bit
    used = sorted(set(table.ravel().tolist()))
    small = lb.KV8Cache(k[used].contiguous(), ks[used].contiguous(), v[used].contiguous(), vs[used].contiguous())
    renamed = np.vectorize(used.index)(table).astype(np.int32)
    for rows in ([1, 1], [150, 120]):
        q = torch.randn((sum(rows), 2 * H, D), device="cuda").bfloat16()
        a = attend(lb, cache, table, lens, q, 0.1, starts(rows))
        b = attend(lb, small, renamed, lens, q, 0.1, starts(rows))
        assert torch.equal(a, b)


def test_binding_refusals(lb):
    cache = make_cache(lb, 14, 4, 2, 32, 64)
    table, lens = i32([[0, 1]]), i32([40])
    q = torch.zeros((1, 4, 64), device="cuda", dtype=torch.bfloat16)
    x = torch.zeros((1, 2, 64), device="cuda")
    ws = torch.zeros(lb.lowbit_kv8_attention_workspace_bytes(cache, 1, 1, 4), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        lb.lowbit_kv8_attention(cache, table.long(), lens, q, q, 0.1, workspace=ws)
    with pytest.raises(ValueError):
        lb.lowbit_kv8_attention(cache, table, lens, q.float(), q, 0.1, workspace=ws)
    with pytest.raises(ValueError):
        lb.lowbit_kv8_attention(cache, table, lens, q[:, :, :32], q, 0.1, workspace=ws)
    with pytest.raises(lb.LowbitError):
        lb.lowbit_kv8_attention(cache, table, lens, q, q, 0.1, workspace=ws[:-16])
    with pytest.raises(lb.LowbitError):
        lb.lowbit_kv8_attention(cache, table, lens, q, q, float("nan"), workspace=ws)
    with pytest.raises(lb.LowbitError):
        lb.lowbit_kv8_attention(cache, table, lens, q[:, :3].contiguous(), q[:, :3].contiguous(), 0.1, workspace=ws)
    with pytest.raises(ValueError):
        lb.lowbit_kv8_append(cache, table, lens.cpu(), x, x)
    with pytest.raises(ValueError):
        lb.lowbit_kv8_append(cache, table, lens, x.transpose(1, 2), x)
    with pytest.raises(ValueError):
        lb.lowbit_kv8_read(cache, table, lens, x, x.bfloat16())
    with pytest.raises(lb.LowbitError):  # two rows, one sequence, and no row_start
        lb.lowbit_kv8_append(cache, table, lens, x.expand(2, 2, 64).contiguous(), x.expand(2, 2, 64).contiguous())
