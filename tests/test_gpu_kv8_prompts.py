"""The prompts' kernel of the KV8 attention (tcgen05) as a serving program runs it: captured and replayed while lengths, rows
and pages change, beside other calls on other streams, with lengths, pages and rows out of range, strided rows, many short
sequences.  Every call here is large enough to take that kernel, which each test asserts."""
import numpy as np
import pytest
import torch

import attention_bounds as ab
from test_gpu_decode_step import Block, HIDDEN, tokens
from test_gpu_kv8 import attend, i32, make_batch, make_cache, starts
from test_gpu_kv8_bounds import check, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lb(cuda_device):
    from decode_packed_bit_b200 import build
    build.build()
    from decode_packed_bit_b200 import lowbit
    return lowbit


def workspace(lb, cache, B, T, Q):
    return torch.zeros(lb.lowbit_kv8_attention_workspace_bytes(cache, B, T, Q), dtype=torch.uint8, device="cuda")


# lengths and row starts that a replay meets: other ones, an idle slot, none at all, beyond the table, negative
STEPS = [([600, 300, 200], [0, 100, 190, 270]), ([33, 640, 90], [0, 1, 270, 270]), ([0, 300, 200], [0, 0, 130, 270]),
         ([5000, -7, 64], [0, 90, 180, 270]), ([100, 20, 270], [0, 90, 150, 200]), ([0, 0, 0], [0, 90, 180, 270])]


@pytest.mark.parametrize("D,P", [(64, 32), (128, 64)])
def test_graph_follows_lengths_and_two_streams(lb, D, P):
    H, G, T = 4, 8, 270
    assert ab.prompts(H, G, 3, T)
    n_pages, table = make_batch(3, [640, 640, 640], P)
    table = np.ascontiguousarray(table[:, : 640 // P])  # as wide as the longest: 5000 is clamped to 640
    cache = make_cache(lb, 5, n_pages, H, P, D)
    q = queries(1, T, H * G, D)
    t, ln, st = i32(table), i32(STEPS[0][0]), i32(STEPS[0][1])
    outs, graphs, streams = [], [], []
    for _ in range(2):
        out, ws = torch.full_like(q, -7.0), workspace(lb, cache, 3, T, H * G)
        lb.lowbit_kv8_attention(cache, t, ln, q, out, 0.1, row_start=st, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lb.lowbit_kv8_attention(cache, t, ln, q, out, 0.1, row_start=st, workspace=ws)
        outs.append(out)
        graphs.append((graph, ws))
        streams.append(torch.cuda.Stream())
    # a decode batch on a third stream, all the while
    side, one = torch.cuda.Stream(), queries(2, 3, H * G, D)
    beside, side_ws = torch.empty_like(one), workspace(lb, cache, 3, 3, H * G)
    side_len = i32([600, 77, 300])
    torch.cuda.synchronize()
    for lens, rs in STEPS:
        ln.copy_(i32(lens))
        st.copy_(i32(rs))
        for out in outs:
            out.fill_(-7.0)
        torch.cuda.synchronize()
        for (graph, _), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                for _ in range(3):
                    graph.replay()
        with torch.cuda.stream(side):
            for _ in range(5):
                lb.lowbit_kv8_attention(cache, t, side_len, one, beside, 0.1, workspace=side_ws)
        torch.cuda.synchronize()
        check(cache, table, lens, q, 0.1, rs, outs[0])
        assert torch.equal(outs[0], outs[1])
        assert torch.equal(outs[0], attend(lb, cache, table, lens, q, 0.1, rs))  # eager, the same bits
        check(cache, table, [600, 77, 300], one, 0.1, None, beside)
        assert lb.lowbit_fault_flags() == (16 if max(lens) > 640 or min(lens) < 0 else 0)


@pytest.mark.parametrize("D", [64, 128])
def test_pages_lengths_and_rows_out_of_range(lb, D):
    H, G, P, lens, rows = 4, 8, 32, [400, 330, 150], [150, 100, 110]
    T = sum(rows)
    assert ab.prompts(H, G, 3, T)
    n_pages, table = make_batch(6, lens, P)
    cache = make_cache(lb, 6, n_pages, H, P, D)
    table = table[:, :13].copy()
    table[0, 2], table[0, 3], table[0, 12], table[1, 0], table[1, 5] = -1, n_pages, 1 << 30, -(1 << 31), (1 << 31) - 1
    table[2, :] = 1 << 30
    q = queries(3, T, H * G, D)
    assert lb.lowbit_fault_flags() == 0
    out = attend(lb, cache, table, lens, q, 0.1, starts(rows))
    assert lb.lowbit_fault_flags() == 16
    check(cache, table, lens, q, 0.1, starts(rows), out)
    assert (out[250:] == 0).all()
    table[2, :] = table[1, :]
    for lens in ([10 ** 6, -3, 150], [2 ** 31 - 1, -2 ** 31, 1]):
        out = attend(lb, cache, table, lens, q, 0.1, starts(rows))
        check(cache, table, lens, q, 0.1, starts(rows), out)
        assert lb.lowbit_fault_flags() == 16
    lens = [400, 330, 150]
    for rs in ([0, 120, 300, 100000], [-5, 100, 200, T], [T + 2, T + 3, T + 4, T + 5], [50, 50, 300, 301]):
        rs = np.array(rs, np.int32)
        out = attend(lb, cache, table, lens, q, 0.1, rs)
        check(cache, table, lens, q, 0.1, rs, out)
        assert lb.lowbit_fault_flags() == 16  # the absent pages, or the rows


@pytest.mark.parametrize("D", [64, 128])
def test_strides(lb, D):
    H, G, P, lens, rows = 2, 16, 64, [300, 200], [180, 90]
    T, Q = sum(rows), H * G
    assert ab.prompts(H, G, 2, T)
    n_pages, table = make_batch(8, lens, P)
    cache = make_cache(lb, 8, n_pages, H, P, D)
    buf = queries(4, T + 2, Q * D + 72)
    q = buf[:T, 8: 8 + Q * D].view(T, Q, D)
    res = torch.full((T + 2, Q * D + 40), -7.0, device="cuda", dtype=torch.bfloat16)
    out = res[:T, 16: 16 + Q * D].view(T, Q, D)
    attend(lb, cache, table, lens, q, 0.1, starts(rows), out=out)
    check(cache, table, lens, q, 0.1, starts(rows), out)
    assert (res[:, :16] == -7.0).all() and (res[:, 16 + Q * D:] == -7.0).all() and (res[T:] == -7.0).all()
    z = q.clone()  # in place: every row of q is read by the one CTA that writes it
    attend(lb, cache, table, lens, z, 0.1, starts(rows), out=z)
    assert torch.equal(z, out)


def test_many_short_sequences(lb):
    """More pairs of tiles than a CTA's threads rank by length: they go in the order of the rows."""
    H, G, D, P, B = 2, 8, 64, 32, 450
    g = np.random.default_rng(2)
    rows = [int(x) for x in g.integers(8, 40, B)]
    lens = [max(0, r + int(x)) for r, x in zip(rows, g.integers(-10, 60, B))]
    assert ab.prompts(H, G, B, sum(rows))
    n_pages, table = make_batch(2, lens, P)
    cache = make_cache(lb, 2, n_pages, H, P, D)
    q = queries(5, sum(rows) + 3, H * G, D)
    out = attend(lb, cache, table, lens, q, 0.125, starts(rows))
    check(cache, table, lens, q, 0.125, starts(rows), out)
    assert lb.lowbit_fault_flags() == 0


@pytest.mark.parametrize("G,H", [(1, 16), (3, 8), (5, 8), (32, 4), (64, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_groups_of_heads(lb, G, H, D):
    """Rows that do not fill a tile of 128, one and many heads to a cache head, lengths where tiles and steps end."""
    P = 128
    most = -(-8192 // (G * H))
    lens = [most + 1, 128, 129, 256, 127, 1]
    rows = [most, 60, 129, 1, 127, 1]
    while sum(rows) * G < 64 * len(rows):
        rows[0], lens[0] = rows[0] * 2, lens[0] * 2
    assert ab.prompts(H, G, len(lens), sum(rows))
    n_pages, table = make_batch(G, lens, P)
    cache = make_cache(lb, G + 1, n_pages, H, P, D)
    q = queries(G, sum(rows), H * G, D)
    out = attend(lb, cache, table, lens, q, D ** -0.5, starts(rows))
    check(cache, table, lens, q, D ** -0.5, starts(rows), out)


def test_decoder_block_with_long_prompts(lb):
    """Projections, adapters, rotary positions, cache and attention together, with prompts of this size, and the same
    captured: the eager bits, twice over."""
    rows = [600, 70, 0, 430]
    T = sum(rows)
    assert ab.prompts(2, 4, 4, T)
    rs = starts(rows)
    ids = i32([i for i, n in zip([0, 2, 1, -1], rows) for _ in range(n)])
    positions, lens, x = i32([p for n in rows for p in range(n)]), i32(rows), tokens(7, T)
    eager, replayed = Block(lb, 6, 4, T, 20), Block(lb, 6, 4, T, 20)
    o, rec = eager.step(x, ids, positions, lens, i32(rs), keep=True)
    eager.check(x, ids, positions, lens, i32(rs), o, rec)
    check(eager.cache, eager.table, rows, rec["rope"][0], 64 ** -0.5, rs, rec["att"])
    drs = i32(rs)
    replayed.step(x, ids, positions, lens, drs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = replayed.step(x, ids, positions, lens, drs)
    for seed in (7, 8):
        x.copy_(tokens(seed, T))
        graph.replay()
        assert torch.equal(out, eager.step(x, ids, positions, lens, drs)[0])
        for name in ("k", "k_scales", "v", "v_scales"):
            assert torch.equal(getattr(eager.cache, name), getattr(replayed.cache, name))
    assert out.shape == (T, HIDDEN) and lb.lowbit_fault_flags() == 0
