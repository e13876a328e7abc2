"""The decode-side calls at the ends of their sizes: very deep and very shallow adapters, many rows, many heads, many
sequences, streams given as objects and as integers, host threads that call at once."""
import threading

import numpy as np
import pytest
import torch

import decode_reference as ref
import test_gpu_lora as lora
import test_gpu_rope as rope
from parity_util import host
from test_gpu_kv8 import attend, i32, make_batch, make_cache, starts
from test_gpu_kv8_bounds import check, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lb(cuda_device):
    from decode_packed_bit_b200 import build
    build.build()
    from decode_packed_bit_b200 import lowbit
    return lowbit


@pytest.mark.parametrize("M,N,K,rank,L", [(1, 8, 65536, 8, 1), (2, 1, 131072, 16, 3), (300, 3, 40960, 128, 2), (5, 1, 64, 8, 1),
                                          (1, 100000, 64, 8, 2), (40000, 5, 64, 8, 7), (70000, 1, 64, 24, 300)])
def test_adapters(lb, M, N, K, rank, L):
    x, ids, a, b, base, ranks, scales = lora.make(M + K, M, N, K, rank, L)
    y = torch.full((M, N), float("nan"), device="cuda")
    lb.lowbit_lora_add(x, ids, a[0], b[0], base[0], y, ranks, scales, lora.workspace(lb, 1, M, N, K, rank))
    take = np.unique(np.linspace(0, M - 1, 500).astype(int))  # the definition is a loop
    at = torch.from_numpy(take).cuda()
    lora.check(y[at], x[at], ids[at], a[0], b[0], base[0][at], ranks, scales, f"M={M} N={N} K={K} rank={rank}")
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("M,hq,hk,D,rot", [(200000, 1, 1, 8, 8), (1, 4096, 0, 64, 64), (2, 0, 3000, 24, 6), (70000, 2, 0, 16, 2), (1, 1, 0, 8, 2)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope(lb, M, hq, hk, D, rot, interleaved):
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    q = torch.randn((M, hq, D), generator=g, device="cuda") if hq else None
    k = torch.randn((M, hk, D), generator=g, device="cuda") if hk else None
    pos = torch.randint(0, 1 << 20, (M,), generator=g, device="cuda", dtype=torch.int32)
    qo, ko = (None if t is None else torch.full_like(t, float("nan")) for t in (q, k))
    lb.lowbit_rope(q, qo, k, ko, pos, lb.lowbit_rope_phases(rot).cuda(), interleaved=interleaved)
    at = torch.from_numpy(np.unique(np.linspace(0, M - 1, 300).astype(int))).cuda()
    for x, y in ((q, qo), (k, ko)):
        if x is not None:
            assert torch.isfinite(y).all()
            rope.check(y[at], x[at], pos[at], rope.frequencies(rot), interleaved, 1.0)


@pytest.mark.parametrize("H,G,D,P,B,most", [(1024, 1, 64, 32, 3, 1), (300, 4, 128, 32, 2, 3), (64, 64, 64, 32, 2, 2), (2, 4, 64, 32, 20000, 1),
                                            (1, 1, 64, 128, 5000, 3)])
def test_cache_and_attention(lb, H, G, D, P, B, most):
    g = np.random.default_rng(H + B)
    rows = [1] * B if most == 1 else [int(r) for r in g.integers(0, most + 1, B)]
    lens = [int(n) for n in g.integers(0, 50, B)]
    n_pages, table = make_batch(B, lens, P)
    cache = make_cache(lb, B, n_pages, H, P, D)
    rs, T = starts(rows), sum(rows)
    x = torch.randn((T, H, D), device="cuda")
    want = ref.append(host(cache.k), host(cache.k_scales), host(x), lens, table, rs) if H * T < 40000 else None
    for row_start in ([None] if most == 1 else []) + [i32(rs)]:
        lb.lowbit_kv8_append(cache, i32(table), i32(lens), x, x, row_start=row_start)
        if want:
            assert np.array_equal(host(cache.k), want[0]) and np.array_equal(host(cache.k_scales), want[1])
        back = torch.empty_like(x)
        lb.lowbit_kv8_read(cache, i32(table), i32(lens), back, None, row_start=row_start)
        without = torch.tensor([lens[b] - rows[b] + i < 0 for b in range(B) for i in range(rows[b])], device="cuda")
        assert (back[without] == 0).all()
        assert float((back - x)[~without].abs().max()) <= float(x.abs().max()) / 254 * 1.0001
    q = queries(B, T, H * G, D)
    out = attend(lb, cache, table, lens, q, 0.125, rs)
    check(cache, table, lens, q, 0.125, rs, out)
    assert lb.lowbit_fault_flags() == 0


def test_streams_given(lb):
    """None, an object, its integer: the call runs there, behind what was enqueued there before."""
    lens, P, H, G, D = [200, 90], 32, 2, 4, 64
    n_pages, table = make_batch(1, lens, P)
    cache = make_cache(lb, 1, n_pages, H, P, D)
    q = queries(2, 2, H * G, D)
    want = attend(lb, cache, table, lens, q, 0.1, None)
    t, n = i32(table), i32(lens)
    side = torch.cuda.Stream()
    ws = torch.zeros(lb.lowbit_kv8_attention_workspace_bytes(cache, 2, 2, H * G), dtype=torch.uint8, device="cuda")
    for given in (side, side.cuda_stream):
        late, out = torch.zeros_like(q), torch.zeros_like(q)
        w = torch.randn((4096, 4096), device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(4):
                w @ w
            late.copy_(q)
        lb.lowbit_kv8_attention(cache, t, n, late, out, 0.1, workspace=ws, stream=given)
        side.synchronize()
        assert torch.equal(out, want)


def test_host_threads(lb):
    """Threads with streams and workspaces of their own, all five calls, at once."""
    P, H, G, D, r, L = 32, 2, 4, 64, 16, 3
    done, failed = [], []

    def work(seed):
        try:
            torch.cuda.set_device(0)
            stream = torch.cuda.Stream()
            lens = [100 + seed, 37]
            n_pages, table = make_batch(seed, [300, 300], P)
            with torch.cuda.stream(stream):
                cache = make_cache(lb, seed, n_pages, H, P, D)
                x, ids, a, b, base, ranks, scales = lora.make(seed, 2, H * G * D, 256, r, L)
                q, k = torch.empty((2, H * G, D), device="cuda", dtype=torch.bfloat16), torch.randn((2, H, D), device="cuda").bfloat16()
                y, lws = torch.empty_like(base[0]), lora.workspace(lb, 1, 2, H * G * D, 256, r)
                ws = torch.zeros(lb.lowbit_kv8_attention_workspace_bytes(cache, 2, 2, H * G), dtype=torch.uint8, device="cuda")
                t, n, pos, phases = i32(table), i32(lens), i32([99 + seed, 36]), lb.lowbit_rope_phases(D).cuda()
                first = None
                for _ in range(60):
                    lb.lowbit_lora_add(x, ids, a[0], b[0], base[0], y, ranks, scales, lws)
                    lb.lowbit_rope(y.view(2, H * G, D), q, None, None, pos, phases)
                    lb.lowbit_kv8_append(cache, t, n, k, k)
                    out, back = torch.empty_like(q), torch.empty_like(k)
                    lb.lowbit_kv8_attention(cache, t, n, q, out, 0.125, workspace=ws)
                    lb.lowbit_kv8_read(cache, t, n, back, None)
                    now = [z.clone() for z in (y, q, out, back)]
                    first = first or now
                    stream.synchronize()
                    assert all(torch.equal(p, z) for p, z in zip(first, now))
                lora.check(y, x, ids, a[0], b[0], base[0], ranks, scales, f"thread {seed}")
                check(cache, table, lens, q, 0.125, None, out)
            done.append(seed)
        except BaseException as e:  # noqa: BLE001 - reported below
            failed.append((seed, repr(e)))

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(s,)) for s in range(1, 7)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not failed and sorted(done) == [1, 2, 3, 4, 5, 6], failed
    assert lb.lowbit_fault_flags() == 0
