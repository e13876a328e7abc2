"""GPU parity of lowbit_rope against the definition in 64 bits: both layouts, part of the head, every pair of types,
far and negative positions, scalings, strides, in place.  Tolerances: the angle's float carries half a turn to 2^-24,
so sine and cosine are off by at most 2^-22 with sincospif's own error, and the two products and their sum by three
roundings; 2^-20 (|a| + |b|) magnitude covers them.  A bf16 output adds half a step, 2^-8 of the value."""
import math

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


def frequencies(rot, base=10000.0):
    return [base ** (-2.0 * j / rot) for j in range(rot // 2)]


def check(got, x, positions, freq, interleaved, magnitude):
    x64 = x.detach().cpu().double().numpy()
    want = ref.rope(x64, host(positions), freq, interleaved, magnitude)
    half = len(freq)
    other = np.zeros_like(x64)
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    other[..., ia] = other[..., ib] = np.abs(x64[..., ia]) + np.abs(x64[..., ib])
    tol = 2.0 ** -20 * abs(magnitude) * other
    if got.dtype is torch.bfloat16:
        tol = tol * 1.01 + 2.0 ** -8 * np.abs(want)
    diff = np.abs(got.detach().cpu().double().numpy() - want)
    assert (diff <= tol).all(), f"{(diff > tol).sum()} of {diff.size} off, worst {(diff - tol).max():.3e}"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("src,dst", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.bfloat16),
                                     (torch.float32, torch.float32), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("M,hq,hk,D,rot", [(1, 4, 1, 128, 128), (7, 5, 3, 64, 32), (3, 2, 2, 24, 10), (2, 1, 1, 8, 2),
                                           (130, 40, 8, 128, 64), (5, 3, 1, 256, 256), (2, 1, 2, 1024, 1024)])
def test_matches_definition(lb, M, hq, hk, D, rot, src, dst, interleaved):
    g = torch.Generator(device="cuda")
    g.manual_seed(M * D + rot)
    q = torch.randn((M, hq, D), generator=g, device="cuda").to(src)
    k = torch.randn((M, hk, D), generator=g, device="cuda").to(src)
    pos = torch.randint(0, 1 << 20, (M,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = (1 << 31) - 1 if M > 1 else 0
    if M > 2:
        pos[1] = -12345
    f = frequencies(rot)
    phases = lb.lowbit_rope_phases(rot).cuda()
    qo, ko = torch.full_like(q, float("nan"), dtype=dst), torch.full_like(k, float("nan"), dtype=dst)
    lb.lowbit_rope(q, qo, k, ko, pos, phases, interleaved=interleaved, magnitude=1.25)
    check(qo, q, pos, f, interleaved, 1.25)
    check(ko, k, pos, f, interleaved, 1.25)
    if src is dst:  # in place, one of the two absent
        z = q.clone()
        lb.lowbit_rope(z, z, None, None, pos, phases, interleaved=interleaved, magnitude=1.25)
        assert torch.equal(z, qo)
    only = torch.empty_like(ko)
    lb.lowbit_rope(None, None, k, only, pos, phases, interleaved=interleaved, magnitude=1.25)
    assert torch.equal(only, ko)


def test_strided_rows_leave_the_rest(lb):
    """q and k inside one buffer of q, k and v, turned in place: v stays."""
    M, hq, hk, D = 19, 6, 2, 64
    qkv = torch.randn((M, (hq + 2 * hk) * D), device="cuda")
    before = qkv.clone()
    q = qkv[:, : hq * D].view(M, hq, D)
    k = qkv[:, hq * D:(hq + hk) * D].view(M, hk, D)
    pos = torch.arange(M, device="cuda", dtype=torch.int32) * 1000
    lb.lowbit_rope(q, q, k, k, pos, lb.lowbit_rope_phases(D).cuda())
    check(q, before[:, : hq * D].reshape(M, hq, D), pos, frequencies(D), False, 1.0)
    check(k, before[:, hq * D:(hq + hk) * D].reshape(M, hk, D), pos, frequencies(D), False, 1.0)
    assert torch.equal(qkv[:, (hq + hk) * D:], before[:, (hq + hk) * D:])


def test_relative_positions_only(lb):
    """Products of turned queries and keys depend on the difference of their positions, far out as well as near."""
    D = 128
    q, k = torch.randn((1, 1, D), device="cuda"), torch.randn((1, 1, D), device="cuda")
    phases = lb.lowbit_rope_phases(D).cuda()
    dots = []
    for at in (0, 1000, 1 << 20, (1 << 31) - 64):
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        lb.lowbit_rope(q, qo, None, None, torch.tensor([at + 13], dtype=torch.int32, device="cuda"), phases)
        lb.lowbit_rope(None, None, k, ko, torch.tensor([at], dtype=torch.int32, device="cuda"), phases)
        dots.append(float((qo.double() * ko.double()).sum()))
    norm = float(q.double().norm() * k.double().norm())
    # four roundings of 2^-20 a value pair at most, and a frequency's own rounding of 2^-65 turns a position
    assert max(dots) - min(dots) <= 2.0 ** -18 * norm


def test_graph_follows_positions(lb):
    M, D = 4, 64
    q = torch.randn((M, 2, D), device="cuda")
    out = torch.empty_like(q)
    pos = torch.zeros(M, dtype=torch.int32, device="cuda")
    phases = lb.lowbit_rope_phases(D).cuda()
    lb.lowbit_rope(q, out, None, None, pos, phases)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lb.lowbit_rope(q, out, None, None, pos, phases)
    for step in (5, 6):
        pos.fill_(step)
        graph.replay()
        check(out, q, pos, frequencies(D), False, 1.0)
