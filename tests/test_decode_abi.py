"""Refusals and host-side parts of the decode-side entry points (adapters, rotary positions, KV8 cache).  CPU only:
every case fails validation, is an empty no-op, or runs on the host."""
import ctypes
import functools
import math

import pytest

from decode_packed_bit_b200 import build as lb_build

FAKE, MIS = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lb():
    lb_build.build()
    from decode_packed_bit_b200 import lowbit
    lowbit.lib()
    return lowbit


def test_lora_refusals(lb):
    f = lb.lib().lowbit_lora_add

    def call(x=FAKE, ids=FAKE, a=FAKE, b=FAKE, ranks=None, scales=None, base=FAKE, y=FAKE, M=4, N=64, K=128, rank=16,
             L=2, ws=FAKE, n=0):
        return f(x, ids, a, b, ranks, scales, base, y, M, N, K, rank, L, ws, n, None)

    need = lb.lowbit_lora_workspace_bytes(1, 4, 64, 128, 16)
    assert need > 0
    assert call(n=need - 1) == 1                       # workspace too small
    assert call(ws=None, n=need) == 1
    assert call(ws=MIS, n=need) == 2
    for name in ("x", "ids", "a", "b", "base", "y"):
        assert call(**{name: None}, n=BIG) == 1, name
        assert call(**{name: MIS}, n=BIG) == 2, name
    assert call(ranks=MIS, n=BIG) == 2
    assert call(scales=MIS, n=BIG) == 2
    assert call(M=0, n=BIG) == 1
    assert call(N=0, n=BIG) == 1
    assert call(L=0, n=BIG) == 1
    assert call(K=96, n=BIG) == 3                      # K % 64
    assert call(rank=12, n=BIG) == 3                   # rank % 8
    assert call(rank=136, n=BIG) == 3                  # rank > 128
    assert call(M=1 << 30, N=1 << 20, n=BIG) == 3      # outputs beyond 2^40
    assert call(L=(1 << 31) - 1, N=4096, n=BIG) == 3   # adapters beyond 2^40
    assert lb.lowbit_lora_workspace_bytes(1, 4, 64, 100, 16) == 0
    g = lb.lib().lowbit_lora_add_group
    pp = ctypes.cast((ctypes.c_void_p * 2)(0x10000, 0x10000), ctypes.c_void_p)
    bad = ctypes.cast((ctypes.c_void_p * 2)(0x10000, 0), ctypes.c_void_p)
    mis = ctypes.cast((ctypes.c_void_p * 2)(0x10000, 0x10008), ctypes.c_void_p)
    assert g(FAKE, FAKE, pp, pp, None, None, pp, pp, 0, 4, 64, 128, 16, 2, FAKE, BIG, None) == 1
    assert g(FAKE, FAKE, pp, pp, None, None, pp, pp, 17, 4, 64, 128, 16, 2, FAKE, BIG, None) == 1
    assert g(FAKE, FAKE, pp, bad, None, None, pp, pp, 2, 4, 64, 128, 16, 2, FAKE, BIG, None) == 1
    assert g(FAKE, FAKE, pp, pp, None, None, mis, pp, 2, 4, 64, 128, 16, 2, FAKE, BIG, None) == 2


def test_rope_refusals(lb):
    f = lb.lib().lowbit_rope

    def call(q=FAKE, qs=256, qo=FAKE, qos=256, qh=2, k=FAKE, ks=128, ko=FAKE, kos=128, kh=1, ti=0, to=1, pos=FAKE,
             ph=FAKE, M=2, D=128, rot=64):
        return f(q, qs, qo, qos, qh, k, ks, ko, kos, kh, ti, to, pos, ph, M, D, rot, 0, 1.0, None)

    other = ctypes.c_void_p(0x20000)
    assert call(qo=other, M=0, ko=other) == 1
    assert call() == 1                                 # in place with different types
    assert call(qo=other, ko=other, qs=248) == 1       # stride below a row
    assert call(qo=other, ko=other, qs=257) == 2
    assert call(qo=other, ko=other, rot=63) == 3
    assert call(qo=other, ko=other, rot=130) == 3
    assert call(qo=other, ko=other, D=12, rot=4) == 3
    assert call(qo=other, ko=other, D=2048) == 3
    assert call(qo=other, ko=other, ti=2) == 1
    assert call(qo=other, ko=other, pos=None) == 1
    assert call(qo=other, ko=other, ph=MIS) == 2
    assert call(q=None, qo=other, ko=other) == 1
    assert call(qo=MIS, ko=other) == 2
    assert call(qh=0, kh=0) == 1
    assert call(qo=other, ko=other, qs=1 << 40) == 3


def test_rope_phases(lb):
    def turns(t):
        return [(int(p) & (2 ** 64 - 1)) / 2.0 ** 64 for p in t.tolist()]

    rot = 64
    plain = [10000.0 ** (-2.0 * j / rot) for j in range(rot // 2)]
    for got, f in zip(turns(lb.lowbit_rope_phases(rot)), plain):
        assert got == pytest.approx(f / (2 * math.pi), rel=1e-14)
    for got, f in zip(turns(lb.lowbit_rope_phases(rot, scaling="linear", factor=4.0)), plain):
        assert got == pytest.approx(f / 4 / (2 * math.pi), rel=1e-14)
    base = turns(lb.lowbit_rope_phases(rot, scaling="base", factor=8.0))
    assert base[0] == pytest.approx(plain[0] / (2 * math.pi), rel=1e-14)
    assert base[-1] == pytest.approx(plain[-1] / 8 / (2 * math.pi), rel=1e-12)
    bands = turns(lb.lowbit_rope_phases(rot, scaling="bands", factor=8.0, trained_length=4096, slow=1.0, fast=32.0))
    for got, f in zip(bands, plain):
        u = 4096 * f / (2 * math.pi)
        c = min(1.0, max(0.0, (u - 1.0) / 31.0))
        assert got == pytest.approx((c * f + (1 - c) * f / 8) / (2 * math.pi), rel=1e-12)
    assert turns(lb.lowbit_rope_phases(2)) == pytest.approx([1 / (2 * math.pi)])
    assert turns(lb.lowbit_rope_phases(2, scaling="base", factor=2.0)) == pytest.approx([1 / (2 * math.pi)])
    f = lb.lib().lowbit_rope_phases
    buf = ctypes.cast((ctypes.c_int64 * 64)(), ctypes.c_void_p)
    assert f(4, 64, 1e4, 1.0, 0.0, 0.0, 0.0, buf) == 1          # unknown scaling
    assert f(0, 63, 1e4, 1.0, 0.0, 0.0, 0.0, buf) == 3
    assert f(0, 64, 1.0, 1.0, 0.0, 0.0, 0.0, buf) == 1          # base <= 1
    assert f(0, 64, float("nan"), 1.0, 0.0, 0.0, 0.0, buf) == 1
    assert f(1, 64, 1e4, 0.5, 0.0, 0.0, 0.0, buf) == 1          # factor < 1
    assert f(3, 64, 1e4, 2.0, 4096.0, 4.0, 4.0, buf) == 1       # fast <= slow
    assert f(0, 64, 1e4, 1.0, 0.0, 0.0, 0.0, None) == 1


def kv8(lb, cache=(), batch=()):
    c = dict(k=0x10000, k_scales=0x10000, v=0x10000, v_scales=0x10000, n_pages=8, n_heads=2, page_tokens=32, head_dim=64)
    b = dict(kv_len=0x10000, page_table=0x10000, row_start=0x10000, n_seqs=2, max_pages=4, n_rows=3)
    c.update(cache)
    b.update(batch)
    return lb._KV8CacheC(**c), lb._KV8BatchC(**b)


def test_argument_blocks(lb):
    """A block carries every parameter to its place: each one's refusal comes back through it as it does from the call."""
    torch = pytest.importorskip("torch")
    from decode_packed_bit_b200 import _marshal as m
    L = lb.lib()
    at = 0x10000

    def call(name, *words):
        return m.call(ctypes.cast(getattr(L, f"lowbit_{name}_args"), ctypes.c_void_p).value, *words)

    def lora(x=at, ids=at, ranks=0, scales=0, R=1, M=4, N=64, K=128, rank=16, adapters=2, ws=at, n=BIG, a=at, b=at, base=at, y=at):
        return call("lora_add_group", x, ids, ranks, scales, R, M, N, K, rank, adapters, ws, n, 0, a, b, base, y)

    for name in ("x", "ids", "a", "b", "base", "y"):
        assert lora(**{name: 0}) == 1 and lora(**{name: at + 8}) == 2, name
    assert lora(ranks=at + 8) == 2 and lora(scales=at + 8) == 2 and lora(ws=at + 8) == 2 and lora(ws=0) == 1
    assert lora(R=0) == 1 and lora(R=17) == 1 and lora(M=0) == 1 and lora(N=0) == 1 and lora(K=96) == 3
    assert lora(rank=12) == 3 and lora(adapters=0) == 1 and lora(n=16) == 1

    names = "q qs qo qos qh k ks ko kos kh ti to pos ph M D rot inter mag stream".split()
    base = dict(q=at, qs=256, qo=2 * at, qos=256, qh=2, k=at, ks=128, ko=2 * at, kos=128, kh=1, ti=0, to=1, pos=at, ph=at,
                M=2, D=128, rot=64, inter=0, mag=1.0, stream=0)

    def rope(**kw):
        return call("rope", *[{**base, **kw}[n] for n in names])

    for name in ("q", "qo", "k", "ko", "pos", "ph"):
        assert rope(**{name: 0}) == 1 and rope(**{name: at + 8}) == 2, name
    for name in ("qs", "qos", "ks", "kos"):
        assert rope(**{name: 0}) == 1 and rope(**{name: 1 << 40}) == 3, name
    assert rope(qh=-1) == 1 and rope(kh=-1) == 1 and rope(ti=2) == 1 and rope(to=2) == 1 and rope(M=0) == 1
    assert rope(D=12) == 3 and rope(rot=63) == 3

    c, b = kv8(lb)
    cache, batch = ctypes.addressof(c), [at, at, at, 2, 4, 3]
    append, read, attend = (functools.partial(call, n) for n in ("kv8_append", "kv8_read", "kv8_attention"))
    good = [at, 128, 0, at, 128, 0, 0]
    for i, bad in ((0, at + 8), (1, 132), (3, at + 8), (4, 132)):
        assert append(cache, *batch, *good[:i], bad, *good[i + 1:]) == 2
    for i, bad in ((2, 2), (5, 2)):
        assert append(cache, *batch, *good[:i], bad, *good[i + 1:]) == 1
    assert read(cache, *batch, at + 8, 0, 0, 0) == 2 and read(cache, *batch, 0, at + 8, 0, 0) == 2
    assert read(cache, *batch, at, 0, 5, 0) == 1
    good = [at, 256, 4, 0.1, at, 256, at, BIG, 0]
    for i, bad, status in ((0, at + 8, 2), (1, 260, 2), (2, 3, 1), (3, float("nan"), 1), (4, at + 8, 2), (5, 260, 2), (6, at + 8, 2),
                           (7, 16, 1)):
        assert attend(cache, *batch, *good[:i], bad, *good[i + 1:]) == status, i
    for i, bad, status in ((0, 0, 1), (1, at + 4, 2), (2, at + 4, 2), (3, -1, 1), (4, 0, 1), (5, -1, 1)):
        broken = batch[:i] + [bad] + batch[i + 1:]
        assert append(cache, *broken, at, 128, 0, at, 128, 0, 0) == status
        assert read(cache, *broken, at, at, 0, 0) == status
        assert attend(cache, *broken, *good) == status
    for f, n in ((append, 14), (read, 11), (attend, 16)):
        assert f(None, *batch, *[0] * (n - 7)) == 1
    for name in ("lora_add_group", "rope", "kv8_append", "kv8_read", "kv8_attention"):
        assert getattr(L, f"lowbit_{name}_args")(None) == 1
    # the module's own refusals
    with pytest.raises(TypeError):
        m.call(1, *[0] * 200)
    with pytest.raises(TypeError):
        m.call()
    with pytest.raises(TypeError):
        m.call(1, "x")
    with pytest.raises(OverflowError):
        m.call(1, 1 << 63)
    t = torch.zeros((2, 3, 8))
    for f in (m.dense, m.rows):
        with pytest.raises(ValueError, match="x: expected .* on cuda:0, got torch.float32"):
            f(t, torch.float32, (2, 3, 8), "x", 0)  # not on a GPU
        with pytest.raises(TypeError):
            f(None, torch.float32, (2, 3, 8), "x", 0)
        with pytest.raises(TypeError):
            f(t, torch.float32, [2, 3, 8], "x", 0)
        with pytest.raises(TypeError):
            f(t, torch.float32, (2, 3, 8), "x")
    with pytest.raises(ValueError):
        m.scratch(t, 0)
    for kind in (t.to_sparse(), t.to("meta")):
        for f in (lambda x: m.dense(x, torch.float32, (2, 3, 8), "x", 0), lambda x: m.rows(x, torch.float32, (2, 3, 8), "x", 0),
                  lambda x: m.scratch(x, 0)):
            with pytest.raises((ValueError, RuntimeError)):
                f(kind)
    assert m.scratch(None, 0) == (0, 0)


def test_sizes_whose_indices_would_wrap(lb):
    assert lb.lowbit_lora_workspace_bytes(1, 1, (1 << 25) + 8, 64, 8) == 0   # more column ranges than a grid has
    assert lb.lowbit_lora_workspace_bytes(1, 1, 1 << 25, 64, 8) > 0
    L = lb.lib()
    for batch in (dict(max_pages=(1 << 25) + 1), dict(n_seqs=(1 << 30) + 1)):
        c, b = kv8(lb, batch=batch)
        assert L.lowbit_kv8_read(ctypes.byref(c), ctypes.byref(b), FAKE, FAKE, 0, None) == 3
        assert L.lowbit_kv8_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 4) == 0


def test_lora_group_outputs_are_apart(lb):
    def arr(*p):
        return ctypes.cast((ctypes.c_void_p * len(p))(*p), ctypes.c_void_p)

    g, ab = lb.lib().lowbit_lora_add_group, arr(0x10000, 0x10000)
    for base, y in ((arr(0x30000, 0x40000), arr(0x50000, 0x50000)),    # one output for two projections
                    (arr(0x30000, 0x50000), arr(0x50000, 0x60000))):   # an output that is another's base
        assert g(FAKE, FAKE, ab, ab, None, None, base, y, 2, 4, 64, 128, 16, 2, FAKE, BIG, None) == 1


REFUSED = [
    (dict(k=None), {}, 1), (dict(v=None), {}, 1), (dict(k_scales=None), {}, 1), (dict(v_scales=None), {}, 1),
    (dict(k=0x10008), {}, 2), (dict(v_scales=0x10004), {}, 2), (dict(n_pages=0), {}, 1), (dict(n_heads=0), {}, 1),
    (dict(page_tokens=48), {}, 3), (dict(page_tokens=256), {}, 3), (dict(head_dim=96), {}, 3), (dict(n_heads=1025), {}, 3),
    (dict(n_pages=1 << 30, n_heads=2), {}, 3), ({}, dict(kv_len=None), 1), ({}, dict(page_table=None), 1),
    ({}, dict(kv_len=0x10004), 2), ({}, dict(row_start=0x10004), 2), ({}, dict(n_seqs=-1), 1), ({}, dict(n_rows=-1), 1),
    ({}, dict(max_pages=0), 1), ({}, dict(max_pages=1 << 26), 3), ({}, dict(row_start=None), 1)]


@pytest.mark.parametrize("cache,batch,status", REFUSED)
def test_kv8_refusals(lb, cache, batch, status):
    c, b = kv8(lb, cache, batch)
    L, rc, rb = lb.lib(), ctypes.byref(c), ctypes.byref(b)
    assert L.lowbit_kv8_append(rc, rb, FAKE, 128, 0, FAKE, 128, 0, None) == status
    assert L.lowbit_kv8_read(rc, rb, FAKE, FAKE, 0, None) == status
    assert L.lowbit_kv8_attention(rc, rb, FAKE, 256, 4, 0.1, FAKE, 256, FAKE, BIG, None) == status
    assert L.lowbit_kv8_attention_workspace_bytes(rc, rb, 4) == 0


def test_kv8_operand_refusals(lb):
    c, b = kv8(lb)
    L, rc, rb = lb.lib(), ctypes.byref(c), ctypes.byref(b)
    a = L.lowbit_kv8_append
    assert a(None, rb, FAKE, 128, 0, FAKE, 128, 0, None) == 1
    assert a(rc, None, FAKE, 128, 0, FAKE, 128, 0, None) == 1
    assert a(rc, rb, None, 128, 0, FAKE, 128, 0, None) == 1
    assert a(rc, rb, FAKE, 120, 0, FAKE, 128, 0, None) == 1      # stride below a row
    assert a(rc, rb, FAKE, 132, 0, FAKE, 128, 0, None) == 2
    assert a(rc, rb, FAKE, 128, 2, FAKE, 128, 0, None) == 1      # unknown type
    assert a(rc, rb, FAKE, 128, 0, MIS, 128, 0, None) == 2
    assert a(rc, rb, FAKE, 1 << 40, 0, FAKE, 128, 0, None) == 3
    assert L.lowbit_kv8_read(rc, rb, MIS, None, 0, None) == 2
    assert L.lowbit_kv8_read(rc, rb, FAKE, None, 5, None) == 1
    assert L.lowbit_kv8_read(rc, rb, None, None, 0, None) == 0   # nothing asked for
    t = L.lowbit_kv8_attention
    need = L.lowbit_kv8_attention_workspace_bytes(rc, rb, 4)
    assert need > 0
    assert t(rc, rb, FAKE, 256, 4, 0.1, FAKE, 256, FAKE, need - 1, None) == 1
    assert t(rc, rb, FAKE, 256, 4, 0.1, FAKE, 256, None, need, None) == 1
    assert t(rc, rb, FAKE, 256, 4, 0.1, FAKE, 256, MIS, need, None) == 2
    assert t(rc, rb, FAKE, 256, 3, 0.1, FAKE, 256, FAKE, need, None) == 1     # heads not a multiple
    assert t(rc, rb, FAKE, 1 << 20, 260, 0.1, FAKE, 1 << 20, FAKE, need, None) == 3   # 130 heads a cache head
    assert t(rc, rb, FAKE, 256, 4, float("nan"), FAKE, 256, FAKE, need, None) == 1
    assert t(rc, rb, FAKE, 256, 4, float("inf"), FAKE, 256, FAKE, need, None) == 1
    assert t(rc, rb, FAKE, 248, 4, 0.1, FAKE, 256, FAKE, need, None) == 1
    assert t(rc, rb, FAKE, 256, 4, 0.1, FAKE, 260, FAKE, need, None) == 2
    assert t(rc, rb, None, 256, 4, 0.1, FAKE, 256, FAKE, need, None) == 1
    c, b = kv8(lb, batch=dict(n_rows=0))
    assert t(ctypes.byref(c), ctypes.byref(b), None, 256, 4, 0.1, None, 256, None, 0, None) == 0   # no rows: no-op
    c, b = kv8(lb, batch=dict(n_seqs=0, row_start=None, n_rows=0))
    assert a(ctypes.byref(c), ctypes.byref(b), None, 128, 0, None, 128, 0, None) == 0
