"""The oracle of the attention bounds itself, on the CPU: an output rounded as the kernels may round it passes, one with a
small mistake planted does not."""
import numpy as np
import pytest

import attention_bounds as ab


def bf16(x):
    u = x.astype(np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def make(H, G, D, P, n, rows, scale, number):
    g = np.random.default_rng(n)
    pages = -(-n // P)
    k, v = (g.integers(-127, 128, (pages, H, P, D)).astype(np.int8) for _ in range(2))
    ks, vs = (g.uniform(0.005, 0.025, (pages, H)).astype(np.float32) for _ in range(2))
    table = np.arange(pages, dtype=np.int32)[None]
    q = bf16(g.standard_normal((rows, H * G, D)))
    out = np.zeros_like(q)
    for h in range(H):
        kk = (k[:, h].astype(np.float64) * ks[:, h].astype(np.float64)[:, None, None]).reshape(-1, D)[:n]
        vv = (v[:, h].astype(np.float64) * vs[:, h].astype(np.float64)[:, None, None]).reshape(-1, D)[:n]
        for r in range(rows):
            seen = n - rows + r + 1
            s = scale * number(q[r, h * G:(h + 1) * G]) @ kk[:seen].T
            p = np.exp(s - s.max(1, keepdims=True))
            out[r, h * G:(h + 1) * G] = p / p.sum(1, keepdims=True) @ vv[:seen]
    return (k, ks, v, vs), table, q, bf16(out)


@pytest.mark.parametrize("H,G,D,P,n,rows,number", [(1, 4, 64, 32, 300, 3, ab.fixed_point), (2, 64, 64, 64, 130, 64, ab.as_f16)])
@pytest.mark.parametrize("scale", [0.1, 300.0])
def test_bound_holds_and_notices(H, G, D, P, n, rows, number, scale):
    cache, table, q, out = make(H, G, D, P, n, rows, scale, number)
    assert ab.prompts(H, G, 1, rows) == (number is ab.as_f16)
    rs = np.array([0, rows], np.int32)
    loose = 0.0 if scale < 1 else 0.02
    assert ab.check(cache, table, [n], q, scale, rs, out, loose=loose) <= 1.0
    for r, j, d, by in ((0, 0, 5, 0.05), (rows - 1, G - 1, D - 1, -0.05)):
        wrong = out.copy()
        wrong[r, j, d] += by * 127 * 0.025
        with pytest.raises(AssertionError, match="off"):
            ab.check(cache, table, [n], q, scale, rs, wrong, loose=loose)
    if scale < 1:  # one token fewer than there are (a large scale leaves a single one that counts)
        with pytest.raises(AssertionError):
            ab.check(cache, table, [n - 1], q, scale, rs, out, loose=loose)
    wrong = out.copy()
    wrong[0] = np.nan
    with pytest.raises(AssertionError):
        ab.check(cache, table, [n], q, scale, rs, wrong, loose=loose)
