"""What lowbit_kv8_attention may differ by from its definition, derived for each of its two kernels, per element.

With weights w_t in place of the probabilities p_t, in numerator and denominator alike, a row's output moves by
    sum_t (w_t - p_t) (v_t - o) / sum_t w_t,
because sum_t p_t (v_t - o) = 0; so with |w_t - p_t| <= c_t by at most
    (sum_t c_t |v_t| + |o| sum_t c_t) / (1 - sum_t c_t).
A factor that all weights share does nothing, so errors are counted from the token with the largest score.  The kernels'
own number for q (fixed point, f16) is a rounding that the header states; it is taken here as they take it, and
everything else is in 64 bits.

Few rows of a sequence (integer tensor cores):
  q       rint(q 32512 / qmax) steps of qmax / 32512, in fp32.
  scores  int32 sums, exact.  Within a 32-token tile the difference from its largest is taken in integers; the factor
          (qmax / 32512) |scale| log2(e) ks has 5 roundings of 2^-24, the product with the difference three: 2^-21 of
          |s_t - s_tile|.  A tile's largest score is rounded the same way, and so is the unit's maximum that it is
          subtracted from: 2^-21 of |s_tile| + |s_max| for the tiles other than the largest token's.  Exponentials:
          2^-20.
  p       half a step of 1 / 65280 of the tile's largest, 2^-16 / 1.99 of it.
Prompts (tcgen05):
  q       f16 after a power of two that brings qmax to [1, 2).
  scores  fp32 sums of D products; every one of D / 16 steps adds 16 products and the sum so far, each cut at 2^-23 of
          the largest term: 17 D / 16 cuts of 2^-23 sum |q k|, for the token and for the largest.  Products with the
          page's factor and the reference in fp32 as above: 2^-21 of |s_t - s_max| within the largest token's page,
          of |s_t| + |s_max| + |log vs| in others.  Exponentials: 2^-20.
  p       f16: 2^-11 of itself (half a step), or half of the smallest step 2^-24 where it is subnormal; the numerator
          holds it rounded, the denominator not.  p is exp2(x - m + 7) with x = s + log2(vs), vs = 2^-60 for a page
          of zeros, and m of at most the row's largest x: half of that step is at most 2^-32 of exp(x_max - x_t) p_t.
Both: fp32 sums over n tokens in tiles, 2^-24 (n / 32 + 64) sum_t p_t |v_t|; exponentials below 2^-126 are zero, n 2^-126 of
the largest value; the output 2^-8 of itself (bf16), or half of its smallest step, 2^-134."""
import numpy as np

LN2 = float(np.log(2.0))


def prompts(H, G, n_seqs, n_rows):
    """Whether a call of these sizes goes to the kernel for prompts."""
    return n_rows * G >= 64 * n_seqs and n_rows * G * H >= 8192


def fixed_point(q):
    """q [rows][D] float64 (bf16 values) as the integer kernel takes it."""
    x = q.astype(np.float32)
    top = np.abs(x).max(1, keepdims=True)
    some = top >= np.float32(2.0 ** -100)
    inv = np.where(some, np.float32(32512) / np.where(some, top, np.float32(1)), np.float32(0))
    return np.rint(x * inv).astype(np.float64) * top.astype(np.float64) / 32512


def as_f16(q):
    """q as the tcgen05 kernel takes it."""
    top = np.abs(q).max(1, keepdims=True)
    some = top >= 2.0 ** -100
    power = np.exp2(np.minimum(np.floor(np.log2(np.where(some, top, 1.0))), 126.0))
    return np.where(some, (q / power).astype(np.float16).astype(np.float64) * power, 0.0)


def check(cache, table, lens, q, scale, row_start, out, untouched=-7.0, vacuous=0.05, loose=0.0):
    """cache: (k, k_scales, v, v_scales) as numpy; q, out float64 [rows][heads][D].  The bound has to stay below `vacuous`
    of the largest value, so that it can fail, but for a share `loose` of the rows.  Returns the worst share of it."""
    k, ks, v, vs = cache
    pages, H, P, D = k.shape
    T, Q, _ = q.shape
    G, B = Q // H, len(lens)
    tc = prompts(H, G, B, T)
    seen = np.zeros(T, bool)
    worst, n_rows, n_loose = 0.0, 0, 0
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * P)
        lo, hi = (b, b + 1) if row_start is None else (int(row_start[b]), int(row_start[b + 1]))
        lo = min(max(lo, 0), T)
        hi = min(max(hi, lo), T)
        seen[lo:hi] = True
        pos = n - (hi - lo) + np.arange(hi - lo)
        if hi == lo:
            continue
        ids = table[b, : -(-n // P)].astype(np.int64)
        there = np.repeat((ids >= 0) & (ids < pages), P)[:n]
        ids = np.where((ids >= 0) & (ids < pages), ids, 0)
        visible = there[None, :] & (np.arange(n)[None, :] <= pos[:, None])  # [rows][n]
        for h in range(H):
            got = out[lo:hi, h * G:(h + 1) * G].reshape(-1, D)
            vis = np.repeat(visible, G, 0)
            some = vis.any(1) if n else np.zeros(len(vis), bool)
            assert (got[~some] == 0).all(), f"sequence {b}: rows that see nothing are not zero"
            rows = q[lo:hi, h * G:(h + 1) * G].reshape(-1, D)
            finite = np.isfinite(rows).all(1)
            assert np.isnan(got[some & ~finite]).all(), f"sequence {b}: rows of q that are not finite"
            take = some & finite
            if not take.any():
                continue
            rows, got, vis = rows[take], got[take], vis[take]
            ksn, vsn = np.repeat(ks[ids, h].astype(np.float64), P)[:n], np.repeat(vs[ids, h].astype(np.float64), P)[:n]
            kk = k[ids, h].reshape(-1, D)[:n].astype(np.float64) * ksn[:, None]
            vv = v[ids, h].reshape(-1, D)[:n].astype(np.float64) * vsn[:, None]
            kk[~there], vv[~there] = 0.0, 0.0
            qx = as_f16(rows) if tc else fixed_point(rows)
            s = np.where(vis, scale * (qx @ kk.T), -np.inf)
            top = s.max(1, keepdims=True)
            at = s.argmax(1)[:, None]
            total = np.exp(s - top).sum(1, keepdims=True)
            p = np.exp(s - top) / total
            o = p @ vv
            fin = np.where(vis, s, top)
            token = np.arange(n)[None]
            if tc:
                size = abs(scale) * (np.abs(qx) @ np.abs(kk).T)
                lv = np.abs(np.log(np.where(vsn > 2.0 ** -100, vsn, 2.0 ** -60)))[None]
                e = np.where(token // P == at // P, np.abs(fin - top), np.abs(fin) + np.abs(top) + lv + lv.max())
                e = 2.0 ** -21 * e + 17 * D / 16 * 2.0 ** -23 * (size + np.take_along_axis(size, at, 1)) + 2.0 ** -20
                e = np.where(token == at, 0.0, e)
                # in units of x = s + ln vs, whose maximum the reference follows; a page of zeros stands with 2^-60 there,
                # and has nothing to lose itself
                x = np.where(vis, s + np.log(np.where(vsn > 2.0 ** -100, vsn, 2.0 ** -60))[None], -np.inf)
                xm = x.max(1, keepdims=True)
                lost = np.where(vis & (vsn > 2.0 ** -100)[None], xm - np.where(vis, x, xm), -np.inf)
                d = np.where(vis, np.exp(np.minimum(lost + fin - top, 700.0)) / total * 2.0 ** -32, 0.0) + p * 2.0 ** -11
            else:
                tiles = -(-n // 32)
                pad = np.full((len(s), tiles * 32), -np.inf)
                pad[:, :n] = s
                st = np.repeat(pad.reshape(len(s), tiles, 32).max(2), 32, 1)[:, :n]
                sf = np.where(np.isfinite(st), st, top)
                e = 2.0 ** -21 * (np.abs(fin - sf) + np.where(token // 32 == at // 32, 0.0, np.abs(sf) + np.abs(top))) + 2.0 ** -20
                d = np.where(vis, np.exp(st - top) / total * 2.0 ** -16 / 1.99, 0.0)
            c = np.where(vis, np.where(e < 1, p * np.expm1(np.minimum(e, 1.0)), np.exp(np.minimum(fin - top + e, 700.0)) / total), 0.0) + d
            moved = c.sum(1, keepdims=True)
            ok = moved < 0.5
            most = np.abs(vv).max()
            tol = (c @ np.abs(vv) + np.abs(o) * moved) / np.where(ok, 1 - moved, 1.0)
            tol = tol + 2.0 ** -24 * (n / 32 + 64) * (p @ np.abs(vv))
            tol = (tol + n * 2.0 ** -126 * most) * 1.01 + 2.0 ** -8 * np.abs(o) * 1.01 + 2.0 ** -134
            says = (ok & (tol <= vacuous * most + 1e-40)).all(1)
            n_rows, n_loose = n_rows + len(says), n_loose + int((~says).sum())
            diff = np.where(ok, np.abs(got - o), 0.0)
            assert np.isfinite(got).all(), f"sequence {b} head {h}: not finite"
            worst = max(worst, float((diff / tol).max()))
            assert (diff <= tol).all(), (f"sequence {b} head {h}: {(diff > tol).sum()} of {diff.size} off in {(diff > tol).any(1).sum()} rows, "
                                         f"worst {(diff / tol).max():.2f} times the bound, {(diff - tol).max():.3e} above it")
    assert (out[~seen] == untouched).all(), "rows behind the last sequence were written"
    assert n_loose <= loose * n_rows, f"the bound says nothing of {n_loose} rows of {n_rows}"
    return worst
