"""The decode-side operators (adapters, rotary positions, KV8 cache and its attention) from their definitions in
include/lowbit.h, in 64 bits with plain loops; nothing of the library is used."""
import numpy as np


def bf16_to_f64(t):
    return t.detach().cpu().float().numpy().astype(np.float64)


def lora(x, ids, a, b, base, ranks, scales):
    """y and sum |.| per element (x [M][K], a [L][r][K], b [L][N][r], base [M][N]; float64)."""
    y, ab = base.copy(), np.abs(base)
    for m, i in enumerate(ids):
        if 0 <= i < a.shape[0]:
            r = a.shape[1] if ranks is None else min(max(int(ranks[i]), 0), a.shape[1])
            s = 1.0 if scales is None else float(scales[i])
            y[m] += s * (b[i, :, :r] @ (a[i, :r] @ x[m]))
            ab[m] += abs(s) * (np.abs(b[i, :, :r]) @ (np.abs(a[i, :r]) @ np.abs(x[m])))
    return y, ab


def rope(x, positions, frequencies, interleaved, magnitude):
    """x [M][H][D] float64, frequencies [rot / 2] in radians per position."""
    y = x.copy()
    half = len(frequencies)
    for m, p in enumerate(positions):
        # the angle mod one turn in extended precision: positions reach 2^31
        turns = np.longdouble(int(p)) * (np.asarray(frequencies, np.longdouble) / (2 * np.longdouble(np.pi)))
        w = ((turns - np.floor(turns)) * 2 * np.longdouble(np.pi)).astype(np.float64)
        c, s = magnitude * np.cos(w), magnitude * np.sin(w)
        ia = np.arange(half) * 2 if interleaved else np.arange(half)
        ib = ia + 1 if interleaved else ia + half
        u, v = x[m][:, ia], x[m][:, ib]
        y[m][:, ia], y[m][:, ib] = u * c - v * s, v * c + u * s
    return y


def places(kv_len, page_table, row_start, n_rows, page_tokens, n_pages):
    """(row, sequence, position, page or -1, slot) of every row that has a place."""
    cap = page_table.shape[1] * page_tokens
    for b in range(len(kv_len)):
        length = min(max(int(kv_len[b]), 0), cap)
        lo, hi = (b, b + 1) if row_start is None else (int(row_start[b]), int(row_start[b + 1]))
        lo = min(max(lo, 0), n_rows)
        hi = min(max(hi, lo), n_rows)
        for r in range(lo, hi):
            pos = length - (hi - lo) + (r - lo)
            page = int(page_table[b, pos // page_tokens]) if pos >= 0 else -1
            yield r, b, pos, page if 0 <= page < n_pages else -1, pos % page_tokens


def append(codes, scales, x, kv_len, page_table, row_start):
    """codes int8 [pages][H][P][D] and scales fp32 [pages][H], updated copies; x [rows][H][D] float32 values."""
    codes, scales = codes.copy(), scales.copy()
    pages, H, P, D = codes.shape
    x = np.nan_to_num(x.astype(np.float32), nan=0.0, posinf=np.finfo(np.float32).max, neginf=np.finfo(np.float32).min)
    groups = {}
    for r, b, pos, page, slot in places(kv_len, page_table, row_start, len(x), P, pages):
        if pos >= 0 and page >= 0:
            groups.setdefault(page, []).append((slot, r))
    for page, new in groups.items():
        first = min(s for s, _ in new)
        for h in range(H):
            top = max(np.abs(x[r, h]).max() for _, r in new)
            fresh = np.float32(np.float64(top) / 127.0)
            was = np.float32(max(scales[page, h], 0.0)) if first else np.float32(0)
            now = max(was, fresh)
            if now > was:
                old = codes[page, h, :first].astype(np.float64) * np.float64(was) / np.float64(now)
                codes[page, h, :first] = np.rint(old).astype(np.int8)
            for slot, r in new:
                q = np.rint(x[r, h].astype(np.float64) / np.float64(now)) if now > 0 else np.zeros(D)
                codes[page, h, slot] = np.clip(q, -127, 127).astype(np.int8)
            scales[page, h] = now
    return codes, scales


def attention(k, ks, v, vs, q, scale, kv_len, page_table, row_start):
    """out, and a bound of what the kernel's fixed-point steps may add, per element (rows without a sequence: None)."""
    pages, H, P, D = k.shape
    T, Q, _ = q.shape
    G = Q // H
    out, tol = [None] * T, [None] * T
    for r, b, pos, _, _ in places(kv_len, page_table, row_start, T, P, pages):
        out[r], tol[r] = np.zeros((Q, D)), np.zeros((Q, D))
        n = pos + 1
        if n <= 0:
            continue
        ids = page_table[b, : -(-n // P)]
        ok = np.repeat((ids >= 0) & (ids < pages), P)[:n]
        ids = np.where((ids >= 0) & (ids < pages), ids, 0)
        if not ok.any():
            continue
        for h in range(H):
            kk = (k[ids, h].astype(np.float64) * ks[ids, h].astype(np.float64)[:, None, None]).reshape(-1, D)[:n][ok]
            vv = (v[ids, h].astype(np.float64) * vs[ids, h].astype(np.float64)[:, None, None]).reshape(-1, D)[:n][ok]
            for j in range(h * G, (h + 1) * G):
                s = scale * (kk @ q[r, j])
                p = np.exp(s - s.max())
                o = p @ vv / p.sum()
                out[r][j] = o
                # q's fixed point: half a step of qmax / 32512 per entry; fp32 rounding of s and exp2 (2^-21 of
                # |s|, 2^-20); probabilities: half a step of 1 / 65280 of a 32-token tile's largest, at most 32 of
                # them beside a sum of at least that largest; each in numerator and denominator; bf16 at the end
                ds = abs(scale) * np.abs(kk).sum(1).max() * np.abs(q[r, j]).max() / 65024 + np.abs(s).max() * 2.0 ** -21 + 2.0 ** -20
                tol[r][j] = 2.0 ** -8 * np.abs(o) + 2 * np.abs(vv).max() * (np.expm1(2 * ds) + 32 * 2.0 ** -17)
    return out, tol
