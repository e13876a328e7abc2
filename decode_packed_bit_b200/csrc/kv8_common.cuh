// kv8_common.cuh -- what the kernels of the KV8 cache share: the checked view
// of a batch's device arrays, and typed 8-value loads.
//
// Lengths, pages and rows live in device memory, so the host cannot check
// them.  Every kernel reads them through the helpers here, which clamp what is
// out of range and record it in a fault word, so that no value of theirs can
// lead an access out of a buffer.
#pragma once

#include "common.cuh"

namespace lowbit {

struct Kv8View {
    const int32_t *kv_len, *page_table, *row_start;
    int n_seqs, max_pages, n_rows;
    int n_pages, H, P, D;
    int P_log2, D_log2;  // P is 32, 64 or 128, D 64 or 128: shifts in place of divisions
};

inline Kv8View kv8_view(const lowbit_kv8_cache &c, const lowbit_kv8_batch &b)
{
    return Kv8View{b.kv_len, b.page_table, b.row_start, b.n_seqs, b.max_pages, b.n_rows,
                   c.n_pages, c.n_heads, c.page_tokens, c.head_dim,
                   c.page_tokens == 32 ? 5 : c.page_tokens == 64 ? 6 : 7, c.head_dim == 64 ? 6 : 7};
}

// Sequence b: rows [r0, r0 + n), of which the first is position len - n.
struct Kv8Seq {
    int r0, n, len;
};

// `fault` is set when something had to be clamped.
__device__ __forceinline__ Kv8Seq kv8_seq(const Kv8View &v, int b, unsigned *fault)
{
    Kv8Seq s;
    const int cap = v.max_pages * v.P, raw = __ldg(v.kv_len + b);
    s.len = min(max(raw, 0), cap);
    bool bad = s.len != raw;
    if (v.row_start) {
        const int lo = __ldg(v.row_start + b), hi = __ldg(v.row_start + b + 1);
        s.r0 = min(max(lo, 0), v.n_rows);
        const int e = min(max(hi, s.r0), v.n_rows);
        s.n = e - s.r0;
        bad |= s.r0 != lo || e != hi;
    } else {
        s.r0 = b;
        s.n = 1;
    }
    if (bad) atomicExch(fault, 1u);
    return s;
}

// The page of token block j of sequence b, or -1.
__device__ __forceinline__ int kv8_page(const Kv8View &v, int b, int j, unsigned *fault)
{
    const int p = __ldg(v.page_table + (int64_t)b * v.max_pages + j);
    if ((unsigned)p < (unsigned)v.n_pages) return p;
    atomicExch(fault, 1u);
    return -1;
}

// The last sequence whose first item lies at or before `item`, where sequence
// b's items begin at row_start[b] / T + per * b: an upper bound of its tiles
// of T rows that needs no pass over the batch.  -1 when there is none.
__device__ __forceinline__ int kv8_find_seq(const Kv8View &v, int item, int T, int per)
{
    int lo = -1, hi = v.n_seqs - 1;
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        const int64_t f = max(__ldg(v.row_start + mid), 0) / T + (int64_t)per * mid;
        if (f <= item)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// The same by a whole warp for one item: 32 sequences are looked at at once, so
// that up to 32 take one memory latency, up to 1024 two.
__device__ __forceinline__ int kv8_find_seq_warp(const Kv8View &v, int item, int T, int per)
{
    int lo = -1, hi = v.n_seqs - 1;
    const int lane = threadIdx.x & 31;
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32, mid = lo + (lane + 1) * step;
        bool at = false;
        if (mid <= hi) at = max(__ldg(v.row_start + mid), 0) / T + (int64_t)per * mid <= item;
        // they hold for the first lanes where row_start does not fall; else what
        // is found may begin after `item`, which the caller checks
        const int n = __popc(__ballot_sync(0xffffffffu, at));
        const int top = lo + n * step;
        hi = n < 32 ? min(hi, top + step - 1) : hi;
        lo = min(top, hi);
    }
    return lo;
}

}  // namespace lowbit
