// kv8_attn.cu -- attention of a few rows per sequence over the KV8 cache
// (int8 codes in pages, one fp32 scale per page and head).
//
// out[r] = sum_t softmax_t(scale q[r] . k[t]) v[t] over the tokens t a row
// sees, in one pass over the cache with a running maximum and sum per row.
// Both products run on the integer tensor cores with the codes as they lie in
// memory (mma.sync m16n8k32):
//   - a row of q becomes 16-bit fixed point of its own largest value, split
//     into two int8 limbs; limbs and row share one MMA (rows 0-7 the high, 8-15
//     the low limb), so a thread holds both sums of a row and joins them with a
//     shift.  The rounding is at most 2^-16 of the row's largest value, against
//     2^-9 of each value in q's own bf16.
//   - a tile's probabilities, relative to the tile's own maximum, become 16-bit
//     fixed point the same way (two uint8 limbs, at most 2^-17 of the tile's
//     largest off), and meet v's codes; the exact int32 sum of a tile is
//     scaled by v's page scale and the running maximum in fp32.
// Nothing is converted per cached value but the byte transposition of v (4
// tokens x 4 entries, 8 PRMT per 16 bytes).
//
// Layout of the work.  A unit is (sequence, cache head, RT * 8 query rows); its
// tokens come in tiles of 32.  All tiles of all units, in order, are cut into
// equal ranges, one per CTA (one CTA per SM); lengths are read on the device,
// so a captured graph follows them.  The warps of a CTA take a range's tiles in
// turn, each with its own cp.async ring of key and value halves of tiles, which
// runs on across the ends of units, and join their partial sums through shared
// memory at the end of a unit; a unit cut between CTAs is joined in
// CTA order by the last of them to arrive (a counter in the workspace, left
// zeroed), so the result does not depend on timing.
#include <algorithm>
#include <cfloat>

#include "kv8_common.cuh"

namespace lowbit {

__device__ unsigned g_at_fault;  // a length, page or row was out of range

int kv8_attn_fault_flag()
{
    unsigned v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_at_fault, sizeof(v)) != cudaSuccess) return -1;
    cudaMemcpyToSymbol(g_at_fault, &zero, sizeof(zero));
    return (int)v;
}

constexpr int kAtWarps = 12;  // 168 registers a thread; with 8 warps the chains of a tile's steps showed
constexpr int kAtThreads = kAtWarps * 32;
constexpr int kAtTile = 32;  // tokens
constexpr int kAtMaxRT = 2;

struct Kv8Attn {
    Kv8View v;
    const int8_t *k, *vv;
    const float *ks, *vs;
    const uint16_t *q;
    uint16_t *out;
    int64_t q_stride, out_stride;
    int G;            // query heads per cache head
    int page_log2;
    float scale_log2; // scale * log2(e)
    unsigned *counters;   // [CTAs], zero between calls
    float *part_ml;       // [2 CTAs][rows][2]
    float *part_o;        // [2 CTAs][rows][D]
};

template <int D, int RT>
struct AttnShape {
    static constexpr int kHalf = kAtTile * D;        // bytes of a tile's keys, or of its values
    static constexpr int kRows = RT * 8;
    static constexpr int kMergeBytes = kAtWarps * 8 * D * 4;  // eight rows at a time
    static constexpr int kFixed = kMergeBytes + 2 * 2 * kAtWarps * kRows * 4 + RT * D * 16 + 2 * kRows * 4;
    static constexpr int kHalves = std::min(6, (int)((226 * 1024 - kFixed) / (kAtWarps * (kHalf + 4))));
    static constexpr int kRing = kAtWarps * kHalves * kHalf;
    static constexpr int kQ = kRing;                                       // q fragments, [RT][D / 32][32] x 16 bytes
    static constexpr int kMerge = kQ + RT * D * 16;
    static constexpr int kStats = kMerge + kMergeBytes;                    // [2][m, l][warp][rows] fp32
    static constexpr int kRowInfo = kStats + 2 * 2 * kAtWarps * kRows * 4; // [rows] factor, [rows] limit
    static constexpr int kScales = kRowInfo + 2 * kRows * 4;               // [warp][half] fp32
    static constexpr int kBytes = kScales + kAtWarps * kHalves * 4;
    static_assert(kHalves >= 3 && kBytes <= 226 * 1024 + 512, "attention ring does not fit");
};

__device__ __forceinline__ void at_cp16(unsigned dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void at_cp4(unsigned dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void at_mma_ss(int (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void at_mma_us(int (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 at_lds16(unsigned a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 at_lds8(unsigned a)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ float at_exp2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// x, but 0 for -inf: a reference that -inf may be subtracted from
__device__ __forceinline__ float at_ref(float m) { return m == -INFINITY ? 0.f : m; }

// Where a range of work stands: segment [ta, tb) of the tiles of unit u of
// sequence b.  Tiles from `seen` on are visible to no row of the unit.
struct AttnWalk {
    int64_t left;  // tiles of the range from this segment's start on
    int b, u, units, tiles, ta, tb, seen, h;
    Kv8Seq s;
    int rts;  // row tiles of the sequence
};

__device__ __forceinline__ int at_tiles(int len) { return max(1, (len + kAtTile - 1) / kAtTile); }

template <int RT>
__device__ __forceinline__ void at_sequence(AttnWalk &w, const Kv8Attn &a, int b)
{
    w.b = b;
    w.s = kv8_seq(a.v, b, &g_at_fault);
    w.rts = (int)(((int64_t)w.s.n * a.G + RT * 8 - 1) / (RT * 8));
    w.units = w.rts * a.v.H;
    w.tiles = at_tiles(w.s.len);
}

template <int RT>
__device__ __forceinline__ void at_segment(AttnWalk &w, const Kv8Attn &a)
{
    w.tb = (int)min((int64_t)w.tiles, w.ta + w.left);
    w.h = w.u / w.rts;
    // what the unit's last row sees
    const int last = min(w.s.n - 1, ((w.u - w.h * w.rts + 1) * RT * 8 - 1) / a.G);
    const int vis = min(max(w.s.len - w.s.n + last + 1, 0), w.s.len);
    w.seen = (vis + kAtTile - 1) / kAtTile;
}

// On to the next segment; false at the end of the range.
template <int RT>
__device__ __forceinline__ bool at_next(AttnWalk &w, const Kv8Attn &a)
{
    w.left -= w.tb - w.ta;
    if (w.left <= 0) return false;
    if (w.tb == w.tiles) {
        w.ta = 0;
        if (++w.u == w.units) {
            w.u = 0;
            do {
                if (w.b + 1 >= a.v.n_seqs) return false;
                at_sequence<RT>(w, a, w.b + 1);
            } while (w.units == 0);
        }
    } else {
        w.ta = w.tb;
    }
    at_segment<RT>(w, a);
    return true;
}

template <int D, int RT>
__global__ void __launch_bounds__(kAtThreads, 1) k_kv8_attn(const Kv8Attn a)
{
    using S = AttnShape<D, RT>;
    constexpr int ROWS = RT * 8, NJ = D / 8, NH = S::kHalves, KS = D / 32;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t sh_sum[kAtWarps], sh_units[kAtWarps];
    __shared__ int64_t sh_off;
    __shared__ int sh_b, sh_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    pdl_launch_dependents();
    pdl_wait_primary();

    // ---- this CTA's range of the batch's tiles ----
    const int per = (a.v.n_seqs + kAtThreads - 1) / kAtThreads;
    const int s0 = min(tid * per, a.v.n_seqs), s1 = min(s0 + per, a.v.n_seqs);
    auto seq_work = [&](int b, int64_t &units) -> int64_t {
        AttnWalk w;
        at_sequence<RT>(w, a, b);
        units += w.units;
        return (int64_t)w.units * w.tiles;
    };
    int64_t mine = 0, units = 0;
    for (int b = s0; b < s1; ++b) mine += seq_work(b, units);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
        units += __shfl_xor_sync(0xffffffffu, units, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) {
        sh_sum[warp] = incl;
        sh_units[warp] = units;
    }
    __syncthreads();
    int64_t total = 0, before = 0;
    units = 0;
#pragma unroll
    for (int w = 0; w < kAtWarps; ++w) {
        if (w < warp) before += sh_sum[w];
        total += sh_sum[w];
        units += sh_units[w];
    }
    if (total == 0) return;
    // CTAs: one per unit where units are short (no joining between CTAs), else
    // enough that a range has three tiles for each warp
    const int64_t C = min(min((int64_t)gridDim.x, total), max(units, (total + 3 * kAtWarps - 1) / (3 * kAtWarps)));
    if (blockIdx.x >= C) return;
    const int64_t w0 = blockIdx.x * total / C, w1 = (blockIdx.x + 1) * total / C;
    {
        const int64_t excl = before + incl - mine;
        if (w0 >= excl && w0 < excl + mine) {
            int64_t off = w0 - excl, u = 0;
            int b = s0;
            for (int64_t x; off >= (x = seq_work(b, u)); ++b) off -= x;
            sh_b = b;
            sh_off = off;
        }
    }
    __syncthreads();
    AttnWalk cw;
    cw.left = w1 - w0;
    at_sequence<RT>(cw, a, sh_b);
    cw.u = (int)(sh_off / cw.tiles);
    cw.ta = (int)(sh_off % cw.tiles);
    at_segment<RT>(cw, a);
    int64_t wpos = w0;  // of cw's segment

    // ---- this warp's ring ----
    const unsigned smem0 = (unsigned)__cvta_generic_to_shared(smem);
    const unsigned ring = smem0 + warp * NH * S::kHalf, scal = smem0 + S::kScales + warp * NH * 4;
    // 16-byte slots of 128-byte lines, permuted so that the fragment loads below
    // meet eight different ones; lane l copies pieces l, l + 32, ...
    constexpr int CH = D / 16;
    const int prow = lane / CH, pch = lane % CH;
    const unsigned kdst = D == 128 ? prow * 128 + ((pch ^ (4 * (prow & 1))) << 4) : (prow >> 1) * 128 + (((prow & 1) * 4 + pch) << 4);
    const unsigned vdst = D == 128 ? prow * 128 + (pch << 4) : (prow >> 1) * 128 + (((prow & 1) * 4 + pch) << 4);
    AttnWalk ld = cw;
    int ld_tile = ld.ta + warp, ld_slot = 0;
    bool ld_more = true, ld_value = false;
    int64_t ld_at = 0;   // byte offset of the tile, this lane's first piece
    int64_t ld_ph = -1;  // its page and head, -1 for an absent page
    unsigned present = 0;  // one bit per slot: keys that are there
    // Copies the next half of a tile (nothing at the end of the range).
    auto issue = [&]() {
        if (!ld_value) {
            while (ld_more && ld_tile >= min(ld.tb, ld.seen)) {
                ld_more = at_next<RT>(ld, a);
                ld_tile = ld.ta + warp;
            }
            ld_ph = -1;
            if (ld_more) {
                const int tok = ld_tile * kAtTile;
                const int page = kv8_page(a.v, ld.b, tok >> a.page_log2, &g_at_fault);
                if (page >= 0) {
                    ld_ph = (int64_t)page * a.v.H + ld.h;
                    ld_at = ((ld_ph << a.page_log2) + (tok & (a.v.P - 1))) * D + lane * 16;
                }
                ld_tile += kAtWarps;
            }
            present = ld_ph >= 0 ? present | (1u << ld_slot) : present & ~(1u << ld_slot);
        }
        if (ld_ph >= 0) {
            const int8_t *src = (ld_value ? a.vv : a.k) + ld_at;
            const unsigned st = ring + ld_slot * S::kHalf;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                // rows advance by 32 / CH: 4 (D = 128) or 8 (two lines by two)
                if (ld_value) {
                    const unsigned x = D == 128 ? (unsigned)(2 * (i & 3)) << 4 : (unsigned)(2 * ((2 * i + (prow >> 2)) & 3)) << 4;
                    at_cp16(st + i * 512 + (vdst ^ x), src + i * 512);
                } else {
                    at_cp16(st + i * 512 + kdst, src + i * 512);
                }
            }
            if (lane == 0) at_cp4(scal + ld_slot * 4, (ld_value ? a.vs : a.ks) + ld_ph);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        ld_value = !ld_value;
        ld_slot = ld_slot + 1 == NH ? 0 : ld_slot + 1;
    };
#pragma unroll 1
    for (int i = 0; i < NH - 1; ++i) issue();
    int slot = 0;

    // ---- q of a unit's rows as two int8 limbs, in fragment order ----
    // Thread x < ROWS D / 8 takes 8 entries of row x / (D / 8); a segment's q is
    // loaded while the segment before it is worked on.
    constexpr int QT = D / 8;  // threads per row
    const int qrow = tid / QT, qpart = tid % QT;
    uint4 qraw = make_uint4(0, 0, 0, 0);
    auto load_q = [&](const AttnWalk &w) {
        qraw = make_uint4(0, 0, 0, 0);
        const int r = w.u % w.rts * ROWS + qrow, i = r / a.G;
        if (qrow < ROWS && i < w.s.n)
            qraw = __ldg(reinterpret_cast<const uint4 *>(a.q + (int64_t)(w.s.r0 + i) * a.q_stride +
                                                         (int64_t)(w.h * a.G + r % a.G) * D + qpart * 8));
    };
    float *row_f = reinterpret_cast<float *>(smem + S::kRowInfo);
    int *row_lim = reinterpret_cast<int *>(row_f + ROWS);
    auto store_q = [&](const AttnWalk &w) {
        if (tid >= ROWS * QT) return;
        const int r = w.u % w.rts * ROWS + qrow, i = r / a.G;
        // rows past the sequence's see what is there, as zeros
        const int lim = i < w.s.n ? min(max(w.s.len - w.s.n + i + 1, 0), w.s.len) : w.s.len;
        const uint32_t raw[4] = {qraw.x, qraw.y, qraw.z, qraw.w};
        float f[8];
        float top = 0.f;
        bool bad = false;
#pragma unroll
        for (int y = 0; y < 8; ++y) {
            f[y] = __uint_as_float(y & 1 ? raw[y / 2] & 0xFFFF0000u : raw[y / 2] << 16);
            top = fmaxf(top, fabsf(f[y]));
            bad |= !(fabsf(f[y]) <= FLT_MAX);
        }
        const unsigned group = QT == 16 ? 0xFFFFu << (lane & 16) : 0xFFu << (lane & 24);
#pragma unroll
        for (int o = 1; o < QT; o <<= 1) top = fmaxf(top, __shfl_xor_sync(group, top, o));
        bad = (__ballot_sync(group, bad) & group) != 0;
        const float inv = top >= 0x1p-100f && !bad ? 32512.f / top : 0.f;
        uint32_t limb[4] = {0, 0, 0, 0};  // hi and lo of entries 0-3, of 4-7
#pragma unroll
        for (int y = 0; y < 8; ++y) {
            const int v = __float2int_rn(f[y] * inv), vh = (v + 128) >> 8;
            limb[y / 4 * 2] |= (uint32_t)(vh & 0xFF) << (8 * (y & 3));
            limb[y / 4 * 2 + 1] |= (uint32_t)((v - vh * 256) & 0xFF) << (8 * (y & 3));
        }
        // entries 8 qpart ..: 16-byte chunk qpart / 2 of a key, which lane t =
        // chunk % 4 of fragments 2 (chunk / 4) and the next one holds
        const int ch = qpart >> 1, frag = 2 * (ch >> 2) + (qpart & 1);
        reinterpret_cast<uint4 *>(smem + S::kQ)[((qrow >> 3) * KS + frag) * 32 + (qrow & 7) * 4 + (ch & 3)] =
            make_uint4(limb[0], limb[1], limb[2], limb[3]);
        if (qpart == 0) {
            row_f[qrow] = bad && lim > 0 ? NAN : top * (1.f / 32512.f) * a.scale_log2;
            row_lim[qrow] = lim;
        }
    };
    load_q(cw);
    store_q(cw);
    __syncthreads();

    float *merge = reinterpret_cast<float *>(smem + S::kMerge);
    int parity = 0;

    while (true) {
        AttnWalk nw = cw;
        const bool more = at_next<RT>(nw, a);
        if (more) load_q(nw);
        const int h = cw.h, row0 = cw.u % cw.rts * ROWS;
        float rowf[RT];
        int lim[RT], lim_min = INT_MAX;
#pragma unroll
        for (int m = 0; m < RT; ++m) {
            rowf[m] = row_f[m * 8 + g];
            lim[m] = row_lim[m * 8 + g];
            lim_min = min(lim_min, lim[m]);
        }
        lim_min = __reduce_min_sync(0xffffffffu, lim_min);

        float o[RT][NJ][2], mx[RT], l[RT];
#pragma unroll
        for (int m = 0; m < RT; ++m) {
            mx[m] = -INFINITY;
            l[m] = 0.f;
#pragma unroll
            for (int j = 0; j < NJ; ++j) o[m][j][0] = o[m][j][1] = 0.f;
        }

        for (int tile = cw.ta + warp; tile < min(cw.tb, cw.seen); tile += kAtWarps) {
            asm volatile("cp.async.wait_group %0;" ::"n"(NH - 2) : "memory");
            __syncwarp();
            const bool there = (present >> slot) & 1;
            issue();  // into the slot read last, while this one is worked on
            uint32_t pf[RT][4];
            float fac[RT], al[RT];
            bool same = true;
            if (there) {
                const unsigned st = ring + slot * S::kHalf;
                float ks;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(ks) : "r"(scal + slot * 4));
                // scores: column n of block j is token 16 (j / 2) + 4 (n / 2) +
                // 2 (j % 2) + n % 2, so that a thread's scores are those of the
                // tokens its probability fragment holds
                int acc[RT][4][4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int m = 0; m < RT; ++m)
#pragma unroll
                        for (int x = 0; x < 4; ++x) acc[m][j][x] = 0;
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    uint32_t qf[RT][2][4];
#pragma unroll
                    for (int m = 0; m < RT; ++m)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint4 u = at_lds16(smem0 + S::kQ + ((m * KS + 2 * c + y) * 32 + lane) * 16);
                            qf[m][y][0] = u.x; qf[m][y][1] = u.y; qf[m][y][2] = u.z; qf[m][y][3] = u.w;
                        }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int tr = 16 * (j >> 1) + 4 * (g >> 1) + 2 * (j & 1) + (g & 1);
                        const int sl = D == 128 ? ((t + 4 * c) ^ (4 * (g & 1))) : (g & 1) * 4 + t;
                        const uint4 x = at_lds16(st + (D == 128 ? tr : tr >> 1) * 128 + (sl << 4));
#pragma unroll
                        for (int m = 0; m < RT; ++m) {
                            at_mma_ss(acc[m][j], qf[m][0], x.x, x.y);
                            at_mma_ss(acc[m][j], qf[m][1], x.z, x.w);
                        }
                    }
                }
                const bool masked = (tile + 1) * kAtTile > lim_min;
#pragma unroll
                for (int m = 0; m < RT; ++m) {
                    const float f = rowf[m] * ks;
                    float s[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) {  // token 16 (x / 4) + 4 t + x % 4
                        const int j = 2 * (x >> 2) + ((x >> 1) & 1), e = x & 1;
                        s[x] = (float)(acc[m][j][e] * 256 + acc[m][j][2 + e]) * f;
                    }
                    if (masked) {
                        const int tok = tile * kAtTile + 4 * t;
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            if (tok + 16 * (x >> 2) + (x & 3) >= lim[m]) s[x] = -INFINITY;
                    }
                    float tm = s[0];
#pragma unroll
                    for (int x = 1; x < 8; ++x) tm = fmaxf(tm, s[x]);
                    tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 1));
                    tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 2));
                    const float ref = at_ref(tm);
                    uint32_t v[8], sum = 0;
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        v[x] = __float2uint_rn(at_exp2(s[x] - ref) * 65280.f);
                        sum += v[x];
                    }
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const uint32_t a01 = __byte_perm(v[4 * hh], v[4 * hh + 1], 0x5410),
                                       a23 = __byte_perm(v[4 * hh + 2], v[4 * hh + 3], 0x5410);
                        pf[m][2 * hh] = __byte_perm(a01, a23, 0x7531);
                        pf[m][2 * hh + 1] = __byte_perm(a01, a23, 0x6420);
                    }
                    const float mn = fmaxf(mx[m], tm), rn = at_ref(mn);
                    al[m] = at_exp2(mx[m] - rn);
                    // 0 * rowf: a NaN row stays one where masked tokens hide it
                    fac[m] = at_exp2(tm - rn) * (1.f / 65280.f) + 0.f * rowf[m];
                    l[m] = l[m] * al[m] + (float)sum * fac[m];
                    same = same && mx[m] == mn;
                    mx[m] = mn;
                }
            }
            // rows whose maximum stands keep their sums as they are
            if (!__all_sync(0xffffffffu, same)) {
#pragma unroll
                for (int m = 0; m < RT; ++m)
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        o[m][j][0] *= al[m];
                        o[m][j][1] *= al[m];
                    }
            }
            slot = slot + 1 == NH ? 0 : slot + 1;
            asm volatile("cp.async.wait_group %0;" ::"n"(NH - 2) : "memory");
            __syncwarp();
            issue();
            if (there) {
                const unsigned vb = ring + slot * S::kHalf;
                float vs;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(vs) : "r"(scal + slot * 4));
#pragma unroll
                for (int m = 0; m < RT; ++m) fac[m] *= vs;
                // products with v: column n of block j is entry (D / 8) n + j
                constexpr int VW = D / 32;  // words of a token's entries per thread
                uint32_t x[2][4][VW];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = 16 * hh + 4 * t + i;
                        if constexpr (D == 128) {
                            const uint4 u = at_lds16(vb + row * 128 + ((g ^ (2 * t)) << 4));
                            x[hh][i][0] = u.x; x[hh][i][1] = u.y; x[hh][i][2] = u.z; x[hh][i][3] = u.w;
                        } else {
                            const int sl = (row & 1) * 4 + (g >> 1);
                            const uint2 u = at_lds8(vb + (row >> 1) * 128 + ((sl ^ (2 * t)) << 4) + (g & 1) * 8);
                            x[hh][i][0] = u.x; x[hh][i][1] = u.y;
                        }
                    }
#pragma unroll
                for (int w = 0; w < VW; ++w) {
                    uint32_t b[2][4];
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const uint32_t t0 = __byte_perm(x[hh][0][w], x[hh][1][w], 0x5140),
                                       t1 = __byte_perm(x[hh][2][w], x[hh][3][w], 0x5140),
                                       t2 = __byte_perm(x[hh][0][w], x[hh][1][w], 0x7362),
                                       t3 = __byte_perm(x[hh][2][w], x[hh][3][w], 0x7362);
                        b[hh][0] = __byte_perm(t0, t1, 0x5410);
                        b[hh][1] = __byte_perm(t0, t1, 0x7632);
                        b[hh][2] = __byte_perm(t2, t3, 0x5410);
                        b[hh][3] = __byte_perm(t2, t3, 0x7632);
                    }
#pragma unroll
                    for (int y = 0; y < 4; ++y)
#pragma unroll
                        for (int m = 0; m < RT; ++m) {
                            int c[4] = {0, 0, 0, 0};
                            at_mma_us(c, pf[m], b[0][y], b[1][y]);
                            o[m][4 * w + y][0] = fmaf((float)(c[0] * 256 + c[2]), fac[m], o[m][4 * w + y][0]);
                            o[m][4 * w + y][1] = fmaf((float)(c[1] * 256 + c[3]), fac[m], o[m][4 * w + y][1]);
                        }
                }
            }
            slot = slot + 1 == NH ? 0 : slot + 1;
        }

        // ---- join the warps' sums ----
        // (statistics alternate between two places: the next segment's may be
        // written while this one's are still read)
        float *stat_m = reinterpret_cast<float *>(smem + S::kStats) + parity * 2 * kAtWarps * ROWS;
        float *stat_l = stat_m + kAtWarps * ROWS;
        parity ^= 1;
#pragma unroll
        for (int m = 0; m < RT; ++m) {
            l[m] += __shfl_xor_sync(0xffffffffu, l[m], 1);
            l[m] += __shfl_xor_sync(0xffffffffu, l[m], 2);
            if (t == 0) {
                stat_m[warp * ROWS + m * 8 + g] = mx[m];
                stat_l[warp * ROWS + m * 8 + g] = l[m];
            }
        }
        __syncthreads();
        const bool whole = cw.ta == 0 && cw.tb == cw.tiles;
        const int part = 2 * blockIdx.x + (cw.ta == 0 ? 1 : 0);
#pragma unroll
        for (int m = 0; m < RT; ++m) {
            if (m > 0) __syncthreads();  // the sums of the rows before are read
            {
                const int row = m * 8 + g;
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < kAtWarps; ++w) top = fmaxf(top, stat_m[w * ROWS + row]);
                const float f = at_exp2(mx[m] - at_ref(top));
                float4 *dst = reinterpret_cast<float4 *>(merge + (warp * 8 + g) * D + t * (D / 4));
                const int sw = D == 128 ? (g & 1) * 4 + t : (g & 1) * 2 + (t >> 1);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    // entries 4 i .. 4 i + 3 of the thread's D / 4 consecutive ones
                    const int e = i / (D / 32), j = 4 * (i % (D / 32));
                    dst[i ^ sw] = make_float4(o[m][j][e] * f, o[m][j + 1][e] * f, o[m][j + 2][e] * f, o[m][j + 3][e] * f);
                }
            }
            if (m == 0 && more) store_q(nw);  // every warp is done with this segment's
            __syncthreads();
            if (tid < 8 * D / 4) {
                const int r8 = tid / (D / 4), row = m * 8 + r8, d4 = tid % (D / 4), tt = d4 / (D / 16), x = d4 % (D / 16);
                const int sw = D == 128 ? (r8 & 1) * 4 + tt : (r8 & 1) * 2 + (tt >> 1);
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < kAtWarps; ++w) top = fmaxf(top, stat_m[w * ROWS + row]);
                float sum = 0.f;
                float4 acc4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kAtWarps; ++w) {
                    sum += stat_l[w * ROWS + row] * at_exp2(stat_m[w * ROWS + row] - at_ref(top));
                    const float4 v = reinterpret_cast<const float4 *>(merge + (w * 8 + r8) * D + tt * (D / 4))[x ^ sw];
                    acc4.x += v.x; acc4.y += v.y; acc4.z += v.z; acc4.w += v.w;
                }
                if (whole) {
                    const int r = row0 + row, ri = r / a.G;
                    if (ri < cw.s.n) {
                        const float inv = sum == 0.f ? 0.f : 1.f / sum;
                        uint16_t *op = a.out + (int64_t)(cw.s.r0 + ri) * a.out_stride + (int64_t)(h * a.G + r % a.G) * D;
                        uint2 pk;
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(pk.x) : "f"(acc4.y * inv), "f"(acc4.x * inv));
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(pk.y) : "f"(acc4.w * inv), "f"(acc4.z * inv));
                        reinterpret_cast<uint2 *>(op)[d4] = pk;
                    }
                } else {
                    reinterpret_cast<float4 *>(a.part_o + ((int64_t)part * ROWS + row) * D)[d4] = acc4;
                    if (d4 == 0)
                        reinterpret_cast<float2 *>(a.part_ml)[(int64_t)part * ROWS + row] = make_float2(top, sum);
                }
            }
        }
        if (!whole) {
            // the CTAs that share the unit: its first tile's to its last's
            const int64_t u0 = wpos - cw.ta, u1 = u0 + cw.tiles - 1;
            const int c0 = (int)(((u0 + 1) * C - 1) / total), c1 = (int)(((u1 + 1) * C - 1) / total);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const bool last = atomicAdd(a.counters + c0, 1u) == (unsigned)(c1 - c0);
                if (last) a.counters[c0] = 0;
                __threadfence();
                sh_last = last;
            }
            __syncthreads();
            if (sh_last) {
                const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml);
                for (int i = tid; i < ROWS * D / 4; i += kAtThreads) {
                    const int row = i / (D / 4), d4 = i % (D / 4);
                    const int r = row0 + row, ri = r / a.G;
                    if (ri >= cw.s.n) continue;
                    // parts in CTA order: the first CTA's holds the unit's start
                    float top = -INFINITY;
                    for (int c = c0; c <= c1; ++c)
                        top = fmaxf(top, __ldcg(&ml[(int64_t)(2 * c + (c == c0)) * ROWS + row]).x);
                    const float ref = at_ref(top);
                    float sum = 0.f;
                    float4 acc4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                    for (int c = c0; c <= c1; ++c) {
                        const int64_t pr = (int64_t)(2 * c + (c == c0)) * ROWS + row;
                        const float2 x = __ldcg(&ml[pr]);
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(a.part_o + pr * D) + d4);
                        const float f = at_exp2(x.x - ref);
                        sum += x.y * f;
                        acc4.x += v.x * f; acc4.y += v.y * f; acc4.z += v.z * f; acc4.w += v.w * f;
                    }
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    uint16_t *op = a.out + (int64_t)(cw.s.r0 + ri) * a.out_stride + (int64_t)(h * a.G + r % a.G) * D;
                    uint2 pk;
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(pk.x) : "f"(acc4.y * inv), "f"(acc4.x * inv));
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(pk.y) : "f"(acc4.w * inv), "f"(acc4.z * inv));
                    reinterpret_cast<uint2 *>(op)[d4] = pk;
                }
            }
        }
        wpos += cw.tb - cw.ta;
        if (!more) break;
        cw = nw;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

static int attn_ctas()
{
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

size_t kv8_attn_workspace_bytes(const lowbit_kv8_cache &c)
{
    const size_t ctas = attn_ctas(), rows = kAtMaxRT * 8;
    return align256(ctas * 4) + align256(2 * ctas * rows * 8) + align256(2 * ctas * rows * c.head_dim * 4);
}

lowbit_status kv8_attn_launch(const lowbit_kv8_cache &c, const lowbit_kv8_batch &b, const uint16_t *q,
                              int64_t q_stride, int q_heads, float scale, uint16_t *out, int64_t out_stride,
                              void *workspace, cudaStream_t st)
{
    Kv8Attn a;
    a.v = kv8_view(c, b);
    a.k = c.k; a.vv = c.v; a.ks = c.k_scales; a.vs = c.v_scales;
    a.q = q; a.out = out; a.q_stride = q_stride; a.out_stride = out_stride;
    a.G = q_heads / c.n_heads;
    a.page_log2 = c.page_tokens == 32 ? 5 : c.page_tokens == 64 ? 6 : 7;
    a.scale_log2 = scale * 1.4426950408889634f;
    const int ctas = attn_ctas();
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.counters = reinterpret_cast<unsigned *>(ws);
    ws += align256((size_t)ctas * 4);
    a.part_ml = reinterpret_cast<float *>(ws);
    ws += align256((size_t)2 * ctas * kAtMaxRT * 8 * 8);
    a.part_o = reinterpret_cast<float *>(ws);
    if (!&g_at_fault) return LOWBIT_ERR_CUDA;
    // eight query rows per tile where that holds a sequence's rows, else sixteen
    // (each tile of keys and values is then read for twice the rows)
    const bool one = (int64_t)b.n_rows * a.G <= 8 * (int64_t)b.n_seqs;
    void (*kern)(const Kv8Attn);
    int smem;
    if (c.head_dim == 128) {
        kern = one ? k_kv8_attn<128, 1> : k_kv8_attn<128, 2>;
        smem = one ? AttnShape<128, 1>::kBytes : AttnShape<128, 2>::kBytes;
    } else {
        kern = one ? k_kv8_attn<64, 1> : k_kv8_attn<64, 2>;
        smem = one ? AttnShape<64, 1>::kBytes : AttnShape<64, 2>::kBytes;
    }
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return LOWBIT_ERR_CUDA;
    const cudaError_t e = launch_pdl(kern, dim3(ctas), dim3(kAtThreads), smem, st, a);
    return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

}  // namespace lowbit
