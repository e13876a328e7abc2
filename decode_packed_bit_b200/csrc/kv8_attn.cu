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
// Nothing is converted per cached value: a key's bytes are a fragment as they
// lie, and ldmatrix transposes v's (tokens have to run along a fragment's words).
//
// Layout of the work.  A unit is (sequence, cache head, RT * 8 query rows); its
// tokens come in tiles of 32.  All tiles of all units, in order, are cut into
// equal ranges, one per CTA (one CTA per SM), and a CTA's range into equal ranges
// for its warps; lengths are read on the device, so a captured graph follows
// them.  A warp goes through its range alone, with a cp.async ring of key and
// value halves of tiles that runs on across the ends of units, and writes the
// units that lie wholly within.  What it has of a unit cut at its range's start
// or end stays in shared memory; one barrier later the CTA joins those parts in
// order.  A unit cut between CTAs is joined, in CTA order, by the last of them to
// arrive (a counter in the workspace, left zeroed), so the result does not
// depend on timing.
//
// Measured: 64 sequences of up to 8192 tokens, 40 query heads on 8 cache heads of
// 128, one row each 65 us, 5.2 TB/s over the whole launch (2 us until a CTA knows its
// range, 60 for the tiles, 3 for a CTA's join and 2 for the last units'); one
// sequence of 131071 tokens, four rows, 67.4 us, 4.0 TB/s (eight warps with 16 rows
// each: issue and latency); 777 tokens 11 us, a chain of loads and of code that is
// fetched and run once.
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
    float scale_log2; // |scale| * log2(e)
    float limbs;      // 32512 with the sign of scale
    unsigned *counters;   // [CTAs], zero between calls
    float *part_ml;       // [2 CTAs][rows][2]
    float *part_o;        // [2 CTAs][rows][D]
};

template <int D, int RT>
struct AttnShape {
    static constexpr int kWarps = RT == 1 ? 12 : 8;  // 168 or 255 registers a thread
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kRows = RT * 8;
    static constexpr int kHalf = kAtTile * D;                              // bytes of a tile's keys, or of its values
    static constexpr int kPitch = D + 8;                                  // floats per row of a part: no bank conflicts
    static constexpr int kPart = kRows * kPitch * 4;                       // a part's sums
    static constexpr int kQBytes = RT * D * 16;                            // q fragments of a warp, [RT][D / 32][32] x 16 bytes
    static constexpr int kFixed = kWarps * (kPart + kQBytes + 2 * 2 * kRows * 4);
    static constexpr int kFit = (224 * 1024 - kFixed) / (kWarps * (kHalf + 4));
    static constexpr int kHalves = kFit >= 5 ? 5 : 3;  // odd: what a place in the loop copies is keys, or values, always
    static constexpr int kRing = kWarps * kHalves * kHalf;
    static constexpr int kQ = kRing;
    static constexpr int kHead = kQ + kWarps * kQBytes;                    // sums of a unit cut at the warp's start
    static constexpr int kStats = kHead + kWarps * kPart;                  // [m, l][2 warps][rows] fp32
    static constexpr int kScales = kStats + 2 * 2 * kWarps * kRows * 4;    // [warp][half] fp32
    static constexpr int kBytes = kScales + kWarps * kHalves * 4;
    static_assert(kHalves >= 3 && kHalves * kHalf >= kPart && kBytes <= 225 * 1024, "attention ring does not fit");
};

__device__ __forceinline__ void at_cp16(unsigned dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void at_cp4(unsigned dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// FIRST: the sums start at zero.
template <bool FIRST>
__device__ __forceinline__ void at_mma_ss(int (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if (FIRST)
        asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                     : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(0));
    else
        asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void at_mma_us(int (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(0));
}
// Bytes of 32 rows x 16 columns, one row address per lane, transposed: {b[0], b[2]}
// and {b[1], b[3]} are the B fragments (k = row) of columns 0-7 and 8-15.
__device__ __forceinline__ void at_ldsm_t(uint32_t (&b)[4], unsigned addr)
{
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
                 : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                 : "r"(addr));
}
__device__ __forceinline__ uint4 at_lds16(unsigned a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ float at_exp2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kAtLog2P = 15.994353436858858f;  // log2(65280): 255 * 256, so that both limbs fit a byte

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

// A part of a unit that a warp has less than all tiles of.
struct AttnPart {
    int64_t start;  // the unit's first tile, in the whole work
    int tiles, r0, row0, h, n;
    bool there;
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

// The first segment of the range of `left` tiles that starts `off` tiles after
// sequence b's first.
template <int RT>
__device__ __forceinline__ void at_start(AttnWalk &w, const Kv8Attn &a, int b, int64_t off, int64_t left)
{
    at_sequence<RT>(w, a, b);
    while (off >= (int64_t)w.units * w.tiles) {
        off -= (int64_t)w.units * w.tiles;
        at_sequence<RT>(w, a, w.b + 1);
    }
    w.left = left;
    w.u = (int)(off / w.tiles);
    w.ta = (int)(off % w.tiles);
    at_segment<RT>(w, a);
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

__device__ __forceinline__ uint32_t at_bf16x2(float lo, float hi)
{
    uint32_t v;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(hi), "f"(lo));
    return v;
}
__device__ __forceinline__ void at_store4(uint16_t *p, const float4 &v, float f)
{
    *reinterpret_cast<uint2 *>(p) = make_uint2(at_bf16x2(v.x * f, v.y * f), at_bf16x2(v.z * f, v.w * f));
}

template <int D, int RT>
__global__ void __launch_bounds__(AttnShape<D, RT>::kThreads, 1) k_kv8_attn(const Kv8Attn a)
{
    using S = AttnShape<D, RT>;
    constexpr int W = S::kWarps, ROWS = S::kRows, NJ = D / 8, NH = S::kHalves, KS = D / 32;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t sh_sum[W], sh_units[W];
    __shared__ int64_t sh_off;
    __shared__ int sh_b, sh_first[2], sh_n[2];
    // a warp's parts of cut units: the head is 2 warp, the tail 2 warp + 1
    __shared__ AttnPart parts[2 * W];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    pdl_launch_dependents();
    pdl_wait_primary();

    // ---- this CTA's range of the batch's tiles ----
    const int per = (a.v.n_seqs + S::kThreads - 1) / S::kThreads;
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
    if (tid < 2 * W) parts[tid].there = false;
    __syncthreads();
    int64_t total = 0, before = 0;
    units = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        if (w < warp) before += sh_sum[w];
        total += sh_sum[w];
        units += sh_units[w];
    }
    if (total == 0) return;
    // CTAs: one per unit where units are short (no joining between CTAs), else
    // enough that a warp has three tiles
    const int64_t C = min(min((int64_t)gridDim.x, total), max(units, (total + 3 * W - 1) / (3 * W)));
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
    // ---- this warp's range (none is empty before another that is not) ----
    const int64_t active = min((int64_t)W, w1 - w0);
    const int64_t v0 = min((int64_t)warp, active) * (w1 - w0) / active, v1 = min((int64_t)warp + 1, active) * (w1 - w0) / active;
    const unsigned smem0 = (unsigned)__cvta_generic_to_shared(smem);
    float *stat_m = reinterpret_cast<float *>(smem + S::kStats), *stat_l = stat_m + 2 * W * ROWS;
    if (v1 > v0) {
    AttnWalk cw;
    at_start<RT>(cw, a, sh_b, sh_off + v0, v1 - v0);
    int64_t wpos = w0 + v0;  // of cw's segment

    // ---- this warp's ring ----
    const unsigned ring = smem0 + warp * NH * S::kHalf, scal = smem0 + S::kScales + warp * NH * 4;
    // 16-byte slots of 128-byte lines, permuted so that the fragment loads below
    // meet eight different ones; lane l copies pieces l, l + 32, ...
    constexpr int CH = D / 16;
    const int prow = lane / CH, pch = lane % CH;
    const unsigned kdst = D == 128 ? prow * 128 + ((pch ^ (4 * (prow & 1))) << 4) : (prow >> 1) * 128 + (((prow & 1) * 4 + pch) << 4);
    const unsigned vdst = D == 128 ? prow * 128 + ((pch ^ prow) << 4)
                                   : (prow >> 1) * 128 + (((prow & 1) * 4 + (pch ^ (prow >> 1))) << 4);
    // this lane's row of a tile's values, for the transposing loads
    const unsigned vrow = D == 128 ? lane * 128 + ((lane & 7) << 4) : (lane >> 1) * 128 + (lane & 1) * 64 + (((lane >> 1) & 3) << 4);
    AttnWalk ld = cw;
    int ld_tile = ld.ta, ld_slot = 0;
    bool ld_more = true;
    int64_t ld_ph = -1;  // the tile's page and head, -1 for an absent page
    const int8_t *ld_v = nullptr;  // its values, this lane's first piece
    unsigned present = 0;  // one bit per slot: keys that are there
    // Copies the next tile's keys (nothing at the end of the range), then its values.
    auto issue_k = [&]() {
        while (ld_more && ld_tile >= min(ld.tb, ld.seen)) {
            ld_more = at_next<RT>(ld, a);
            ld_tile = ld.ta;
        }
        ld_ph = -1;
        present &= ~(1u << ld_slot);
        if (ld_more) {
            const int tok = ld_tile * kAtTile;
            const int page = kv8_page(a.v, ld.b, tok >> a.v.P_log2, &g_at_fault);
            ++ld_tile;
            if (page >= 0) {
                present |= 1u << ld_slot;
                ld_ph = (int64_t)page * a.v.H + ld.h;
                const int64_t at = ((ld_ph << a.v.P_log2) + (tok & (a.v.P - 1))) * D + lane * 16;
                const int8_t *src = a.k + at;
                ld_v = a.vv + at;
                const unsigned st = ring + ld_slot * S::kHalf + kdst;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) at_cp16(st + i * 512, src + i * 512);
                if (lane == 0) at_cp4(scal + ld_slot * 4, a.ks + ld_ph);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        ld_slot = ld_slot + 1 == NH ? 0 : ld_slot + 1;
    };
    auto issue_v = [&]() {
        if (ld_ph >= 0) {
            const unsigned st = ring + ld_slot * S::kHalf + vdst;
            // rows advance by 4 (D = 128, two permutations in turn) or 8
#pragma unroll
            for (int i = 0; i < D / 16; ++i) at_cp16((D == 128 && (i & 1) ? st ^ 64 : st) + i * 512, ld_v + i * 512);
            if (lane == 0) at_cp4(scal + ld_slot * 4, a.vs + ld_ph);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        ld_slot = ld_slot + 1 == NH ? 0 : ld_slot + 1;
    };
#pragma unroll 1
    for (int i = 0; i < NH / 2; ++i) {
        issue_k();
        issue_v();
    }
    int slot = 0;
    const unsigned qsm = smem0 + S::kQ + warp * S::kQBytes;

    while (true) {
        const int h = cw.h, row0 = (cw.u - h * cw.rts) * ROWS;
        // ---- q of the unit's rows as two int8 limbs, in fragment order ----
        float rowf[RT];
        int lim[RT], lim_min = INT_MAX;
        __syncwarp();
#pragma unroll
        for (int m = 0; m < RT; ++m) {
            const int r = row0 + m * 8 + g, i = r / a.G;
            const bool valid = i < cw.s.n;
            // rows past the sequence's see what is there, as zeros
            lim[m] = valid ? min(max(cw.s.len - cw.s.n + i + 1, 0), cw.s.len) : cw.s.len;
            lim_min = min(lim_min, lim[m]);
            const uint16_t *qp = a.q + (int64_t)(cw.s.r0 + i) * a.q_stride + (int64_t)(h * a.G + r % a.G) * D + t * 16;
            uint4 u[D / 64][2];
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    u[c][x] = valid ? __ldg(reinterpret_cast<const uint4 *>(qp + c * 64 + x * 8)) : make_uint4(0, 0, 0, 0);
            float top = 0.f;
            bool bad = false;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const uint32_t w = reinterpret_cast<const uint32_t *>(u[c])[x];
                    const float f0 = fabsf(__uint_as_float(w << 16)), f1 = fabsf(__uint_as_float(w & 0xFFFF0000u));
                    top = fmaxf(top, fmaxf(f0, f1));
                    bad |= !(f0 <= FLT_MAX) || !(f1 <= FLT_MAX);
                }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            bad |= __shfl_xor_sync(0xffffffffu, (int)bad, 1) != 0;
            bad |= __shfl_xor_sync(0xffffffffu, (int)bad, 2) != 0;
            const float inv = top >= 0x1p-100f && !bad ? a.limbs / top : 0.f;
            // a row that sees nothing gives zeros whatever it holds: `fac` below takes 0 * rowf
            rowf[m] = lim[m] <= 0 ? 0.f : bad ? NAN : top * (1.f / 32512.f) * a.scale_log2;
            // 16-byte chunk t + 4 c of a key meets entries 64 c + 16 t ..: two
            // fragments of 8 entries each
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t raw[4] = {u[c][x].x, u[c][x].y, u[c][x].z, u[c][x].w};
                    uint32_t limb[4] = {0, 0, 0, 0};  // hi and lo of entries 0-3, of 4-7
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const float f = __uint_as_float(y & 1 ? raw[y / 2] & 0xFFFF0000u : raw[y / 2] << 16);
                        const int v = __float2int_rn(f * inv), vh = (v + 128) >> 8;
                        limb[y / 4 * 2] |= (uint32_t)(vh & 0xFF) << (8 * (y & 3));
                        limb[y / 4 * 2 + 1] |= (uint32_t)((v - vh * 256) & 0xFF) << (8 * (y & 3));
                    }
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(qsm + ((m * KS + 2 * c + x) * 32 + lane) * 16),
                                 "r"(limb[0]), "r"(limb[1]), "r"(limb[2]), "r"(limb[3])
                                 : "memory");
                }
        }
        lim_min = __reduce_min_sync(0xffffffffu, lim_min);  // (a lane reads back what it wrote itself)

        float o[RT][NJ][2], mx[RT], l[RT];
#pragma unroll
        for (int m = 0; m < RT; ++m) {
            mx[m] = -INFINITY;
            l[m] = 0.f;
#pragma unroll
            for (int j = 0; j < NJ; ++j) o[m][j][0] = o[m][j][1] = 0.f;
        }

        for (int tile = cw.ta; tile < min(cw.tb, cw.seen); ++tile) {
            asm volatile("cp.async.wait_group %0;" ::"n"(NH - 2) : "memory");
            __syncwarp();
            const bool there = (present >> slot) & 1;
            issue_k();  // into the slot read last, while this one is worked on
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
                for (int c = 0; c < D / 64; ++c) {
                    uint32_t qf[RT][2][4];
#pragma unroll
                    for (int m = 0; m < RT; ++m)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint4 u = at_lds16(qsm + ((m * KS + 2 * c + y) * 32 + lane) * 16);
                            qf[m][y][0] = u.x; qf[m][y][1] = u.y; qf[m][y][2] = u.z; qf[m][y][3] = u.w;
                        }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int tr = 16 * (j >> 1) + 4 * (g >> 1) + 2 * (j & 1) + (g & 1);
                        const int sl = D == 128 ? ((t + 4 * c) ^ (4 * (g & 1))) : (g & 1) * 4 + t;
                        const uint4 x = at_lds16(st + (D == 128 ? tr : tr >> 1) * 128 + (sl << 4));
#pragma unroll
                        for (int m = 0; m < RT; ++m) {
                            if (c == 0)
                                at_mma_ss<true>(acc[m][j], qf[m][0], x.x, x.y);
                            else
                                at_mma_ss<false>(acc[m][j], qf[m][0], x.x, x.y);
                            at_mma_ss<false>(acc[m][j], qf[m][1], x.z, x.w);
                        }
                    }
                }
                const bool masked = (tile + 1) * kAtTile > lim_min;
#pragma unroll
                for (int m = 0; m < RT; ++m) {
                    const float f = rowf[m] * ks;  // >= 0: the largest score is the largest integer's
                    int s[8], top = INT_MIN;
                    const int tok = tile * kAtTile + 4 * t;
#pragma unroll
                    for (int x = 0; x < 8; ++x) {  // token 16 (x / 4) + 4 t + x % 4
                        const int j = 2 * (x >> 2) + ((x >> 1) & 1), e = x & 1;
                        s[x] = acc[m][j][e] * 256 + acc[m][j][2 + e];
                    }
                    if (masked) {
                        asm volatile("" ::: "memory");  // a branch, not eight selections in every tile
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            if (tok + 16 * (x >> 2) + (x & 3) >= lim[m]) s[x] = INT_MIN;
                    }
#pragma unroll
                    for (int x = 0; x < 8; ++x) top = max(top, s[x]);
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    // the sums of limbs stay above INT_MIN
                    const float tm = top == INT_MIN ? -INFINITY : (float)top * f;
                    // probabilities in parts of 1 / 65280 of the tile's largest.  The difference
                    // from it is taken in integers: exact, and the largest's own is 65280 at any
                    // score.  (Taken in fp32, from scores of 2^16 on an ulp of tm is enough to
                    // lift it past the 16 bits that the limbs hold.)  What wraps is masked.
                    uint32_t v[8], sum = 0;
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        v[x] = __float2uint_rn(at_exp2(fmaf((float)(int)((unsigned)s[x] - (unsigned)top), f, kAtLog2P)));
                    }
                    if (masked) {
                        asm volatile("" ::: "memory");
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            if (s[x] == INT_MIN) v[x] = 0;  // a small f alone would not make it so
                    }
#pragma unroll
                    for (int x = 0; x < 8; ++x) sum += v[x];
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
            issue_v();
            if (there) {
                const unsigned vb = ring + slot * S::kHalf;
                float vs;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(vs) : "r"(scal + slot * 4));
#pragma unroll
                for (int m = 0; m < RT; ++m) fac[m] *= vs;
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t b[4];
                    at_ldsm_t(b, (vb + vrow) ^ (c << 4));
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int m = 0; m < RT; ++m) {
                            int p[4];
                            at_mma_us(p, pf[m], b[y], b[2 + y]);
                            o[m][2 * c + y][0] = fmaf((float)(p[0] * 256 + p[2]), fac[m], o[m][2 * c + y][0]);
                            o[m][2 * c + y][1] = fmaf((float)(p[1] * 256 + p[3]), fac[m], o[m][2 * c + y][1]);
                        }
                }
            }
            slot = slot + 1 == NH ? 0 : slot + 1;
        }

        // ---- the segment's end: out, or a part of a cut unit ----
        const bool from = cw.ta == 0, to = cw.tb == cw.tiles;
        AttnWalk nw = cw;
        const bool more = at_next<RT>(nw, a);
        const int part = 2 * warp + (from ? 1 : 0);
        if (!more) asm volatile("cp.async.wait_group 0;" ::: "memory");  // the ring may take the tail
        __syncwarp();
#pragma unroll
        for (int m = 0; m < RT; ++m) {
            l[m] += __shfl_xor_sync(0xffffffffu, l[m], 1);
            l[m] += __shfl_xor_sync(0xffffffffu, l[m], 2);
            if (from && to) {
                const int r = row0 + m * 8 + g, ri = r / a.G;
                if (ri < cw.s.n) {
                    const float inv = l[m] == 0.f ? 0.f : 1.f / l[m];
                    uint16_t *op = a.out + (int64_t)(cw.s.r0 + ri) * a.out_stride + (int64_t)(h * a.G + r % a.G) * D + 2 * t;
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
                        *reinterpret_cast<uint32_t *>(op + 8 * j) = at_bf16x2(o[m][j][0] * inv, o[m][j][1] * inv);
                }
            } else {
                float *dst = reinterpret_cast<float *>(from ? smem + warp * NH * S::kHalf : smem + S::kHead + warp * S::kPart) +
                             (m * 8 + g) * S::kPitch + 2 * t;
#pragma unroll
                for (int j = 0; j < NJ; ++j) *reinterpret_cast<float2 *>(dst + 8 * j) = make_float2(o[m][j][0], o[m][j][1]);
                if (t == 0) {
                    stat_m[part * ROWS + m * 8 + g] = mx[m];
                    stat_l[part * ROWS + m * 8 + g] = l[m];
                }
            }
        }
        if (!(from && to) && lane == 0) parts[part] = AttnPart{wpos - cw.ta, cw.tiles, cw.s.r0, row0, h, cw.s.n, true};
        if (!more) break;
        wpos += cw.tb - cw.ta;
        cw = nw;
    }
    }
    __syncthreads();

    // ---- join the parts of units cut between warps ----
    // Lane p is part p; a unit's begin with the tail of the warp it starts in (or
    // with the head of the CTA's first).
    const bool there = lane < 2 * W && parts[min(lane, 2 * W - 1)].there;
    const unsigned all = __ballot_sync(0xffffffffu, there);
    const unsigned begins = __ballot_sync(0xffffffffu, there && ((lane & 1) || lane == 0)), upto = (2u << lane) - 1;
    const unsigned ends = __ballot_sync(0xffffffffu, there && (!(all & ~upto) || (begins >> (__ffs(all & ~upto) - 1) & 1)));
    auto out_at = [&](const AttnPart &u, int row, int d4) -> uint16_t * {  // null past the sequence's rows
        const int r = u.row0 + row, ri = r / a.G;
        return ri < u.n ? a.out + (int64_t)(u.r0 + ri) * a.out_stride + (int64_t)(u.h * a.G + r % a.G) * D + d4 * 4 : nullptr;
    };
    // First what each part counts for: a warp has a row, so that a unit's maximum and
    // sum are scans over its lanes.  (Loops that are not unrolled: this code runs
    // once, and fetching it is most of its time.)
    float *tops = reinterpret_cast<float *>(smem + S::kQ);  // q's fragments are done with
    for (int row = warp; row < ROWS; row += W) {
        const int first = 31 - __clz(begins & upto), at = lane * ROWS + row;
        const int last = ends & ~(upto >> 1) ? __ffs(ends & ~(upto >> 1)) - 1 : 31;
        float m = there ? stat_m[at] : -INFINITY, l = there ? stat_l[at] : 0.f, top = m;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_up_sync(0xffffffffu, top, o);
            if (lane - o >= first) top = fmaxf(top, x);
        }
        top = __shfl_sync(0xffffffffu, top, last);
        const float f = at_exp2(m - at_ref(top));
        l *= f;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_up_sync(0xffffffffu, l, o);
            if (lane - o >= first) l += x;
        }
        l = __shfl_sync(0xffffffffu, l, last);
        if (there) {
            stat_m[at] = f;
            stat_l[at] = l;
            tops[at] = top;
        }
    }
    __syncthreads();
#pragma unroll 1
    for (int x = tid; x < ROWS * (D / 4); x += S::kThreads) {
        const int row = x / (D / 4), d4 = x % (D / 4);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kBatch = 4;
#pragma unroll 1
        for (unsigned todo = all; todo;) {
            int p[kBatch];
            float f[kBatch];
            float4 v[kBatch];
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                p[q] = __ffs(todo) - 1;
                todo &= todo - 1;
                if (p[q] >= 0) {
                    f[q] = stat_m[p[q] * ROWS + row];
                    v[q] = *reinterpret_cast<const float4 *>(
                        reinterpret_cast<const float *>(p[q] & 1 ? smem + (p[q] >> 1) * NH * S::kHalf : smem + S::kHead + (p[q] >> 1) * S::kPart) +
                        row * S::kPitch + d4 * 4);
                }
            }
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                if (p[q] < 0) break;
                if (begins >> p[q] & 1) o = make_float4(0.f, 0.f, 0.f, 0.f);
                o.x += v[q].x * f[q]; o.y += v[q].y * f[q]; o.z += v[q].z * f[q]; o.w += v[q].w * f[q];
                if (ends >> p[q] & 1) {
                    const AttnPart &u = parts[p[q]];
                    const float sum = stat_l[p[q] * ROWS + row];
                    if (u.start >= w0 && u.start + u.tiles <= w1) {
                        if (uint16_t *op = out_at(u, row, d4)) at_store4(op, o, sum == 0.f ? 0.f : 1.f / sum);
                    } else {
                        // the CTA's part: 0 of a unit that started before its range, else 1
                        const int64_t pr = (2 * (int64_t)blockIdx.x + (u.start >= w0 ? 1 : 0)) * ROWS + row;
                        reinterpret_cast<float4 *>(a.part_o + pr * D)[d4] = o;
                        if (d4 == 0) reinterpret_cast<float2 *>(a.part_ml)[pr] = make_float2(tops[p[q] * ROWS + row], sum);
                    }
                }
            }
        }
    }
    // ---- join the parts of units cut between CTAs: the first and the last unit ----
    __syncthreads();  // the CTA's parts are written; the counters' release carries them
    if (warp < 2 && lane == 0) {
        int n = 0, c0 = 0;
        if (all) {
            const AttnPart &u = parts[warp == 0 ? __ffs(all) - 1 : 31 - __clz(all)];
            const bool again = warp == 1 && u.start == parts[__ffs(all) - 1].start;
            if (!again && !(u.start >= w0 && u.start + u.tiles <= w1)) {
                // the CTAs that share the unit: its first tile's to its last's
                c0 = (int)(((u.start + 1) * C - 1) / total);
                const int c1 = (int)(((u.start + u.tiles) * C - 1) / total);
                unsigned seen;
                asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(seen) : "l"(a.counters + c0) : "memory");
                if (seen == (unsigned)(c1 - c0)) {
                    a.counters[c0] = 0;
                    n = c1 - c0 + 1;
                }
            }
        }
        sh_first[warp] = c0;
        sh_n[warp] = n;
    }
    __syncthreads();
    for (int k = 0; k < 2; ++k) {
        const int n = sh_n[k], c0 = sh_first[k];
        if (n == 0) continue;
        const AttnPart &u = parts[k == 0 ? __ffs(all) - 1 : 31 - __clz(all)];
        // parts in CTA order; the first CTA's holds the unit's start
        auto part = [&](int c, int row) { return (2 * (int64_t)(c0 + c) + (c == 0 ? 1 : 0)) * ROWS + row; };
        const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml);
        float *fac = reinterpret_cast<float *>(smem), *inv = fac + ROWS * n;  // over the ring
        __syncthreads();
        for (int row = warp; row < ROWS; row += W) {
            const float2 s = lane < n ? __ldcg(ml + part(lane, row)) : make_float2(-INFINITY, 0.f);
            float top = s.x;
            for (int c = lane + 32; c < n; c += 32) top = fmaxf(top, __ldcg(ml + part(c, row)).x);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float ref = at_ref(top), f = at_exp2(s.x - ref);
            float sum = s.y * f;
            if (lane < n) fac[row * n + lane] = f;
            for (int c = lane + 32; c < n; c += 32) {
                const float2 x = __ldcg(ml + part(c, row));
                const float g = at_exp2(x.x - ref);
                fac[row * n + c] = g;
                sum += x.y * g;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) inv[row] = sum == 0.f ? 0.f : 1.f / sum;
        }
        __syncthreads();
        // a batch's loads are all under way before the first is used
        constexpr int kItems = ROWS * (D / 4), NI = (kItems + S::kThreads - 1) / S::kThreads, kBatch = 20 / NI;
        float4 o[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < n; c += kBatch) {
            float4 v[NI][kBatch];
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int q = 0; q < kBatch; ++q) {
                    const int x = tid + i * S::kThreads;
                    if (x < kItems && c + q < n)
                        v[i][q] = __ldcg(reinterpret_cast<const float4 *>(a.part_o + part(c + q, x / (D / 4)) * D) + x % (D / 4));
                }
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int q = 0; q < kBatch; ++q) {
                    const int x = tid + i * S::kThreads;
                    if (x < kItems && c + q < n) {
                        const float f = fac[x / (D / 4) * n + c + q];
                        o[i].x += v[i][q].x * f; o[i].y += v[i][q].y * f; o[i].z += v[i][q].z * f; o[i].w += v[i][q].w * f;
                    }
                }
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int x = tid + i * S::kThreads;
            if (x < kItems)
                if (uint16_t *op = out_at(u, x / (D / 4), x % (D / 4))) at_store4(op, o[i], inv[x / (D / 4)]);
        }
    }
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
    a.scale_log2 = fabsf(scale) * 1.4426950408889634f;
    a.limbs = scale < 0.f ? -32512.f : 32512.f;
    const int ctas = attn_ctas();
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.counters = reinterpret_cast<unsigned *>(ws);
    ws += align256((size_t)ctas * 4);
    a.part_ml = reinterpret_cast<float *>(ws);
    ws += align256((size_t)2 * ctas * kAtMaxRT * 8 * 8);
    a.part_o = reinterpret_cast<float *>(ws);
    // Eight query rows per tile where that holds a sequence's rows, or where there
    // are few units and L2 holds the cache, so that the units of the same tokens, side
    // by side on neighbouring SMs, read it from HBM once (1 sequence x 4 rows x 8192
    // tokens 17.7 us against 24.3 with sixteen, 32 x 2 rows x 1024 tokens 12.1 against
    // 22.8).  Else sixteen, so that a tile of keys and values is read for twice the
    // rows: what L2 does not hold comes from HBM again with eight (9 x 4 rows x 16384
    // tokens, 302 MB, 119 us against 190; 8 x 4 x 32768, 537 MB, 109 against 148; many
    // units, 64 x 4 x 4096, 111 against 173; 1 x 4 x 131071, 268 MB, by run 62-72
    // against 67).  Lengths are on the device, so the rule takes what the cache and the
    // page table could hold: a pool and a table of more than 128 MB get sixteen rows,
    // however short the sequences are.
    constexpr int64_t kShared = int64_t(128) << 20;
    const int64_t seqs = b.n_seqs, tiles = ((int64_t)b.n_rows * a.G + 8 * seqs - 1) / (8 * seqs);
    const int64_t bytes = std::min<int64_t>(c.n_pages, seqs * b.max_pages) * c.n_heads * c.page_tokens * c.head_dim * 2;
    const bool one = tiles <= 1 || (tiles * seqs * c.n_heads <= 2 * ctas && bytes <= kShared);
    void (*kern)(const Kv8Attn);
    int smem, threads;
    if (c.head_dim == 128) {
        kern = one ? k_kv8_attn<128, 1> : k_kv8_attn<128, 2>;
        smem = one ? AttnShape<128, 1>::kBytes : AttnShape<128, 2>::kBytes;
        threads = one ? AttnShape<128, 1>::kThreads : AttnShape<128, 2>::kThreads;
    } else {
        kern = one ? k_kv8_attn<64, 1> : k_kv8_attn<64, 2>;
        smem = one ? AttnShape<64, 1>::kBytes : AttnShape<64, 2>::kBytes;
        threads = one ? AttnShape<64, 1>::kThreads : AttnShape<64, 2>::kThreads;
    }
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return LOWBIT_ERR_CUDA;
    const cudaError_t e = launch_pdl(kern, dim3(ctas), dim3(threads), smem, st, a);
    return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

}  // namespace lowbit
