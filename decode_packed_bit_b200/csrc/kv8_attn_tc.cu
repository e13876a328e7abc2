// kv8_attn_tc.cu -- attention of many rows per sequence (prompts) over the KV8
// cache, on the 5th-generation tensor cores (tcgen05.mma kind::f16).
//
// out[r] = sum_t softmax_t(scale q[r] . k[t]) v[t], t up to the row's position,
// in one pass with a running maximum and sum per row (Milakov and Gimelshein,
// "Online normalizer calculation for softmax", 2018).  Both products take the
// cache's codes as f16, which holds them exactly:
//   - a row of q is scaled by a power of two to its own largest value and becomes
//     f16: its bf16 mantissa fits, and entries below 2^-14 of the largest are off
//     by 2^-25 of it at most.  S = Q K^T is then exact but for fp32 sums; the
//     row's power, the softmax scale and k's page scale multiply S.
//   - v's page scale goes into the exponent: with x = s + log2(vs) a probability
//     is exp2(x - m), m a reference 7 below a running maximum of x, so P fits f16 for
//     any scales: at most 2^15, off by 2^-11 of itself, and normal down to 2^-21 of
//     the largest, zero below 2^-32.  (m at the maximum itself left an f16 of 2^-24
//     of it a single bit: where one token leads 4000 others by e^16.4 and has no
//     value of its own, the output was a fifth off.)  O sums P times codes, and the row
//     sum takes P / vs in fp32.
// m follows the maximum only when that is more than 8 ahead, which after the first
// tiles is rare (any reference gives the same quotient): only then O is rescaled
// in tensor memory.
//
// A CTA takes two tiles of up to 128 rows (query tokens x the query heads that
// share a cache head) of one sequence and cache head, which share K and V:
//   warps 0-3, 4-7  softmax of tile 0, 1: a thread has a row, so its maximum and
//                   sum need no exchange; S is read from tensor memory twice, 32
//                   columns at a time, and P goes over S's place there;
//   warps 8-11      turn codes into f16 in shared memory (K-major keys, MN-major
//                   values, 128-byte swizzle), the next tile's codes under way in
//                   registers;
//   warp 12         allocates tensor memory and issues the MMAs, one tile's
//                   products while the other tile is in its softmax.
// At best bound by the exponentials (16 a clock and SM) and the tensor cores alike:
// 128 x 128 scores take about 1024 clocks of either at D = 128.  Measured, three
// prompts of 1900, 1866 and 797 rows over 8192, 1866 and 3509 tokens, 40 query
// heads on 8: 511 us, 0.44 of the cuBLAS bf16 rate; a step of two tiles takes about
// 5400 clocks, of which a tile waits 1700 for its scores, looks for their maximum
// for 850 and makes its probabilities in 2600.  Leaving out the exponentials, or all
// MMAs but one, changes a step by less than a tenth: it is a chain of latencies
// that three warps a scheduler do not fill.
// Every mbarrier wait is bounded in time; one that runs out records a fault and
// the CTA leaves its loops, releases tensor memory and exits.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "kv8_common.cuh"
#include "tc_common.cuh"

namespace lowbit {

__device__ unsigned g_att_range;  // a length, page or row was out of range
__device__ unsigned g_att_fault;  // a bounded wait ran out

constexpr int kAttRows = 128;    // rows of a tile
constexpr int kAttTokens = 128;  // tokens of a step
constexpr int kAttConvWarp = 8, kAttMmaWarp = 12;
constexpr int kAttThreads = 13 * 32;
constexpr int kAttInfo = 4;  // steps of scales kept
constexpr float kAttBelow = 7.f;        // the reference lies so far below the maximum it was taken from,
constexpr float kAttAhead = 8.f;        // which may have grown by so much: P is at most 2^15
constexpr float kAttUnit = 0x1p-7f;     // the row sum's unit: P / vs at the reference's own maximum

struct Kv8AttnTc {
    Kv8View v;
    const int8_t *k, *vv;
    const float *ks, *vs;
    const uint16_t *q;
    uint16_t *out;
    int64_t q_stride, out_stride;
    int G, tokens;     // query heads per cache head; tokens of a tile: 128 / G
    int items;
    float scale_log2;  // |scale| * log2(e)
    float sign;        // of scale
};

template <int D>
struct AttnTc {
    static constexpr int kHalves = D / 64;                 // 64 entries are a 128-byte row
    static constexpr int kTile = kHalves * 128 * 128;      // bytes of 128 rows of f16
    static constexpr int kQ = 0;                           // [2]
    static constexpr int kK = 2 * kTile;                   // [2 stages]
    static constexpr int kV = 4 * kTile;                   // [2 stages]
    static constexpr int kInfoAt = 6 * kTile;              // [kAttInfo][4 chunks] {ks or -1, log2 vs, kAttUnit / vs, vs != 0}
    static constexpr int kBars = kInfoAt + kAttInfo * 4 * 16;
    static constexpr int kBytes = kBars + 16 * 8 + 16 + 1024;
    static constexpr unsigned kTmem = 512;                 // S 0, S 1, O 0, O 1
};

// Wait for a phase with the whole warp polling: 110 clocks from the arrival to
// going on, against 250 when lane 0 polls and the warp votes on its verdict; a
// step has several such hand-offs in a row.  Bounded as mbar_wait is.
__device__ __forceinline__ bool att_wait(uint64_t *bar, unsigned parity)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const unsigned long long t0 = globaltimer_ns();
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > kTcWaitNs)) {
            atomicExch(&g_att_fault, 1u);
            return false;
        }
    }
}

// Shared-memory descriptors, 128-byte swizzle.  K-major: rows 128 bytes apart,
// 8-row groups 1024.
__device__ __forceinline__ uint64_t att_desc_k(unsigned addr)
{
    return ((uint64_t)(addr >> 4) & 0x3FFFull) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// MN-major: 64 entries of MN a row of 128 bytes, rows (k) 128 bytes apart, 8-row
// groups 1024, the next 64 entries 16384 on.
__device__ __forceinline__ uint64_t att_desc_mn(unsigned addr)
{
    return ((uint64_t)(addr >> 4) & 0x3FFFull) | (1024ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

template <bool ACC>
__device__ __forceinline__ void att_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "n"(ACC ? 1 : 0));
}
template <bool ACC>
__device__ __forceinline__ void att_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "n"(ACC ? 1 : 0));
}

__device__ __forceinline__ void att_ld32(uint32_t addr, uint32_t (&v)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
        "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr));
}
__device__ __forceinline__ void att_ld16(uint32_t addr, uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr));
}
__device__ __forceinline__ void att_st16(uint32_t addr, const uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
// The values that were loaded are operands of the wait: what uses them can then
// not be moved before it (a volatile asm keeps its place among others of its kind only).
__device__ __forceinline__ void att_wait_ld(uint32_t (&v)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                   "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])::"memory");
}
__device__ __forceinline__ void att_wait_ld(uint32_t (&v)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                   "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]),
                   "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]),
                   "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])::"memory");
}
__device__ __forceinline__ void att_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float att_exp2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t att_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four int8 codes -> two words of exact f16: an f16 in [1024, 2048) has steps of 1, so the
// bits 0x6400 + u are 1024 + u for a byte u (Kim, Henry, Fahim and Awadalla, "Who says
// elephants can't run", 2022), and u = code + 128.
__device__ __forceinline__ uint2 att_codes(uint32_t w)
{
    const uint32_t u = w ^ 0x80808080u;
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(a) : "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(b) : "r"(0x64806480u));
    return make_uint2(a, b);
}

// The largest x = s + log2(vs) of 32 columns of a row (columns < left where MASK).
template <bool MASK>
__device__ __forceinline__ float att_top(const uint32_t (&v)[32], const float4 &in, int left, float row_f)
{
    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int y = 0; y < 32; ++y) top[y & 3] = fmaxf(top[y & 3], !MASK || y < left ? __uint_as_float(v[y]) : -INFINITY);
    const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    // (32 tokens without a page have in.x < 0)
    return in.x >= 0.f && (!MASK || most > -INFINITY) ? fmaf(most, row_f * in.x, in.y) : -INFINITY;
}

// Their probabilities, two a word, and their sum over vs in parts of kAttUnit.
template <bool MASK>
__device__ __forceinline__ float att_probs(uint32_t (&p)[16], const uint32_t (&v)[32], const float4 &in, int left, float row_f,
                                           float ref)
{
    const float f = row_f * in.x, g = in.y - ref;
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int y = 0; y < 16; ++y) {
        float p0 = att_exp2(fmaf(__uint_as_float(v[2 * y]), f, g));
        float p1 = att_exp2(fmaf(__uint_as_float(v[2 * y + 1]), f, g));
        if (MASK) {
            if (2 * y >= left) p0 = 0.f;
            if (2 * y + 1 >= left) p1 = 0.f;
        }
        sum[0] += p0;
        sum[1] += p1;
        p[y] = att_f16x2(p0, p1);
    }
    if (in.w == 0.f)  // values of zero, or no page
#pragma unroll
        for (int y = 0; y < 16; ++y) p[y] = 0;
    return in.x >= 0.f ? (sum[0] + sum[1]) * in.z : 0.f;
}

// Two tiles' rows of a sequence: rows [i0, i0 + rows) of sequence b, whose last sees
// `seen` tokens, in `steps` steps.  rows = 0: an item past a sequence's rows.
struct AttUnit {
    int b, i0, rows, seen, steps;
    Kv8Seq s;
};
__device__ __forceinline__ AttUnit att_unit(const Kv8AttnTc &a, int item)
{
    AttUnit u = {};
    const int pair = 2 * a.tokens;
    int nth = 0;
    u.b = item;
    if (a.v.row_start) {
        u.b = kv8_find_seq(a.v, item, pair, 1);
        if (u.b < 0) return u;
        nth = item - (max(__ldg(a.v.row_start + u.b), 0) / pair + u.b);
    }
    u.s = kv8_seq(a.v, u.b, &g_att_range);
    const int64_t i0 = (int64_t)nth * pair;
    if (i0 >= u.s.n) return u;
    u.i0 = (int)i0;
    u.rows = min(pair, u.s.n - u.i0);
    u.seen = min(max(u.s.len - u.s.n + u.i0 + u.rows, 0), u.s.len);
    u.steps = (u.seen + kAttTokens - 1) / kAttTokens;
    return u;
}

template <int D>
__global__ void __launch_bounds__(kAttThreads, 1) k_kv8_attn_tc(const Kv8AttnTc a)
{
    using S = AttnTc<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const unsigned smem0 = smem_u32(smem);
    float4 *info = reinterpret_cast<float4 *>(smem + S::kInfoAt);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::kBars);
    uint64_t *kfull = bars, *kempty = bars + 2, *vfull = bars + 4, *vempty = bars + 6;
    uint64_t *sfull = bars + 8, *pready = bars + 10, *pvdone = bars + 12, *done = bars + 14, *qfull = bars + 15;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 16);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait_primary();

    // ---- the unit: those with more tokens to see first ----
    const int H = a.v.H, h = blockIdx.x % H;
    int item = (int)((a.items - 1) - blockIdx.x / H);  // within a sequence that is the order already
    if (a.v.n_seqs > 1 && a.items <= kAttThreads) {
        // between sequences it is not: every CTA ranks the items by their steps
        // (in the order of the rows, the longest sequence's could come last, and
        // the SMs wait for them: 624 against 511 us for the three prompts above)
        int *cost = reinterpret_cast<int *>(smem);
        if (threadIdx.x < kAttThreads) cost[threadIdx.x] = (int)threadIdx.x < a.items ? att_unit(a, threadIdx.x).steps : -1;
        __syncthreads();
        const int mine = cost[threadIdx.x];
        int rank = 0;
        for (int u = 0; u < a.items; u += 4) {
            const int4 c = reinterpret_cast<const int4 *>(cost)[u / 4];
            const int t = (int)threadIdx.x - u;  // equal ones in order
            rank += c.x > mine || (c.x == mine && t > 0);
            rank += c.y > mine || (c.y == mine && t > 1);
            rank += c.z > mine || (c.z == mine && t > 2);
            rank += c.w > mine || (c.w == mine && t > 3);
        }
        if ((int)threadIdx.x < a.items && rank == (int)(blockIdx.x / H)) cost[kAttThreads] = threadIdx.x;
        __syncthreads();
        item = cost[kAttThreads];
        __syncthreads();  // its place is q's
    }
    const AttUnit unit = att_unit(a, item);
    if (unit.rows == 0) return;
    const Kv8Seq &s = unit.s;
    const int b = unit.b, i0 = unit.i0, rows = unit.rows, seen = unit.seen, steps = unit.steps;
    const bool two = rows > a.tokens;

    if (threadIdx.x == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(kfull + x, 4);
            mbar_init(kempty + x, 1);
            mbar_init(vfull + x, 4);
            mbar_init(vempty + x, 1);
            mbar_init(sfull + x, 2);  // the MMAs, and the thread that knows the scales are there
            mbar_init(pready + x, 4);
            mbar_init(pvdone + x, 1);
        }
        mbar_init(done, 1);
        mbar_init(qfull, kAttConvWarp);
        mbar_fence_init();
    }
    if (warp == kAttMmaWarp) tmem_alloc(tmem_slot, S::kTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;

    // ---- q of a thread's row into shared memory ----
    const int tile = warp >> 2;  // softmax warps
    int lim = seen;  // a place without a row sees everything, as zeros: no masks for its sake
    float row_f = 0.f;
    int64_t out_at = -1;
    if (warp < kAttConvWarp) {
        const int r = threadIdx.x & 127, i = r / a.G, ti = i0 + tile * a.tokens + i;
        const bool valid = i < a.tokens && ti < i0 + rows;
        const uint16_t *qp = a.q;
        if (valid) {
            lim = min(max(s.len - s.n + ti + 1, 0), s.len);
            const int64_t row = s.r0 + ti, col = (int64_t)(h * a.G + r % a.G) * D;
            qp = a.q + row * a.q_stride + col;
            out_at = row * a.out_stride + col;
        }
        // the row twice, 128 bytes of it at a time (all of it in registers would
        // spill): its largest value, then its entries
        float top = 0.f;
        bool bad = false;
#pragma unroll 1
        for (int c0 = 0; c0 < D / 8; c0 += 8) {
            uint4 u[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) u[c] = valid ? __ldg(reinterpret_cast<const uint4 *>(qp) + c0 + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const uint32_t w[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float f0 = fabsf(__uint_as_float(w[y] << 16)), f1 = fabsf(__uint_as_float(w[y] & 0xFFFF0000u));
                    top = fmaxf(top, fmaxf(f0, f1));
                    bad |= !(f0 <= FLT_MAX) || !(f1 <= FLT_MAX);
                }
            }
        }
        // the power of two at or below the largest value (2^126 for 2^127, too)
        const bool some = top >= 0x1p-100f && !bad;
        const uint32_t e = min(__float_as_uint(top) >> 23, 253u);
        const float down = some ? __uint_as_float((254u - e) << 23) * a.sign : 0.f;
        row_f = bad && lim > 0 ? NAN : some ? __uint_as_float(e << 23) * a.scale_log2 : 0.f;
        uint8_t *qs = smem + S::kQ + tile * S::kTile + r * 128;
#pragma unroll 1
        for (int c0 = 0; c0 < D / 8; c0 += 8) {
            uint4 u[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) u[c] = valid ? __ldg(reinterpret_cast<const uint4 *>(qp) + c0 + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const uint32_t w[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
                uint32_t o[4];
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    o[y] = some ? att_f16x2(__uint_as_float(w[y] << 16) * down, __uint_as_float(w[y] & 0xFFFF0000u) * down) : 0u;
                *reinterpret_cast<uint4 *>(qs + (c0 >> 3) * 16384 + ((c ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(qfull);
        if (tile == 0 || two) {
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t ts = tmem + lanes + (uint32_t)(tile * 128), to = tmem + lanes + (uint32_t)(256 + tile * 128);
            float m = -INFINITY, l = 0.f;
            const int lim_min = __reduce_min_sync(0xffffffffu, lim);
            // O *= f, once the products into it so far are done
            auto rescale = [&](int i, float f) {
                if (!att_wait(pvdone + tile, (i - 1) & 1)) return false;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t o[16];
                    att_ld16(to + 16 * c, o);
                    att_wait_ld(o);
#pragma unroll
                    for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                    att_st16(to + 16 * c, o);
                }
                return true;
            };
            for (int i = 0; i < steps; ++i) {
                if (!att_wait(sfull + tile, i & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float4 *inf = info + (i % kAttInfo) * 4;
                const bool masked = (i + 1) * kAttTokens > lim_min;
                const int left = lim - i * kAttTokens;  // columns this row sees
                // 32 columns at a time, in loops that are not unrolled: the roles'
                // code together has to stay in the SM's instruction cache (with
                // both passes unrolled, masked and not, it was fetched from the
                // GPC's cache over and over, which bound the kernel)
                float x = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t v[32];
                    att_ld32(ts + 32 * c, v);
                    const float4 in = inf[c];
                    att_wait_ld(v);
                    x = fmaxf(x, masked ? att_top<true>(v, in, left - 32 * c, row_f) : att_top<false>(v, in, left - 32 * c, row_f));
                    __syncwarp();
                }
                const bool grow = x > m + (kAttBelow + kAttAhead);
                if (__any_sync(0xffffffffu, grow)) {
                    const float now = grow ? x - kAttBelow : m, f = grow ? att_exp2(m - now) : 1.f;
                    m = now;
                    l *= f;
                    if (i > 0 && !rescale(i, f)) {
                        ok = false;
                        break;
                    }
                }
                const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {  // P's columns lie below those of S still to be read
                    uint32_t v[32], p[16];
                    att_ld32(ts + 32 * c, v);
                    const float4 in = inf[c];
                    att_wait_ld(v);
                    l += masked ? att_probs<true>(p, v, in, left - 32 * c, row_f, ref)
                                : att_probs<false>(p, v, in, left - 32 * c, row_f, ref);
                    __syncwarp();
                    att_st16(ts + 16 * c, p);
                }
                att_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pready + tile);
            }
            if (ok && steps > 0) ok = att_wait(pvdone + tile, (steps - 1) & 1);
            tc_fence_after();
            if (ok) {
                const float inv = l == 0.f ? 0.f : kAttUnit / l;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t v[32];
                    if (steps > 0) {
                        att_ld32(to + 32 * c, v);
                        att_wait_ld(v);
                    } else {
#pragma unroll
                        for (int y = 0; y < 32; ++y) v[y] = 0;
                    }
                    if (out_at >= 0) {
                        uint4 *op = reinterpret_cast<uint4 *>(a.out + out_at + 32 * c);
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            uint32_t o[4];
#pragma unroll
                            for (int z = 0; z < 4; ++z)
                                asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                                    : "=r"(o[z])
                                    : "f"(__uint_as_float(v[8 * y + 2 * z + 1]) * inv), "f"(__uint_as_float(v[8 * y + 2 * z]) * inv));
                            op[y] = make_uint4(o[0], o[1], o[2], o[3]);
                        }
                    }
                }
            }
        }
    } else if (warp < kAttMmaWarp) {
        // ---- codes to f16: this thread's 16-byte pieces of a step are rows
        // 8 (4 (x / halves) + w) + lane % 8, pieces 4 (x % halves) + lane / 8 ----
        constexpr int NP = 4 * S::kHalves;
        const int w = warp - kAttConvWarp, r7 = lane & 7, c4 = lane >> 3;
        uint4 rk[NP], rv[NP];
        // Lane c < 4 knows the page of the step's 32 tokens from 32 c on (-1: none),
        // looked up one step ahead of the codes, and the first warp's its scales.
        float2 raw_info = make_float2(-1.f, 0.f);  // ks (-1: no page), vs
        auto pages_of = [&](int i) {
            const int tok = i * kAttTokens + (lane & 3) * 32;
            return tok < seen ? kv8_page(a.v, b, tok >> a.v.P_log2, &g_att_range) : -1;
        };
        const unsigned own = (unsigned)(8 * w + r7) * D + c4 * 16;  // of 32 tokens, this thread's first piece
        auto load = [&](const int8_t *codes, int i, int pages, uint4 (&raw)[NP]) {
            const int8_t *src[4];  // the 32 tokens from 32 y on, null without a page
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int page = __shfl_sync(0xffffffffu, pages, y), slot = (i * kAttTokens + 32 * y) & (a.v.P - 1);
                src[y] = page < 0 ? nullptr : codes + ((((int64_t)page * H + h) << a.v.P_log2) + slot) * D + own;
            }
#pragma unroll
            for (int x = 0; x < NP; ++x) {
                const int8_t *p = src[x / S::kHalves];
                raw[x] = make_uint4(0, 0, 0, 0);
                if (p) raw[x] = __ldg(reinterpret_cast<const uint4 *>(p + (x % S::kHalves) * 64));
            }
        };
        auto load_info = [&](int page) {
            raw_info = make_float2(-1.f, 0.f);
            if (w == 0 && lane < 4 && page >= 0) {
                const int64_t ph = (int64_t)page * H + h;
                raw_info = make_float2(__ldg(a.ks + ph), __ldg(a.vs + ph));
            }
        };
        auto store_info = [&](int i) {
            if (w == 0 && lane < 4) {
                // a page of zeros (its probabilities still count in the row's
                // sum) stands with a scale that never leads the maximum
                const float vs = raw_info.y, e = vs < 0x1p-100f ? 0x1p-60f : vs;
                info[(i % kAttInfo) * 4 + lane] = make_float4(raw_info.x, log2f(e), kAttUnit / e, vs < 0x1p-100f ? 0.f : 1.f);
            }
        };
        auto store = [&](unsigned at, const uint4 (&raw)[NP]) {
#pragma unroll
            for (int x = 0; x < NP; ++x) {
                const int row = 8 * (4 * (x / S::kHalves) + w) + r7;
                const uint2 p0 = att_codes(raw[x].x), p1 = att_codes(raw[x].y), p2 = att_codes(raw[x].z), p3 = att_codes(raw[x].w);
                const unsigned base = at + (x % S::kHalves) * 16384 + row * 128;
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(base + (((2 * c4) ^ r7) << 4)), "r"(p0.x), "r"(p0.y),
                             "r"(p1.x), "r"(p1.y)
                             : "memory");
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(base + (((2 * c4 + 1) ^ r7) << 4)), "r"(p2.x), "r"(p2.y),
                             "r"(p3.x), "r"(p3.y)
                             : "memory");
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
        };
        // Keys run a step ahead of values: the scores of step i + 1 are issued with
        // P V of step i.
        int page_k = pages_of(0), page_v = page_k;  // of the keys, of the values loaded next
        load(a.k, 0, page_k, rk);
        load_info(page_k);
        for (int i = 0; i <= steps; ++i) {
            // keys of step i, values of step i - 1
            const int next = pages_of(i + 1);
            if (i < steps) {
                if (i > 1 && !att_wait(kempty + (i & 1), ((i >> 1) - 1) & 1)) break;
                store_info(i);
                store(smem0 + S::kK + (i & 1) * S::kTile, rk);
                if (lane == 0) mbar_arrive(kfull + (i & 1));
                load(a.k, i + 1, next, rk);
                load_info(next);
            }
            if (i > 0) {
                const int o = i - 1;
                if (o > 1 && !att_wait(vempty + (o & 1), ((o >> 1) - 1) & 1)) break;
                store(smem0 + S::kV + (o & 1) * S::kTile, rv);
                if (lane == 0) mbar_arrive(vfull + (o & 1));
            }
            load(a.vv, i, page_v, rv);
            page_v = next;
        }
    } else {
        // ---- MMAs: f16 operands, fp32 sums, M = 128 ----
        const uint32_t idesc_s = (1u << 4) | ((uint32_t)(kAttTokens >> 3) << 17) | ((uint32_t)(kAttRows >> 4) << 24);
        const uint32_t idesc_o = (1u << 4) | (1u << 16) /*B is MN-major*/ | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(kAttRows >> 4) << 24);
        // MMA operands have to be in uniform registers: what comes from a warp
        // reduction is the same for the whole warp in the compiler's eyes too, and
        // tile and stage are constants of the unrolled code, so that a
        // descriptor is a sum of such a value and an immediate.
        const uint32_t base = __reduce_max_sync(0xffffffffu, tmem);
        const uint32_t sm = __reduce_max_sync(0xffffffffu, smem0);
        const int last = __reduce_max_sync(0xffffffffu, steps);
        const bool both = __any_sync(0xffffffffu, two);
        const uint64_t desc_k0 = att_desc_k(sm), desc_v0 = att_desc_mn(sm + S::kV);
        auto scores = [&](auto tile_c, auto stage_c) {
            constexpr int q = decltype(tile_c)::value, st = decltype(stage_c)::value;
            constexpr int qo = (S::kQ + q * S::kTile) >> 4, ko = (S::kK + st * S::kTile) >> 4;
            if (elect_one()) {
                att_mma_ss<false>(base + q * 128, desc_k0 + qo, desc_k0 + ko, idesc_s);
#pragma unroll
                for (int k = 1; k < D / 16; ++k) {
                    const int at = (k >> 2) * 1024 + (k & 3) * 2;
                    att_mma_ss<true>(base + q * 128, desc_k0 + (qo + at), desc_k0 + (ko + at), idesc_s);
                }
                umma_commit(sfull + q);
                mbar_arrive(sfull + q);
                if (q == 1 || !both) umma_commit(kempty + st);
            }
            __syncwarp();
        };
        auto values = [&](auto tile_c, auto stage_c, bool first) {
            constexpr int q = decltype(tile_c)::value, st = decltype(stage_c)::value;
            constexpr int vo = (st * S::kTile) >> 4;
            const uint32_t d = base + (256 + q * 128), p = base + q * 128;
            if (elect_one()) {
                if (first)
                    att_mma_ts<false>(d, p, desc_v0 + vo, idesc_o);
                else
                    att_mma_ts<true>(d, p, desc_v0 + vo, idesc_o);
#pragma unroll
                for (int k = 1; k < kAttTokens / 16; ++k) att_mma_ts<true>(d, p + 8 * k, desc_v0 + (vo + k * 128), idesc_o);
                umma_commit(pvdone + q);
                if (q == 1 || !both) umma_commit(vempty + st);
            }
            __syncwarp();
        };
        // a tile's P V of step i, then its scores of step i + 1
        auto step = [&](auto tile_c, auto stage_c, int i) {
            constexpr int q = decltype(tile_c)::value, st = decltype(stage_c)::value;
            if (i >= 0) {
                if (!att_wait(pready + q, i & 1)) return false;
                if (q == 0 && !att_wait(vfull + st, (i >> 1) & 1)) return false;
                tc_fence_after();
                values(tile_c, stage_c, i == 0);
            }
            if (i + 1 < last) {
                if (q == 0 && !att_wait(kfull + (st ^ 1), ((i + 1) >> 1) & 1)) return false;
                tc_fence_after();
                scores(tile_c, std::integral_constant<int, st ^ 1>{});
            }
            return true;
        };
        using C0 = std::integral_constant<int, 0>;
        using C1 = std::integral_constant<int, 1>;
        bool go = att_wait(qfull, 0);
        for (int i = -1; go && i < last; i += 2) {  // odd steps lie in stage 1
            if (!step(C0{}, C1{}, i) || (both && !step(C1{}, C1{}, i))) break;
            if (i + 1 >= last) break;
            if (!step(C0{}, C0{}, i + 1) || (both && !step(C1{}, C0{}, i + 1))) break;
        }
        // also after a failed wait: `done` tells that every MMA issued has
        // completed, before tensor memory is released
        if (elect_one()) umma_commit(done);
        __syncwarp();
        att_wait(done, 0);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kAttMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, S::kTmem);
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// Units of the call, at most: pairs of tiles, see kv8_find_seq.
static int64_t attn_tc_units(const lowbit_kv8_cache &c, const lowbit_kv8_batch &b, int q_heads)
{
    const int64_t pair = 2 * (kAttRows / (q_heads / c.n_heads));
    return (b.row_start ? b.n_rows / pair + b.n_seqs : b.n_seqs) * c.n_heads;
}

// Which calls.  Time of the integer kernel over this one's: with 4096 rows (row,
// query head, over all cache heads) 0.50-0.53, 8192 0.98-0.99, 12288 1.46, 16384
// 1.8-1.9, and 1.09 with 64 rows a sequence and head (32 sequences x 16 rows, four heads
// a cache head).  Long contexts are among these (1 sequence, 64 heads on 8: 64 rows over
// 32768 tokens 373 us against 741; 128 rows over 32768 729 against 745, over 131072 2844
// against 2864; 192 rows over 32768 1090 against 746; 1024 rows of 8 heads on 1 over
// 16384 374 against 380), although this kernel does not cut a unit along its tokens
// and leaves most SMs idle there: the 8192 rows are 32 units.  Rows are averaged over the
// call's sequences: a long prompt takes single rows beside it with it.
bool kv8_attn_tc_takes(const lowbit_kv8_cache &c, const lowbit_kv8_batch &b, int q_heads)
{
    const int64_t rows = (int64_t)b.n_rows * (q_heads / c.n_heads);
    return rows >= 64 * (int64_t)b.n_seqs && rows * c.n_heads >= 32 * 256 && attn_tc_units(c, b, q_heads) < (int64_t(1) << 31);
}

lowbit_status kv8_attn_tc_launch(const lowbit_kv8_cache &c, const lowbit_kv8_batch &b, const uint16_t *q,
                                 int64_t q_stride, int q_heads, float scale, uint16_t *out, int64_t out_stride,
                                 cudaStream_t st)
{
    Kv8AttnTc a;
    a.v = kv8_view(c, b);
    a.k = c.k; a.vv = c.v; a.ks = c.k_scales; a.vs = c.v_scales;
    a.q = q; a.out = out; a.q_stride = q_stride; a.out_stride = out_stride;
    a.G = q_heads / c.n_heads;
    a.tokens = kAttRows / a.G;
    a.scale_log2 = fabsf(scale) * 1.4426950408889634f;
    a.sign = scale < 0.f ? -1.f : 1.f;
    const int64_t units = attn_tc_units(c, b, q_heads);
    a.items = (int)(units / c.n_heads);
    void (*kern)(const Kv8AttnTc) = c.head_dim == 128 ? k_kv8_attn_tc<128> : k_kv8_attn_tc<64>;
    const int smem = c.head_dim == 128 ? AttnTc<128>::kBytes : AttnTc<64>::kBytes;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return LOWBIT_ERR_CUDA;
    const cudaError_t e = launch_pdl(kern, dim3((unsigned)units), dim3(kAttThreads), smem, st, a);
    return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

// Bit 0: a length, page or row out of range; bit 1: a bounded wait ran out; < 0:
// not to be read.
int kv8_attn_tc_fault_flags()
{
    unsigned r = 0, f = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&r, g_att_range, sizeof(r)) != cudaSuccess) return -1;
    if (cudaMemcpyFromSymbol(&f, g_att_fault, sizeof(f)) != cudaSuccess) return -1;
    cudaMemcpyToSymbol(g_att_range, &zero, sizeof(zero));
    cudaMemcpyToSymbol(g_att_fault, &zero, sizeof(zero));
    return (r ? 1 : 0) | (f ? 2 : 0);
}

}  // namespace lowbit
