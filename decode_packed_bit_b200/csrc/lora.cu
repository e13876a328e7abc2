// lora.cu -- low-rank adapters of many requests beside a shared projection:
//     t[m] = A_i x[m],  y[m] = base[m] + s_i B_i t[m],  i = ids[m].
//
// Two launches.  The first forms t (fp32): a CTA takes rows, an adapter and a
// slice of K; its warps cut the slice between them and add up through shared
// memory in order.  Each lane's 16-byte loads of x and A are mma.sync m16n8k16
// fragments as they lie in memory (the k order inside a fragment is free as
// long as both operands share it).  The tensor core's accumulation cuts off a
// little with each step, so a warp moves its sums to fp32 adds every 256 k.
// The second launch adds s_i B_i t to base: t is summed over the slices in
// order, scaled and split into three bf16 numbers, which carry its 24 bits (two
// would leave an error of 2^-18 of t beside fp32 outputs); a warp holds the
// split of its rows in registers and walks over columns, 16 at a time, with base
// and B copied some steps ahead into a ring of its own (cp.async).  All it needs
// but t was there before the first launch began, so those copies start before
// it waits for t.  Only rows of the adapter at hand are stored,
// so what another adapter holds (infinities among it) cannot reach them.
//
// Which rows a CTA takes: up to kLoraFewRows rows (decode), 16 rows of one
// adapter, gathered, so that an adapter's weights are read once for them; beyond that
// (prompts, where neighbours share an adapter) blocks of 16 or 32 rows in the
// caller's order, with a pass for each adapter in the block.  Nothing is sorted.
// Bound by the adapters' bytes for decode, by base and y (8 bytes an output)
// for prompts.  Measured: 61 rows of two 5120 -> 17408 projections, ranks up to 64,
// 42.9 us (4.2 TB/s over both launches); 4096 rows, 4096 -> 11008, rank 32, 93.7 us
// (16 and 78, 4.6 TB/s in the second); one row, 4096 -> 4096, rank 16, 4.8 us, latency.
// The first launch moves its bytes at 1.7 to 2.3 TB/s only: its loads go straight
// into registers, 64 contiguous bytes of a row at a time, two steps ahead.
#include <algorithm>

#include "common.cuh"

namespace lowbit {

constexpr int kLoraMaxGroup = 16;
constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;
constexpr int kLoraMaxSlices = 64;
constexpr int kLoraFewRows = kLoraThreads;  // one id per thread

struct LoraArgs {
    const uint16_t *x;
    const int32_t *ids, *ranks;
    const float *scales;
    const uint16_t *a[kLoraMaxGroup], *b[kLoraMaxGroup];
    const float *base[kLoraMaxGroup];
    float *y[kLoraMaxGroup];
    float *t;  // [R][slices][M][rank]
    int M, N, K, rank, L;
    int slices, kslice;  // slices of kslice k (a multiple of 32)
    int cols;            // columns per CTA of the second launch
};

__device__ __forceinline__ void lora_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Of a block's ids (lane r holds row r's, -1 for none): the lanes that hold the
// first row of each distinct adapter.
__device__ __forceinline__ unsigned lora_distinct(int id, int lane)
{
    const unsigned same = __match_any_sync(0xffffffffu, id);
    return __ballot_sync(0xffffffffu, id >= 0 && (same & ((1u << lane) - 1)) == 0);
}

// Past L1: the second launch reads them before it waits for the first.
__device__ __forceinline__ int lora_id(const LoraArgs &a, int64_t m)
{
    if (m >= a.M) return -1;
    const int id = __ldcg(a.ids + m);
    return (unsigned)id < (unsigned)a.L ? id : -1;
}

__device__ __forceinline__ int lora_rank(const LoraArgs &a, int id)
{
    if (id < 0) return 0;
    return a.ranks ? min(max(__ldcg(a.ranks + id), 0), a.rank) : a.rank;
}

template <int NT, int RB>
struct LoraShrink {
    static constexpr int kLd = NT * 8 + 2;                                 // floats per row of a warp's sums
    static constexpr int kBytes = kLoraWarps * RB * 16 * kLd * 4;
};

// A warp's sums over [k0, k1) of the products of 16 RB rows of x (xp: the rows
// this lane loads, null for none) with `rank` rows of A, into shared memory.
template <int NT, int RB>
__device__ __forceinline__ void lora_dot(float *mine, const uint16_t *const (&xp)[RB][2], const uint16_t *w, int rank, int K,
                                         int k0, int k1, int g)
{
    constexpr int LD = LoraShrink<NT, RB>::kLd;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    int kc = k0;
    do {
        float acc[RB][NT][4];
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[b][n][c] = 0.f;
        const int ke = min(k1, kc + 256);
#pragma unroll(NT *RB <= 4 ? 4 : 2)
        for (int k = kc; k < ke; k += 32) {
            uint4 wv[NT], x[RB][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
                wv[n] = n * 8 + g < rank ? __ldg(reinterpret_cast<const uint4 *>(w + (int64_t)n * 8 * K + k)) : zero;
#pragma unroll
            for (int b = 0; b < RB; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    x[b][h] = xp[b][h] ? __ldg(reinterpret_cast<const uint4 *>(xp[b][h] + k)) : zero;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int b = 0; b < RB; ++b) {
                    lora_mma(acc[b][n], x[b][0].x, x[b][1].x, x[b][0].y, x[b][1].y, wv[n].x, wv[n].y);
                    lora_mma(acc[b][n], x[b][0].z, x[b][1].z, x[b][0].w, x[b][1].w, wv[n].z, wv[n].w);
                }
        }
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float2 *p = reinterpret_cast<float2 *>(mine + (b * 16 + h * 8) * LD + n * 8);
                    float2 s = make_float2(acc[b][n][2 * h], acc[b][n][2 * h + 1]);
                    if (kc > k0) {
                        s.x += p->x;
                        s.y += p->y;
                    }
                    *p = s;
                }
        kc += 256;
    } while (kc < k1);
}

// The sum over the CTA's warps of entries r, r + 1 of a row.
template <int NT, int RB>
__device__ __forceinline__ float2 lora_warps_sum(const float *red, int row, int r)
{
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int q = 0; q < kLoraWarps; ++q) {
        const float2 v = *reinterpret_cast<const float2 *>(red + (q * RB * 16 + row) * LoraShrink<NT, RB>::kLd + r);
        s.x += v.x;
        s.y += v.y;
    }
    return s;
}

// This warp's part of a slice of K.
__device__ __forceinline__ int2 lora_range(const LoraArgs &a, int slice, int warp)
{
    const int s0 = slice * a.kslice, s1 = min(a.K, s0 + a.kslice);
    const int sub = ((s1 - s0 + kLoraWarps - 1) / kLoraWarps + 31) / 32 * 32;
    const int k0 = min(s1, s0 + warp * sub);
    return make_int2(k0, min(s1, k0 + sub));
}

// Up to 16 rows of row m's adapter, in order, when m is the first of its adapter,
// or the 17th, 33rd ...: their number, and rows[] filled; 0 for the others and
// for rows without an adapter.  Called by all threads of a CTA, M <=
// kLoraFewRows; warp_n: a word per warp and one more.
struct LoraRows {
    int id, n, rank;
};
__device__ __forceinline__ LoraRows lora_gather(const LoraArgs &a, int m, int *rows, int *warp_n)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int mine = lora_id(a, tid), id = lora_id(a, m);
    const bool same = tid < a.M && mine == id && id >= 0;
    const unsigned vote = __ballot_sync(0xffffffffu, same), below = vote & ((1u << lane) - 1);
    if (lane == 0) warp_n[warp] = __popc(vote);
    __syncthreads();
    int at = __popc(below), n = 0, to_m = 0;  // same rows before this thread's, in all, in the warps before m's
#pragma unroll
    for (int w = 0; w < kLoraWarps; ++w) {
        const int x = warp_n[w];
        if (w < warp) at += x;
        if (w < m >> 5) to_m += x;
        n += x;
    }
    if (tid == m) warp_n[kLoraWarps] = at - to_m;
    __syncthreads();
    const int from = to_m + warp_n[kLoraWarps];
    if (same && at >= from && at < from + 16) rows[at - from] = tid;
    __syncthreads();
    return LoraRows{id, from % 16 ? 0 : min(16, n - from), lora_rank(a, id)};
}

// Few rows: grid (rows x slices, projections); the CTA of an adapter's first row
// takes 16 of its rows, that of the 17th the next, the others leave.
template <int NT>
__global__ void __launch_bounds__(kLoraThreads, NT == 8 ? 2 : 1) k_lora_shrink_few(const LoraArgs a)
{
    using S = LoraShrink<NT, 1>;
    extern __shared__ __align__(16) float red[];
    __shared__ int rows[16], warp_n[kLoraWarps + 1];
    pdl_wait_primary();
    pdl_launch_dependents();  // after the wait: the next launch may read whatever came before this one
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int slice = blockIdx.x % a.slices, m = blockIdx.x / a.slices, target = blockIdx.y;
    const LoraRows own = lora_gather(a, m, rows, warp_n);
    if (own.n == 0) return;
    const int2 k = lora_range(a, slice, warp);
    const uint16_t *w = a.a[target] + ((int64_t)own.id * a.rank + g) * a.K + t * 8;
    float *tp = a.t + ((int64_t)target * a.slices + slice) * a.M * a.rank;
    const int half = a.rank / 2;
    const uint16_t *xp[1][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        xp[0][h] = h * 8 + g < own.n ? a.x + (int64_t)rows[h * 8 + g] * a.K + t * 8 : nullptr;
    lora_dot<NT, 1>(red + (warp * 16 + g) * S::kLd + 2 * t, xp, w, own.rank, a.K, k.x, k.y, g);
    __syncthreads();
    for (int e = threadIdx.x; e < own.n * half; e += kLoraThreads) {
        const int row = e / half, r = e % half * 2;
        *reinterpret_cast<float2 *>(tp + (int64_t)rows[row] * a.rank + r) = lora_warps_sum<NT, 1>(red, row, r);
    }
}

// Many rows: grid (blocks of 16 RB rows x slices, projections, 2): z = 0 takes a
// block's first adapter, z = 1 its others (with one CTA for
// all, the blocks where prompts meet ended last: 102 us for the prompts above, so 93.7).
// NT: rank / 8, rounded up to 2, 4, 8 or 16.
template <int NT, int RB>
__global__ void __launch_bounds__(kLoraThreads) k_lora_shrink(const LoraArgs a)
{
    using S = LoraShrink<NT, RB>;
    extern __shared__ __align__(16) float red[];
    pdl_wait_primary();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int slice = blockIdx.x % a.slices, target = blockIdx.y;
    const int64_t m0 = (int64_t)(blockIdx.x / a.slices) * (16 * RB);
    const int id = lora_id(a, lane < 16 * RB ? m0 + lane : a.M);
    const int my_rank = lora_rank(a, id);
    const int2 k = lora_range(a, slice, warp);
    float *tp = a.t + ((int64_t)target * a.slices + slice) * a.M * a.rank;
    const int half = a.rank / 2;
    unsigned todo = lora_distinct(id, lane);
    const unsigned first = todo & (0u - todo);
    for (todo = blockIdx.z ? todo ^ first : first; todo; todo &= todo - 1) {
        const int src = __ffs(todo) - 1;
        const int i = __shfl_sync(0xffffffffu, id, src), rank = __shfl_sync(0xffffffffu, my_rank, src);
        const uint16_t *xp[RB][2];
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = b * 16 + h * 8 + g;
                xp[b][h] = __shfl_sync(0xffffffffu, id, r) == i ? a.x + (m0 + r) * a.K + t * 8 : nullptr;
            }
        lora_dot<NT, RB>(red + (warp * RB * 16 + g) * S::kLd + 2 * t, xp,
                         a.a[target] + ((int64_t)i * a.rank + g) * a.K + t * 8, rank, a.K, k.x, k.y, g);
        __syncthreads();
        for (int e = threadIdx.x; e < RB * 16 * half; e += kLoraThreads) {
            const int row = e / half, r = e % half * 2;
            if (lora_id(a, m0 + row) == i)
                *reinterpret_cast<float2 *>(tp + (m0 + row) * a.rank + r) = lora_warps_sum<NT, RB>(red, row, r);
        }
        __syncthreads();
    }
}

__device__ __forceinline__ void lora_cp16(unsigned dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// A warp's ring: per stage 16 columns of base for 16 RB rows, then of B.  B's
// column c lies in row (c / 2 % 2) * 8 + c / 4 * 2 + c % 2, which is tile j = c / 2 % 2,
// fragment column g, so that a thread's results are four consecutive columns of
// its rows; rows 32 or 96 bytes apart mod 128 keep the fragment loads (8 bytes a
// lane, four rows a phase) free of bank conflicts.
template <int KT, int RB>
struct LoraRing {
    static constexpr int kPitch = KT == 1 ? 32 : KT == 2 ? 96 : KT * 32 + 32;
    static constexpr int kBase = RB * 16 * 64;
    static constexpr int kStage = kBase + 16 * kPitch;
    static constexpr int kStages = KT >= 4 || RB == 2 ? 3 : 4;
    static constexpr int kBytes = kLoraWarps * kStages * kStage;
    static constexpr int kCtas = KT == 1 && RB == 1 ? 4 : KT <= 4 ? 2 : 1;  // per SM, by registers and ring
    static_assert(kBytes * kCtas <= 220 * 1024, "rings of an SM's CTAs");
};

// Where this lane's pieces (16 bytes) of 16 columns of B go in a stage; the
// pieces themselves lie one after the other in memory, lane by lane.  Bit q of
// the mask: piece q exists and holds entries below the adapter's rank; col: its
// column.
template <int KT, int RB>
struct LoraPieces {
    unsigned dst[KT], mask;
    int col[KT];
    __device__ __forceinline__ void set(int rank, int pool_rank, int lane)
    {
        const int per = pool_rank / 8;
        mask = 0;
#pragma unroll
        for (int q = 0; q < KT; ++q) {
            const int e = lane + 32 * q, c = e / per, ch = e % per;
            if (c < 16 && ch * 8 < rank) mask |= 1u << q;
            col[q] = c;
            dst[q] = ((c >> 1 & 1) * 8 + (c >> 2) * 2 + (c & 1)) * LoraRing<KT, RB>::kPitch + ch * 16;
        }
    }
    // src: this lane's first piece of the 16 columns; left: columns there are
    __device__ __forceinline__ void copy(unsigned to, const uint16_t *src, int left) const
    {
#pragma unroll
        for (int q = 0; q < KT; ++q)
            if ((mask >> q & 1) && col[q] < left) lora_cp16(to + dst[q], src + q * 256);
    }
};

// acc = the block's rows of t (f: their bf16 numbers, in NS fragments) times a stage's 16
// columns of B.  Steps of 16 entries beyond the adapter's rank are left out (with
// one or two steps the branch costs more than it saves: 110 against 93.7 us for
// 4096 rows of rank 32), and in the step that it ends in the entries from the rank on are cleared: they
// may hold anything.
template <int KT, int RB, int NS>
__device__ __forceinline__ void lora_mul(const uint32_t (&f)[RB][KT][NS][4], unsigned src, int rank, int g, int t,
                                         float (&acc)[RB][2][4])
{
#pragma unroll
    for (int q = 0; q < RB; ++q)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[q][j][c] = 0.f;
    const unsigned at = src + g * LoraRing<KT, RB>::kPitch + t * 8;
    uint2 bw[KT][2];
    auto load = [&](int k) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                         : "=r"(bw[k][j].x), "=r"(bw[k][j].y)
                         : "r"(at + j * 8 * LoraRing<KT, RB>::kPitch + k * 32));
    };
    if (KT <= 2)
#pragma unroll
        for (int k = 0; k < KT; ++k) load(k);
#pragma unroll
    for (int k = 0; k < KT; ++k) {
        if (KT > 2) {
            if (k * 16 >= rank) break;
            load(k);
        }
        if (k * 16 + 16 > rank) {
            const int left = rank - (k * 16 + 4 * t);
            const uint32_t mx = left <= 0 ? 0u : left == 1 ? 0xFFFFu : ~0u, my = left < 3 ? 0u : left == 3 ? 0xFFFFu : ~0u;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                bw[k][j].x &= mx;
                bw[k][j].y &= my;
            }
        }
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int q = 0; q < RB; ++q)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    lora_mma(acc[q][j], f[q][k][s][0], f[q][k][s][1], f[q][k][s][2], f[q][k][s][3], bw[k][j].x, bw[k][j].y);
    }
}

// Four columns of a row of base or y where rows are not 16-byte aligned.
__device__ __forceinline__ float4 lora_load4(const float *p, int left)
{
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (left > 0) v.x = __ldcg(p);
    if (left > 1) v.y = __ldcg(p + 1);
    if (left > 2) v.z = __ldcg(p + 2);
    if (left > 3) v.w = __ldcg(p + 3);
    return v;
}
template <bool VEC>
__device__ __forceinline__ void lora_store4(float *p, int left, const float4 &v)
{
    if (VEC) {
        if (left > 0) *reinterpret_cast<float4 *>(p) = v;
    } else {
        if (left > 0) p[0] = v.x;
        if (left > 1) p[1] = v.y;
        if (left > 2) p[2] = v.z;
        if (left > 3) p[3] = v.w;
    }
}

// Four entries of t of row m, adapter i: slices in order, scaled, 0 from the
// rank on.
__device__ __forceinline__ float4 lora_t4(const LoraArgs &a, int target, int64_t m, int i, int rank, int r)
{
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r >= rank) return s;
    const float *p = a.t + ((int64_t)target * a.slices * a.M + m) * a.rank + r;
#pragma unroll 4
    for (int q = 0; q < a.slices; ++q) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(p + (int64_t)q * a.M * a.rank));
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    const float f = a.scales ? __ldcg(a.scales + i) : 1.f;
    s.x *= f;
    s.y = rank - r > 1 ? s.y * f : 0.f;
    s.z = rank - r > 2 ? s.z * f : 0.f;
    s.w = rank - r > 3 ? s.w * f : 0.f;
    return s;
}

// The three bf16 numbers of four values as fragment words: out[s][w * 2].
__device__ __forceinline__ void lora_split(const float4 &v, uint32_t (&f)[3][4], int h)
{
    float p[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int s = 0; s < 3; ++s)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            uint32_t u;
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(p[2 * w + 1]), "f"(p[2 * w]));
            f[s][w * 2 + h] = u;
            p[2 * w] -= __uint_as_float(u << 16);
            p[2 * w + 1] -= __uint_as_float(u & 0xFFFF0000u);
        }
}

// A thread's four columns of tiles 0 and 1: rows g (h = 0) and g + 8 (h = 1).
__device__ __forceinline__ void lora_acc(float4 &o, const float (&acc)[2][4], int h)
{
    o.x += acc[0][2 * h]; o.y += acc[0][2 * h + 1]; o.z += acc[1][2 * h]; o.w += acc[1][2 * h + 1];
}

// One adapter's rows (16 at most) over columns [c0, n_end).  SMALL: up to four, whose
// three numbers lie in one fragment (rows 0-3 the first, 4-7 the second, 8-11
// the third), a third of the MMAs.
template <int KT, bool VEC, bool SMALL>
__device__ __forceinline__ void lora_expand_rows(const LoraArgs &a, const LoraRows &own, const int *rows, uint4 *frag, unsigned ring,
                                                 int c0, int n_end)
{
    using S = LoraRing<KT, 1>;
    constexpr int NS = SMALL ? 1 : 3, NH = SMALL ? 1 : 2, kRows = SMALL ? 4 : 16, kStep = kLoraWarps * 16;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3, target = blockIdx.z;
    const float *base = a.base[target];
    float *y = a.y[target];
    LoraPieces<KT, 1> pieces;
    pieces.set(own.rank, a.rank, lane);
    const uint16_t *b = a.b[target] + (int64_t)own.id * a.N * a.rank + lane * 8;
    int64_t at[NH];  // offsets of this thread's rows, -1 for none
#pragma unroll
    for (int h = 0; h < NH; ++h)
        at[h] = g < kRows && h * 8 + g < own.n ? (int64_t)rows[h * 8 + g] * a.N : -1;
    int n0 = c0 + warp * 16, ahead = n0, put = 0, get = 0;
    auto issue = [&]() {
        if (ahead < n_end) {
            const unsigned st = ring + put * S::kStage;
            if (VEC)
#pragma unroll
                for (int h = 0; h < NH; ++h) {  // row h * 8 + g, columns 4 t ..
                    if (at[h] >= 0 && ahead + 4 * t < a.N)
                        lora_cp16(st + (h * 8 + g) * 64 + t * 16, base + at[h] + ahead + 4 * t);
                }
            pieces.copy(st + S::kBase, b + (int64_t)ahead * a.rank, a.N - ahead);
            ahead += kStep;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        put = put + 1 == S::kStages ? 0 : put + 1;
    };
#pragma unroll
    for (int s = 0; s < S::kStages - 1; ++s) issue();
    pdl_wait_primary();
    for (int e = threadIdx.x; e < KT * 32; e += kLoraThreads) {
        const int k = e / 32, eg = (e & 31) >> 2, et = e & 3;
        uint32_t f[3][4];
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            const int row = h * 8 + (SMALL ? eg & 3 : eg);
            if (row < own.n) v = lora_t4(a, target, rows[row], own.id, own.rank, k * 16 + 4 * et);
            lora_split(v, f, h);
        }
        if (SMALL)
            frag[e] = eg < 4 ? make_uint4(f[0][0], f[2][0], f[0][2], f[2][2]) : make_uint4(f[1][0], 0, f[1][2], 0);
        else
#pragma unroll
            for (int s = 0; s < 3; ++s)
                frag[(k * 3 + s) * 32 + (e & 31)] = make_uint4(f[s][0], f[s][1], f[s][2], f[s][3]);
    }
    __syncthreads();
    uint32_t f[1][KT][NS][4];
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const uint4 u = frag[(k * NS + s) * 32 + lane];
            f[0][k][s][0] = u.x; f[0][k][s][1] = u.y; f[0][k][s][2] = u.z; f[0][k][s][3] = u.w;
        }
    for (; n0 < n_end; n0 += kStep) {
        asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 2) : "memory");
        __syncwarp();
        issue();  // into the stage read last
        const unsigned st = ring + get * S::kStage;
        get = get + 1 == S::kStages ? 0 : get + 1;
        const int n = n0 + 4 * t;
        float4 o[NH];
        float acc[1][2][4];
        lora_mul<KT, 1, NS>(f, st + S::kBase, own.rank, g, t, acc);
        if (SMALL)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c)  // rows g and g + 4, then g + 8
                    acc[0][j][c] += __shfl_xor_sync(0xffffffffu, acc[0][j][c], 16) + acc[0][j][2 + c];
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            if (VEC)
                asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                             : "=f"(o[h].x), "=f"(o[h].y), "=f"(o[h].z), "=f"(o[h].w)
                             : "r"(st + (h * 8 + g) * 64 + t * 16));
            else
                o[h] = lora_load4(base + (at[h] < 0 ? 0 : at[h]) + n, at[h] < 0 ? 0 : a.N - n);
        }
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            lora_acc(o[h], acc[0], h);
            if (at[h] >= 0) lora_store4<VEC>(y + at[h] + n, a.N - n, o[h]);
        }
        __syncwarp();  // every lane has read the stage
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Few rows: grid (rows, column ranges, projections); the CTA of an adapter's
// first (17th, ...) row takes 16 of its rows; a row without an adapter is copied.
// KT: rank / 16, rounded up to 1, 2, 4 or 8; VEC: rows of y are 16-byte aligned.
template <int KT, bool VEC>
__global__ void __launch_bounds__(kLoraThreads, LoraRing<KT, 1>::kCtas) k_lora_expand_few(const LoraArgs a)
{
    using S = LoraRing<KT, 1>;
    extern __shared__ __align__(128) uint8_t ring_mem[];
    __shared__ int rows[16], warp_n[kLoraWarps + 1];
    __shared__ uint4 frag[KT * 3 * 32];
    const unsigned ring = (unsigned)__cvta_generic_to_shared(ring_mem) + (threadIdx.x >> 5) * S::kStages * S::kStage;
    pdl_launch_dependents();
    const LoraRows own = lora_gather(a, blockIdx.x, rows, warp_n);
    const int c0 = blockIdx.y * a.cols, n_end = min(a.N, c0 + a.cols);
    if (own.n == 0) {
        const float *base = a.base[blockIdx.z];
        float *y = a.y[blockIdx.z];
        pdl_wait_primary();
        if (own.id < 0 && y != base)
            for (int n = c0 + threadIdx.x; n < n_end; n += kLoraThreads)
                y[(int64_t)blockIdx.x * a.N + n] = base[(int64_t)blockIdx.x * a.N + n];
        return;
    }
    // (one row, rank 16, 4096 x 4096: 4.8 us against 5.5 with the form for 16 rows)
    if (own.n <= 4)
        lora_expand_rows<KT, VEC, true>(a, own, rows, frag, ring, c0, n_end);
    else
        lora_expand_rows<KT, VEC, false>(a, own, rows, frag, ring, c0, n_end);
}

// Many rows: grid (blocks of 16 RB rows, column ranges, projections):
// neighbours share B.  The ring holds base and the first adapter's B; those of
// a block's further adapters are few and loaded in place.
template <int KT, int RB, bool VEC>
__global__ void __launch_bounds__(kLoraThreads, LoraRing<KT, RB>::kCtas) k_lora_expand(const LoraArgs a)
{
    using S = LoraRing<KT, RB>;
    constexpr int LD = KT * 16 + 4;  // floats per row of t in shared memory
    extern __shared__ __align__(128) uint8_t ring_mem[];
    __shared__ __align__(16) float ts[RB * 16 * LD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const unsigned ring = (unsigned)__cvta_generic_to_shared(ring_mem) + warp * S::kStages * S::kStage;
    pdl_launch_dependents();
    const int target = blockIdx.z;
    const int64_t m0 = (int64_t)blockIdx.x * (16 * RB);
    const int id = lora_id(a, lane < 16 * RB ? m0 + lane : a.M);
    const int my_rank = lora_rank(a, id);
    const unsigned distinct = lora_distinct(id, lane);
    const int first = (__ffs(distinct) - 1) & 31;
    const int id0 = __shfl_sync(0xffffffffu, id, first), rank0 = __shfl_sync(0xffffffffu, my_rank, first);
    const float *base = a.base[target];
    float *y = a.y[target];
    LoraPieces<KT, RB> pieces;
    pieces.set(rank0, a.rank, lane);
    const uint16_t *b = a.b[target] + lane * 8, *b0 = b + (int64_t)max(id0, 0) * a.N * a.rank;
    const int n_end = min(a.N, (int)(blockIdx.y + 1) * a.cols);
    constexpr int kStep = kLoraWarps * 16;
    int n0 = blockIdx.y * a.cols + warp * 16, ahead = n0, put = 0, get = 0;
    auto issue = [&]() {
        if (ahead < n_end) {
            const unsigned st = ring + put * S::kStage;
            if (VEC && ahead + 4 * t < a.N)
#pragma unroll
                for (int q = 0; q < 2 * RB; ++q) {
                    const int64_t r = m0 + q * 8 + g;
                    if (r < a.M) lora_cp16(st + (q * 8 + g) * 64 + t * 16, base + r * a.N + ahead + 4 * t);
                }
            if (distinct) pieces.copy(st + S::kBase, b0 + (int64_t)ahead * a.rank, a.N - ahead);
            ahead += kStep;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        put = put + 1 == S::kStages ? 0 : put + 1;
    };
#pragma unroll
    for (int s = 0; s < S::kStages - 1; ++s) issue();
    pdl_wait_primary();
    if (distinct)
        for (int e = threadIdx.x; e < RB * 16 * KT * 4; e += kLoraThreads) {
            const int row = e / (KT * 4), r = e % (KT * 4) * 4, i = lora_id(a, m0 + row);
            *reinterpret_cast<float4 *>(ts + row * LD + r) = lora_t4(a, target, m0 + row, i, lora_rank(a, i), r);
        }
    __syncthreads();
    uint32_t f[RB][KT][3][4];
    int row_id[RB][2];
#pragma unroll
    for (int q = 0; q < RB; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            row_id[q][h] = __shfl_sync(0xffffffffu, id, q * 16 + h * 8 + g);
#pragma unroll
            for (int k = 0; k < KT; ++k) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (distinct) v = *reinterpret_cast<const float4 *>(ts + (q * 16 + h * 8 + g) * LD + k * 16 + 4 * t);
                lora_split(v, f[q][k], h);
            }
        }
    for (; n0 < n_end; n0 += kStep) {
        asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 2) : "memory");
        __syncwarp();
        issue();  // into the stage read last
        const unsigned st = ring + get * S::kStage;
        get = get + 1 == S::kStages ? 0 : get + 1;
        const int n = n0 + 4 * t;
        float4 o[RB][2];
#pragma unroll
        for (int q = 0; q < RB; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t r = m0 + q * 16 + h * 8 + g;
                if (VEC)
                    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                                 : "=f"(o[q][h].x), "=f"(o[q][h].y), "=f"(o[q][h].z), "=f"(o[q][h].w)
                                 : "r"(st + (q * 16 + h * 8 + g) * 64 + t * 16));
                else
                    o[q][h] = lora_load4(base + min(r, (int64_t)a.M - 1) * a.N + n, r < a.M ? a.N - n : 0);
            }
        int i = id0, rank = rank0;
        for (unsigned todo = distinct; todo;) {
            float acc[RB][2][4];
            lora_mul<KT, RB, 3>(f, st + S::kBase, rank, g, t, acc);
#pragma unroll
            for (int q = 0; q < RB; ++q)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (row_id[q][h] == i) lora_acc(o[q][h], acc[q], h);
            todo &= todo - 1;
            if (todo) {  // the next adapter's B takes the first one's place in the stage
                const int src = __ffs(todo) - 1;
                i = __shfl_sync(0xffffffffu, id, src);
                rank = __shfl_sync(0xffffffffu, my_rank, src);
                __syncwarp();
                LoraPieces<KT, RB> its;
                its.set(rank, a.rank, lane);
                its.copy(st + S::kBase, b + ((int64_t)i * a.N + n0) * a.rank, a.N - n0);
                asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
                __syncwarp();
            }
        }
#pragma unroll
        for (int q = 0; q < RB; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t r = m0 + q * 16 + h * 8 + g;
                if (r < a.M) lora_store4<VEC>(y + r * a.N + n, a.N - n, o[q][h]);
            }
        __syncwarp();  // every lane has read the stage
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

struct LoraPlan {
    bool few;
    int rb, slices, kslice;
};

// few: rows gathered by adapter, where an adapter of the pool has fewer than 16 of
// them on average (4096 x 4096, rank 16, gathered against in blocks: 256 rows of
// 32 adapters in any order 14.0 and 57.0 us, 16 rows of 4 5.4 and 8.9; 64 rows of 4
// adapters in any order 9.9 and 10.0, one adapter after the other 9.9 and 6.1; 256 rows
// of 4 14.9 and 11.7).  The rule sees the pool's size and not the ids, which are on the
// device: 200 rows of 12 adapters in any order go in blocks and take 29 us, where
// 13 adapters' are gathered and take 12.9; and beyond 256 rows all go in blocks, 512 rows of
// 32 adapters 11.7 us in runs and 73 in any order.
// rb: rows per block / 16; 32 rows (each weight loaded for twice the rows) where
// their fragments leave registers for two CTAs per SM (4096 rows of rank 32, 11008
// columns: 93.7 us, with 16 rows 112).  Slices of K: about two
// CTAs per SM in the first launch, of at least 64 k for each warp; a decode
// batch counts as M / 2 adapters (61 rows, rank 64, K = 5120 in 4 slices: 42.9 us for
// both launches; in 2 51, 3 45.1, 6 46.8, 8 46.0).
static LoraPlan lora_plan(bool few, int R, int M, int K, int rank)
{
    LoraPlan p;
    p.few = few;
    p.rb = rank <= 32 ? 2 : 1;
    const int64_t groups = p.few ? (M + 1) / 2 : (M + 16 * p.rb - 1) / (16 * p.rb), want = 2 * 148;
    const int most = std::max(1, K / (64 * kLoraWarps));
    p.slices = (int)std::min<int64_t>(std::max<int64_t>(1, want / (groups * R)), std::min(most, kLoraMaxSlices));
    p.kslice = ((K + p.slices - 1) / p.slices + 31) / 32 * 32;
    p.slices = (K + p.kslice - 1) / p.kslice;
    return p;
}

size_t lora_workspace_bytes(int R, int M, int K, int rank)
{
    int slices = lora_plan(false, R, M, K, rank).slices;  // whatever the pool's size
    if (M <= kLoraFewRows) slices = std::max(slices, lora_plan(true, R, M, K, rank).slices);
    return align256((size_t)R * slices * M * rank * sizeof(float));
}

int lora_max_group() { return kLoraMaxGroup; }

template <typename... KArgs>
static cudaError_t lora_start(void (*kern)(KArgs...), dim3 grid, int smem, const LoraArgs &g, cudaStream_t st)
{
    if (smem > 32 * 1024) {  // with the static arrays beside it, beyond the default 48 KB
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(kern, grid, dim3(kLoraThreads), smem, st, g);
}

template <int KT>  // rank / 16, rounded up to 1, 2, 4 or 8
static cudaError_t lora_run(const LoraPlan &p, dim3 gs, dim3 ge, const LoraArgs &g, cudaStream_t st)
{
    constexpr int NT = 2 * KT, RB = KT <= 2 ? 2 : 1;
    cudaError_t e = p.few ? lora_start(k_lora_shrink_few<NT>, gs, LoraShrink<NT, 1>::kBytes, g, st)
                          : lora_start(k_lora_shrink<NT, RB>, gs, LoraShrink<NT, RB>::kBytes, g, st);
    if (e != cudaSuccess) return e;
    if (g.N % 4 == 0)
        return p.few ? lora_start(k_lora_expand_few<KT, true>, ge, LoraRing<KT, 1>::kBytes, g, st)
                     : lora_start(k_lora_expand<KT, RB, true>, ge, LoraRing<KT, RB>::kBytes, g, st);
    return p.few ? lora_start(k_lora_expand_few<KT, false>, ge, LoraRing<KT, 1>::kBytes, g, st)
                 : lora_start(k_lora_expand<KT, RB, false>, ge, LoraRing<KT, RB>::kBytes, g, st);
}

lowbit_status lora_launch(const uint16_t *x, const int32_t *ids, const uint16_t *const *a, const uint16_t *const *b,
                          const int32_t *ranks, const float *scales, const float *const *base, float *const *y, int R,
                          int M, int N, int K, int rank, int L, void *workspace, cudaStream_t st)
{
    const LoraPlan p = lora_plan(M <= kLoraFewRows && M < 16 * (int64_t)L, R, M, K, rank);
    LoraArgs g = {};
    g.x = x; g.ids = ids; g.ranks = ranks; g.scales = scales;
    for (int r = 0; r < R; ++r) {
        g.a[r] = a[r]; g.b[r] = b[r]; g.base[r] = base[r]; g.y[r] = y[r];
    }
    g.t = static_cast<float *>(workspace);
    g.M = M; g.N = N; g.K = K; g.rank = rank; g.L = L;
    g.slices = p.slices; g.kslice = p.kslice;
    const int64_t groups = p.few ? M : ((int64_t)M + 16 * p.rb - 1) / (16 * p.rb);
    // Columns per CTA of the second launch, in rounds of the CTA's warps: as few as
    // fill the SMs at once (a decode batch counts as M adapters: 10.3 us for 16 rows of
    // three 5120 x 5120 projections against 10.9 as 3 / 4 M and 12.3 as M / 2), at
    // most 20 for few rows and 8 for many.  A CTA has 3 us to go before its first
    // round, but those with more adapters or a higher rank take longer and the SMs
    // wait for the last of them: 61 rows, rank 64, 17408 columns 47.2 us with 8,
    // 44.4 with 12, 42.9 with 20, 47.3 with 27; 4096 rows, rank 32, 11008 columns 93.6
    // us with 8, 98.3 with 12, 102 with 17.
    const int64_t rounds = (N + kLoraWarps * 16 - 1) / (kLoraWarps * 16), slots = (rank <= 16 && p.few ? 4 : rank <= 64 ? 2 : 1) * 148;
    const int64_t each = (rounds * groups * R + slots - 1) / slots;
    g.cols = (int)std::min<int64_t>(std::max<int64_t>(each, 1), p.few ? 20 : 8) * kLoraWarps * 16;
    const dim3 gs((unsigned)(groups * p.slices), R, p.few ? 1 : 2), ge((unsigned)groups, (unsigned)((N + g.cols - 1) / g.cols), R);
    const cudaError_t e = rank <= 16   ? lora_run<1>(p, gs, ge, g, st)
                          : rank <= 32 ? lora_run<2>(p, gs, ge, g, st)
                          : rank <= 64 ? lora_run<4>(p, gs, ge, g, st)
                                       : lora_run<8>(p, gs, ge, g, st);
    return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

}  // namespace lowbit
