// lora.cu -- low-rank adapters of many requests beside a shared projection:
//     t[m] = A_i x[m],  y[m] = base[m] + s_i B_i t[m],  i = ids[m].
//
// Two launches.  The first forms t (fp32) for 16-row blocks and slices of K:
// a warp takes the distinct adapters of its block one after the other, and
// each lane's 16-byte loads of x and A are mma.sync m16n8k16 fragments as they
// lie in memory (the k order inside a fragment is free as long as both operands
// share it).  Only the rows of the adapter at hand are stored, so what another
// adapter holds (infinities among it) cannot reach them.  The second adds s_i B_i t to base: t is
// summed over the slices in order, scaled and split into three bf16 numbers,
// which carry its 24 bits (two would leave an error of 2^-18 of t beside fp32
// outputs); a warp holds the split of its 16 rows in registers and walks
// over columns, 16 at a time, with B's 16-byte loads as fragments again.
//
// Rows stay in the caller's order: nothing is sorted, and a block costs one
// pass over the weights of each adapter in it.  For decode batches that is the
// bytes that have to be read anyway; prompts have one or two adapters a block.
// Bound by the adapters' bytes for decode, by base and y (8 bytes an output)
// for prompts.
#include <algorithm>

#include "common.cuh"

namespace lowbit {

constexpr int kLoraMaxGroup = 16;
constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;
constexpr int kLoraMaxSlices = 64;

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
    int parts;           // warps that share a block's adapters
    int cols;            // columns per CTA of the second launch
};

__device__ __forceinline__ void lora_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Of a block's 16 ids (lane r < 16 holds row r's, -1 for none): the lanes that
// hold the first row of each distinct adapter.
__device__ __forceinline__ unsigned lora_distinct(int id, int lane)
{
    const unsigned same = __match_any_sync(0xffffffffu, id);
    const bool first = lane < 16 && id >= 0 && (same & ((1u << lane) - 1) & 0xFFFFu) == 0;
    return __ballot_sync(0xffffffffu, first);
}

__device__ __forceinline__ int lora_id(const LoraArgs &a, int64_t m)
{
    if (m >= a.M) return -1;
    const int id = __ldg(a.ids + m);
    return (unsigned)id < (unsigned)a.L ? id : -1;
}

__device__ __forceinline__ int lora_rank(const LoraArgs &a, int id)
{
    return a.ranks ? min(max(__ldg(a.ranks + id), 0), a.rank) : a.rank;
}

// One warp: (row block, slice of K, projection, share of the block's adapters).
template <int NT>  // rank / 8, rounded up to 2, 4, 8 or 16
__global__ void __launch_bounds__(kLoraThreads) k_lora_shrink(const LoraArgs a)
{
    pdl_wait_primary();
    pdl_launch_dependents();  // after the wait: the next launch may then read what came before this one
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t task = (int64_t)blockIdx.x * kLoraWarps + (threadIdx.x >> 5);
    const int part = (int)(task % a.parts), slice = (int)(task / a.parts % a.slices);
    const int64_t block = task / ((int64_t)a.parts * a.slices);
    if (block * 16 >= a.M) return;
    const int target = blockIdx.y;
    const int id = lora_id(a, lane < 16 ? block * 16 + lane : a.M);
    unsigned todo = lora_distinct(id, lane);
    const int id_lo = __shfl_sync(0xffffffffu, id, g), id_hi = __shfl_sync(0xffffffffu, id, g + 8);
    const int k0 = slice * a.kslice, k1 = min(a.K, k0 + a.kslice);
    const int64_t m_lo = block * 16 + g, m_hi = m_lo + 8;
    const uint16_t *x_lo = a.x + min(m_lo, (int64_t)a.M - 1) * a.K, *x_hi = a.x + min(m_hi, (int64_t)a.M - 1) * a.K;
    float *tp = a.t + ((int64_t)target * a.slices + slice) * a.M * a.rank;
    for (int nth = 0; todo; ++nth) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        if (nth % a.parts != part) continue;
        const int i = __shfl_sync(0xffffffffu, id, src);
        const int rank = lora_rank(a, i);
        const bool lo = id_lo == i, hi = id_hi == i;
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[n][c] = 0.f;
        const uint16_t *w = a.a[target] + ((int64_t)i * a.rank + g) * a.K;
        const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 2
        for (int k = k0 + t * 8; k < k1; k += 32) {
            const uint4 xl = lo ? __ldg(reinterpret_cast<const uint4 *>(x_lo + k)) : zero;
            const uint4 xh = hi ? __ldg(reinterpret_cast<const uint4 *>(x_hi + k)) : zero;
            uint4 wv[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n)
                wv[n] = n * 8 + g < rank ? __ldg(reinterpret_cast<const uint4 *>(w + (int64_t)n * 8 * a.K + k)) : zero;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                lora_mma(acc[n], xl.x, xh.x, xl.y, xh.y, wv[n].x, wv[n].y);
                lora_mma(acc[n], xl.z, xh.z, xl.w, xh.w, wv[n].z, wv[n].w);
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = n * 8 + 2 * t;
            if (r < a.rank) {
                if (lo) *reinterpret_cast<float2 *>(tp + m_lo * a.rank + r) = make_float2(acc[n][0], acc[n][1]);
                if (hi) *reinterpret_cast<float2 *>(tp + m_hi * a.rank + r) = make_float2(acc[n][2], acc[n][3]);
            }
        }
    }
}

// Grid: (16-row blocks, column ranges, projections): neighbours share B.
template <int KT, bool VEC>  // KT: rank / 16, rounded up to 1, 2, 4 or 8; VEC: rows of y are 16-byte aligned
__global__ void __launch_bounds__(kLoraThreads) k_lora_expand(const LoraArgs a)
{
    constexpr int LD = KT * 16 + 4;  // floats per row of t in shared memory
    __shared__ __align__(16) float ts[16 * LD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    pdl_launch_dependents();
    pdl_wait_primary();
    const int target = blockIdx.z;
    const int64_t m0 = (int64_t)blockIdx.x * 16;
    const int id = lora_id(a, lane < 16 ? m0 + lane : a.M);
    const unsigned distinct = lora_distinct(id, lane);
    const int id_lo = __shfl_sync(0xffffffffu, id, g), id_hi = __shfl_sync(0xffffffffu, id, g + 8);
    // t of the block's rows, slices in order, scaled; 0 past an adapter's rank
    if (distinct)
        for (int e = threadIdx.x; e < 16 * KT * 4; e += kLoraThreads) {
            const int row = e / (KT * 4), r = e % (KT * 4) * 4;
            const int i = lora_id(a, m0 + row);
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i >= 0 && r < a.rank) {
                const float *p = a.t + ((int64_t)target * a.slices * a.M + m0 + row) * a.rank + r;
#pragma unroll 4
                for (int q = 0; q < a.slices; ++q) {
                    const float4 v = *reinterpret_cast<const float4 *>(p + (int64_t)q * a.M * a.rank);
                    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
                }
                const float f = a.scales ? __ldg(a.scales + i) : 1.f;
                const int rank = lora_rank(a, i) - r;
                s.x = rank > 0 ? s.x * f : 0.f;
                s.y = rank > 1 ? s.y * f : 0.f;
                s.z = rank > 2 ? s.z * f : 0.f;
                s.w = rank > 3 ? s.w * f : 0.f;
            }
            *reinterpret_cast<float4 *>(ts + row * LD + r) = s;
        }
    __syncthreads();
    // three bf16 numbers per value: fragment words {row g, g + 8} x {4 t + 0..1, 2..3}
    uint32_t f[KT][3][4];
    if (distinct) {
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                const float4 v = *reinterpret_cast<const float4 *>(ts + (g + 8 * hi) * LD + k * 16 + 4 * t);
                float p[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int s = 0; s < 3; ++s)
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        uint32_t u;
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(p[2 * w + 1]), "f"(p[2 * w]));
                        f[k][s][w * 2 + hi] = u;
                        p[2 * w] -= __uint_as_float(u << 16);
                        p[2 * w + 1] -= __uint_as_float(u & 0xFFFF0000u);
                    }
            }
    }
    const float *base = a.base[target];
    float *y = a.y[target];
    const int64_t r_lo = m0 + g, r_hi = r_lo + 8;
    const int n_end = min(a.N, (int)(blockIdx.y + 1) * a.cols);
    for (int n0 = blockIdx.y * a.cols + warp * 16; n0 < n_end; n0 += kLoraWarps * 16) {
        // column q of block j is n0 + 4 (q / 2) + 2 j + q % 2, so that a thread
        // holds four consecutive columns, n0 + 4 t .., of its two rows
        const int n = n0 + 4 * t;
        float4 o_lo = make_float4(0.f, 0.f, 0.f, 0.f), o_hi = o_lo;
        if (VEC) {
            if (n < a.N) {
                if (r_lo < a.M) o_lo = *reinterpret_cast<const float4 *>(base + r_lo * a.N + n);
                if (r_hi < a.M) o_hi = *reinterpret_cast<const float4 *>(base + r_hi * a.N + n);
            }
        } else {
            float *pl = &o_lo.x, *ph = &o_hi.x;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < a.N) {
                    if (r_lo < a.M) pl[i] = base[r_lo * a.N + n + i];
                    if (r_hi < a.M) ph[i] = base[r_hi * a.N + n + i];
                }
        }
        for (unsigned todo = distinct; todo; todo &= todo - 1) {
            const int i = __shfl_sync(0xffffffffu, id, __ffs(todo) - 1);
            const int rank = lora_rank(a, i);
            const uint16_t *w = a.b[target] + (int64_t)i * a.N * a.rank + 4 * t;
            float acc[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[j][c] = 0.f;
                const int col = n0 + 4 * (g >> 1) + 2 * j + (g & 1);
                uint2 bw[KT];
#pragma unroll
                for (int k = 0; k < KT; ++k) {
                    // entries from the adapter's rank on are cleared: they may hold anything
                    const int left = rank - (k * 16 + 4 * t);
                    bw[k] = make_uint2(0u, 0u);
                    if (left > 0 && col < a.N)
                        bw[k] = __ldg(reinterpret_cast<const uint2 *>(w + (int64_t)col * a.rank + k * 16));
                    if (left < 4) {
                        if (left < 2) bw[k].y = 0; else if (left < 4) bw[k].y &= left < 3 ? 0u : 0xFFFFu;
                        if (left == 1) bw[k].x &= 0xFFFFu;
                    }
                }
#pragma unroll
                for (int k = 0; k < KT; ++k)
#pragma unroll
                    for (int s = 0; s < 3; ++s)
                        lora_mma(acc[j], f[k][s][0], f[k][s][1], f[k][s][2], f[k][s][3], bw[k].x, bw[k].y);
            }
            if (id_lo == i) {
                o_lo.x += acc[0][0]; o_lo.y += acc[0][1]; o_lo.z += acc[1][0]; o_lo.w += acc[1][1];
            }
            if (id_hi == i) {
                o_hi.x += acc[0][2]; o_hi.y += acc[0][3]; o_hi.z += acc[1][2]; o_hi.w += acc[1][3];
            }
        }
        if (VEC) {
            if (n < a.N) {
                if (r_lo < a.M) *reinterpret_cast<float4 *>(y + r_lo * a.N + n) = o_lo;
                if (r_hi < a.M) *reinterpret_cast<float4 *>(y + r_hi * a.N + n) = o_hi;
            }
        } else {
            const float *pl = &o_lo.x, *ph = &o_hi.x;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < a.N) {
                    if (r_lo < a.M) y[r_lo * a.N + n + i] = pl[i];
                    if (r_hi < a.M) y[r_hi * a.N + n + i] = ph[i];
                }
        }
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

struct LoraPlan {
    int slices, kslice, parts;
};

// Warps of the first launch: enough to fill the GPU (about 16 an SM), first by
// sharing a block's adapters, then by slices of K, of at least 128 k each.
static LoraPlan lora_plan(int R, int M, int K)
{
    const int blocks = (M + 15) / 16;
    LoraPlan p;
    const int64_t want = 148 * 16;
    p.parts = (int)std::min<int64_t>(std::min(16, M), std::max<int64_t>(1, want / ((int64_t)blocks * R)));
    const int64_t s = std::max<int64_t>(1, want / ((int64_t)blocks * R * p.parts));
    const int most = std::min(kLoraMaxSlices, (K + 127) / 128);
    p.slices = (int)std::min<int64_t>(s, most);
    p.kslice = ((K + p.slices - 1) / p.slices + 31) / 32 * 32;
    p.slices = (K + p.kslice - 1) / p.kslice;
    return p;
}

size_t lora_workspace_bytes(int R, int M, int K, int rank)
{
    return align256((size_t)R * lora_plan(R, M, K).slices * M * rank * sizeof(float));
}

int lora_max_group() { return kLoraMaxGroup; }

lowbit_status lora_launch(const uint16_t *x, const int32_t *ids, const uint16_t *const *a, const uint16_t *const *b,
                          const int32_t *ranks, const float *scales, const float *const *base, float *const *y, int R,
                          int M, int N, int K, int rank, int L, void *workspace, cudaStream_t st)
{
    const LoraPlan p = lora_plan(R, M, K);
    LoraArgs g = {};
    g.x = x; g.ids = ids; g.ranks = ranks; g.scales = scales;
    for (int r = 0; r < R; ++r) {
        g.a[r] = a[r]; g.b[r] = b[r]; g.base[r] = base[r]; g.y[r] = y[r];
    }
    g.t = static_cast<float *>(workspace);
    g.M = M; g.N = N; g.K = K; g.rank = rank; g.L = L;
    g.slices = p.slices; g.kslice = p.kslice; g.parts = p.parts;
    const int64_t blocks = (M + 15) / 16;
    const int64_t tasks = blocks * p.slices * p.parts;
    void (*shrink)(const LoraArgs) = rank <= 16 ? k_lora_shrink<2> : rank <= 32 ? k_lora_shrink<4>
                                     : rank <= 64 ? k_lora_shrink<8> : k_lora_shrink<16>;
    cudaError_t e = launch_pdl(shrink, dim3((unsigned)((tasks + kLoraWarps - 1) / kLoraWarps), R), dim3(kLoraThreads),
                               0, st, g);
    if (e != cudaSuccess) return LOWBIT_ERR_CUDA;
    // columns per CTA: whole rounds of the CTA's warps, as many as leave about
    // four CTAs per SM
    const int round = kLoraWarps * 16;
    const int64_t ranges = std::max<int64_t>(1, 4 * 148 / (blocks * R));
    g.cols = (int)((((int64_t)N + ranges - 1) / ranges + round - 1) / round * round);
    const bool vec = N % 4 == 0;
    void (*expand)(const LoraArgs) =
        rank <= 16   ? (vec ? k_lora_expand<1, true> : k_lora_expand<1, false>)
        : rank <= 32 ? (vec ? k_lora_expand<2, true> : k_lora_expand<2, false>)
        : rank <= 64 ? (vec ? k_lora_expand<4, true> : k_lora_expand<4, false>)
                     : (vec ? k_lora_expand<8, true> : k_lora_expand<8, false>);
    e = launch_pdl(expand, dim3((unsigned)blocks, (unsigned)((N + g.cols - 1) / g.cols), R), dim3(kLoraThreads), 0, st, g);
    return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

}  // namespace lowbit
