// rope.cu -- rotary positions on query and key heads, one launch for both.
//
// (a, b) -> magnitude (a cos w - b sin w, b cos w + a sin w) for the pairs of
// the first rot entries of a head, w = position * phase in 2^-64 turns.  The
// product wraps in 64-bit integers, which is the reduction mod one turn,
// exactly: a 32-bit float product of a position near 10^6 and a frequency near
// 1 would be off by up to 0.03 rad.  Its top 32 bits become a float in
// [-1, 1) half turns (relative rounding 2^-24) for sincospif.
//
// Bound by HBM (each value read and written once) for many rows and by
// latency for few.  A CTA takes one row and a range of its heads: the row's
// sines are computed once into shared memory and shared by all its heads.
#include <cmath>

#include "common.cuh"

namespace lowbit {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxDim = 1024;

struct RopeArgs {
    const void *in[2];
    void *out[2];
    int64_t in_stride[2], out_stride[2];
    int heads[2];
    const int32_t *positions;
    const uint64_t *phases;
    int D, rot, heads_per_cta;
    float magnitude;
};

__device__ __forceinline__ void rope_store8(float *p, const float (&v)[8])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void rope_store8(uint16_t *p, const float (&v)[8])
{
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]), bf16x2_rn(v[4], v[5]), bf16x2_rn(v[6], v[7]));
}
__device__ __forceinline__ float rope_load1(const float *p) { return *p; }
__device__ __forceinline__ float rope_load1(const uint16_t *p) { return bf16_bits_to_float(*p); }
__device__ __forceinline__ void rope_store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void rope_store1(uint16_t *p, float v) { *p = (uint16_t)bf16x2_rn(v, 0.f); }

// Eight values as they are stored, loaded now and looked at later.
template <typename T>
struct RopeRaw;
template <>
struct RopeRaw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};
template <>
struct RopeRaw<uint16_t> {
    uint4 u;
    __device__ __forceinline__ void load(const uint16_t *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};

// The row's sines into shared memory.
__device__ __forceinline__ void rope_turns(const RopeArgs &a, int64_t m, float2 *turn)
{
    const int64_t pos = a.positions[m];
    for (int j = threadIdx.x; j < a.rot / 2; j += kRopeThreads) {
        const int32_t top = (int32_t)(((uint64_t)pos * a.phases[j]) >> 32);
        float s, c;
        sincospif((float)top * 0x1p-31f, &s, &c);
        turn[j] = make_float2(c * a.magnitude, s * a.magnitude);
    }
}

__device__ __forceinline__ void rope_turn(float &a, float &b, float c, float s)
{
    const float r = a * c - b * s;
    b = b * c + a * s;
    a = r;
}

// A piece's head: source and destination.
template <typename TI, typename TO>
__device__ __forceinline__ void rope_head(const RopeArgs &a, int64_t m, int h, const TI *&src, TO *&dst)
{
    const int which = h >= a.heads[0];
    if (which) h -= a.heads[0];
    src = static_cast<const TI *>(which ? a.in[1] : a.in[0]) + m * (which ? a.in_stride[1] : a.in_stride[0]) + (int64_t)h * a.D;
    dst = static_cast<TO *>(which ? a.out[1] : a.out[0]) + m * (which ? a.out_stride[1] : a.out_stride[0]) + (int64_t)h * a.D;
}

// rot is a multiple of 16 (half layout) or 8 (interleaved): 16-byte pieces of
// pairs.  A thread's first pieces are under way before the sines are computed
// (loaded after them, 8191 rows of 40 heads took 43 us in place of 38); 48
// registers, five CTAs an SM, and three pieces (31.5 us, 5.3 TB/s) do better than
// 64, four CTAs and four (36.3), or 40, six CTAs and two (32.1).
template <typename TI, typename TO, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 5) k_rope(const RopeArgs a)
{
    constexpr int U = (INTER ? 2 : 1) + (sizeof(TI) == 2 ? 1 : 0);  // pieces under way
    __shared__ __align__(16) float2 turn[kRopeMaxDim / 2];  // {cos, sin} * magnitude
    pdl_launch_dependents();
    pdl_wait_primary();
    const int64_t m = blockIdx.x;
    const int half = a.rot / 2, h0 = blockIdx.y * a.heads_per_cta;
    const int nh = min(a.heads_per_cta, a.heads[0] + a.heads[1] - h0);
    // pieces of a head: turned ones first (4 interleaved pairs, or 8 pairs of two
    // 8-value runs), then the copied rest, 8 or 16 values each
    const int turned = INTER ? a.rot / 8 : a.rot / 16, rest = a.D - a.rot;
    const unsigned pieces = turned + (INTER ? rest / 8 : (rest + 8) / 16), total = nh * pieces;
    bool first = true;
    // piece and head of this thread's next piece, advanced without divisions
    unsigned head = threadIdx.x / pieces, c = threadIdx.x % pieces;
    const unsigned dh = kRopeThreads / pieces, dc = kRopeThreads % pieces;
    for (unsigned base = threadIdx.x; first || base < total; base += U * kRopeThreads) {
        RopeRaw<TI> u[U], v[U];
        const TI *src[U];
        TO *dst[U];
        int at[U][2];  // offsets of the piece's two runs (the second for the half layout, -1: none)
        int pair[U];   // its first pair, -1: copied
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const unsigned i = base + k * kRopeThreads;
            pair[k] = -2;
            if (i >= total) continue;
            rope_head(a, m, h0 + (int)head, src[k], dst[k]);
            const int p = (int)c;
            const bool turn_it = p < turned;
            pair[k] = turn_it ? p * (INTER ? 4 : 8) : -1;
            if (INTER) {
                at[k][0] = p * 8;  // rot is 8 turned ones
                at[k][1] = -1;
            } else {
                at[k][0] = turn_it ? p * 8 : a.rot + (p - turned) * 16;
                at[k][1] = turn_it ? half + p * 8 : at[k][0] + 8 < a.D ? at[k][0] + 8 : -1;
            }
            head += dh;
            c += dc;
            if (c >= pieces) {
                c -= pieces;
                ++head;
            }
            u[k].load(src[k] + at[k][0]);
            if (!INTER && at[k][1] >= 0) v[k].load(src[k] + at[k][1]);
        }
        if (first) {
            rope_turns(a, m, turn);
            __syncthreads();
            first = false;
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (pair[k] == -2) continue;
            float x[8], y[8];
            u[k].get(x);
            if (INTER) {
                if (pair[k] >= 0)
#pragma unroll
                    for (int p = 0; p < 4; p += 2) {
                        const float4 w = *reinterpret_cast<const float4 *>(turn + pair[k] + p);
                        rope_turn(x[2 * p], x[2 * p + 1], w.x, w.y);
                        rope_turn(x[2 * p + 2], x[2 * p + 3], w.z, w.w);
                    }
            } else if (at[k][1] >= 0) {
                v[k].get(y);
                if (pair[k] >= 0)
#pragma unroll
                    for (int p = 0; p < 8; p += 2) {
                        const float4 w = *reinterpret_cast<const float4 *>(turn + pair[k] + p);
                        rope_turn(x[p], y[p], w.x, w.y);
                        rope_turn(x[p + 1], y[p + 1], w.z, w.w);
                    }
                rope_store8(dst[k] + at[k][1], y);
            }
            rope_store8(dst[k] + at[k][0], x);
        }
    }
}

// Other widths: one pair or copied value at a time (8191 rows of 40 heads of 128, 40
// entries turned in the half layout: 133 us; in the interleaved one, which the pieces
// above fit, 31.7).
template <typename TI, typename TO, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) k_rope_any(const RopeArgs a)
{
    __shared__ float2 turn[kRopeMaxDim / 2];
    pdl_launch_dependents();
    pdl_wait_primary();
    const int64_t m = blockIdx.x;
    rope_turns(a, m, turn);
    __syncthreads();
    const int half = a.rot / 2, h0 = blockIdx.y * a.heads_per_cta;
    const int nh = min(a.heads_per_cta, a.heads[0] + a.heads[1] - h0);
    const int pieces = half + a.D - a.rot;
    for (int i = threadIdx.x; i < nh * pieces; i += kRopeThreads) {
        const TI *src;
        TO *dst;
        rope_head(a, m, h0 + i / pieces, src, dst);
        const int c = i % pieces;
        if (c >= half) {
            rope_store1(dst + a.rot + c - half, rope_load1(src + a.rot + c - half));
        } else {
            const int ia = INTER ? 2 * c : c, ib = INTER ? 2 * c + 1 : c + half;
            const float u = rope_load1(src + ia), v = rope_load1(src + ib);
            const float2 w = turn[c];
            rope_store1(dst + ia, u * w.x - v * w.y);
            rope_store1(dst + ib, v * w.x + u * w.y);
        }
    }
}

template <typename TI, typename TO>
static void (*rope_kernel(bool inter, bool vec))(const RopeArgs)
{
    if (inter) return vec ? k_rope<TI, TO, true> : k_rope_any<TI, TO, true>;
    return vec ? k_rope<TI, TO, false> : k_rope_any<TI, TO, false>;
}

lowbit_status rope_launch(const void *q, int64_t q_stride, void *q_out, int64_t q_out_stride, int q_heads,
                          const void *k, int64_t k_stride, void *k_out, int64_t k_out_stride, int kv_heads,
                          lowbit_dtype in_type, lowbit_dtype out_type, const int32_t *positions,
                          const int64_t *phases, int M, int D, int rot, int interleaved, float magnitude,
                          cudaStream_t st)
{
    RopeArgs a;
    a.in[0] = q; a.in[1] = k;
    a.out[0] = q_out; a.out[1] = k_out;
    a.in_stride[0] = q_stride; a.in_stride[1] = k_stride;
    a.out_stride[0] = q_out_stride; a.out_stride[1] = k_out_stride;
    a.heads[0] = q_heads; a.heads[1] = kv_heads;
    a.positions = positions;
    a.phases = reinterpret_cast<const uint64_t *>(phases);
    a.D = D; a.rot = rot; a.magnitude = magnitude;
    const bool vec = rot % (interleaved ? 8 : 16) == 0;
    // few rows: cut a row's heads over CTAs until the grid has about two CTAs
    // per SM, but not below one piece per thread
    const int heads = q_heads + kv_heads;
    const int per_head = (vec ? D / (interleaved ? 8 : 16) : D / 2);
    int hpc = heads;
    while (hpc > 1 && (int64_t)M * ((heads + hpc - 1) / hpc) < 2 * 148 && (hpc + 1) / 2 * per_head >= kRopeThreads / 2)
        hpc = (hpc + 1) / 2;
    a.heads_per_cta = hpc;
    auto kern = in_type == LOWBIT_F32
                    ? (out_type == LOWBIT_F32 ? rope_kernel<float, float>(interleaved, vec)
                                              : rope_kernel<float, uint16_t>(interleaved, vec))
                    : (out_type == LOWBIT_F32 ? rope_kernel<uint16_t, float>(interleaved, vec)
                                              : rope_kernel<uint16_t, uint16_t>(interleaved, vec));
    const cudaError_t e = launch_pdl(kern, dim3(M, (heads + hpc - 1) / hpc), dim3(kRopeThreads), 0, st, a);
    return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

// The host table: frequencies in double, then 2^-64 turns per position.
void rope_phases_host(lowbit_rope_scaling scaling, int rot, double base, double factor, double trained_length,
                      double slow, double fast, int64_t *phases)
{
    const double kTurn = 6.283185307179586476925286766559;
    if (scaling == LOWBIT_ROPE_BASE && rot > 2) base *= std::pow(factor, rot / (rot - 2.0));
    for (int j = 0; j < rot / 2; ++j) {
        double f = std::pow(base, -2.0 * j / rot);
        if (scaling == LOWBIT_ROPE_LINEAR) f /= factor;
        if (scaling == LOWBIT_ROPE_BANDS) {
            const double u = trained_length * f / kTurn;
            const double c = u <= slow ? 0.0 : u >= fast ? 1.0 : (u - slow) / (fast - slow);
            f = c * f + (1.0 - c) * (f / factor);
        }
        // whole turns per position change nothing
        const double turns = f / kTurn;
        const double part = std::ldexp(turns - std::floor(turns), 64);
        phases[j] = (int64_t)(part >= 0x1p64 ? 0 : (uint64_t)std::rint(part));
    }
}

}  // namespace lowbit
