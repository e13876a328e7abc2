// kv8_cache.cu -- writing and reading back the KV8 cache (int8 codes in pages,
// one fp32 scale per page and head).
//
// Write: for each page and head that gets new tokens
//     s' = max(s of the older tokens, fp32(max |new| / 127)),
//     older codes rint(c s / s'), new codes rint(x / s').
// Both roundings are the exact ones: a quotient near a tie is taken again in
// double, where two 24-bit operands cannot round onto a tie they do not hit
// (their distance from it is at least 2^-26 of a step).  The result is the same
// bits on every run, whatever the launch shape.
//
// Bound by HBM for prompts (each new value read, a byte written) and by latency
// for a decode step.  One group of threads takes one (page, head, k or v): a
// warp where a call brings about a token per sequence, a CTA where it brings
// whole pages.  The values are read twice (the second time from the L1 or L2
// cache): the scale has to be known before the first code.
#include <cfloat>

#include "kv8_common.cuh"

namespace lowbit {

__device__ unsigned g_kv8_fault;  // a length, page or row was out of range

int kv8_fault_flag()
{
    unsigned v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_kv8_fault, sizeof(v)) != cudaSuccess) return -1;
    cudaMemcpyToSymbol(g_kv8_fault, &zero, sizeof(zero));
    return (int)v;
}

constexpr int kKvThreads = 256;

struct Kv8Append {
    Kv8View v;
    int8_t *codes[2];
    float *scales[2];
    const void *x[2];
    int64_t stride[2];
    int bf16[2];
    int items;
};

// Eight consecutive values as floats; NaN becomes 0 and infinities the largest
// float.
__device__ __forceinline__ void kv8_load8(const void *base, int64_t at, int bf16, float (&v)[8])
{
    if (bf16) {
        const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + at);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + at);
        const float4 a = p[0], b = p[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] == v[i] ? fminf(fmaxf(v[i], -FLT_MAX), FLT_MAX) : 0.f;
}

// rint(x / s), exactly; inv = 1 / s, or 0 where s = 0.
__device__ __forceinline__ int kv8_code(float x, float s, float inv)
{
    const float t = x * inv;
    float q = rintf(t);
    // t is off by 1.5 ulp at most: 2e-5 below 127
    if (!(fabsf(t - q) <= 0.4999f)) q = (float)rint((double)x / (double)s);
    return (int)fminf(fmaxf(q, -127.f), 127.f);
}

template <int G>  // threads per (page, head, k or v): 32 or kKvThreads
__global__ void __launch_bounds__(kKvThreads) k_kv8_append(const Kv8Append a)
{
    __shared__ float red[kKvThreads / 32];
    pdl_launch_dependents();
    pdl_wait_primary();
    const Kv8View &v = a.v;
    const int64_t task = (int64_t)blockIdx.x * (kKvThreads / G) + threadIdx.x / G;
    const int t = threadIdx.x % G;
    const int h = (int)(task % v.H), which = (int)(task / v.H % 2);
    const int64_t item = task / (2 * v.H);
    if (item >= a.items) return;  // whole groups leave, so what follows is uniform in a group
    // the item's sequence, and which of its touched pages
    const int b = v.row_start ? kv8_find_seq(v, (int)item, v.P, 2) : (int)item;
    if (b < 0) return;
    const Kv8Seq s = kv8_seq(v, b, &g_kv8_fault);
    const int nth = v.row_start ? (int)(item - (max(__ldg(v.row_start + b), 0) / v.P + 2 * (int64_t)b)) : 0;
    const int p0 = s.len - s.n, first = max(p0, 0);
    const int64_t j64 = (int64_t)first / v.P + nth;
    if (s.n == 0 || j64 * v.P >= s.len) return;
    const int j = (int)j64;
    const int page = kv8_page(v, b, j, &g_kv8_fault);
    if (page < 0) return;
    const int lo = max(first, j * v.P), hi = min(s.len, (j + 1) * v.P);
    const int older = lo - j * v.P, D8 = v.D / 8, n8 = (hi - lo) * D8;
    const int64_t r0 = s.r0 + (lo - p0);
    const void *x = a.x[which];
    const int64_t stride = a.stride[which];
    const int bf16 = a.bf16[which];
    int8_t *codes = a.codes[which] + ((int64_t)page * v.H + h) * v.P * v.D;
    float *scale = a.scales[which] + (int64_t)page * v.H + h;

    float top = 0.f;
    for (int i = t; i < n8; i += G) {
        float f[8];
        kv8_load8(x, (r0 + i / D8) * stride + (int64_t)h * v.D + i % D8 * 8, bf16, f);
#pragma unroll
        for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(f[k]));
    }
    const float was = older ? fmaxf(*scale, 0.f) : 0.f;
    top = warp_max_nonneg(top);
    if constexpr (G > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
        __syncthreads();
        top = red[0];
#pragma unroll
        for (int i = 1; i < kKvThreads / 32; ++i) top = fmaxf(top, red[i]);
    }
    const float now = fmaxf(was, __fdiv_rn(top, 127.f));
    const float inv = now > 0.f ? __frcp_rn(now) : 0.f;
    if (now > was) {
        const double wd = was, nd = now;
        for (int i = t; i < older * v.D / 16; i += G) {
            uint4 u = reinterpret_cast<const uint4 *>(codes)[i];
            uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t o = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c = (int8_t)(w[k] >> (8 * e));
                    o |= ((uint32_t)(int)rint(c * wd / nd) & 0xFFu) << (8 * e);
                }
                w[k] = o;
            }
            reinterpret_cast<uint4 *>(codes)[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    for (int i = t; i < n8; i += G) {
        float f[8];
        kv8_load8(x, (r0 + i / D8) * stride + (int64_t)h * v.D + i % D8 * 8, bf16, f);
        uint32_t o[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k / 4] |= ((uint32_t)kv8_code(f[k], now, inv) & 0xFFu) << (8 * (k % 4));
        reinterpret_cast<uint2 *>(codes)[older * D8 + i] = make_uint2(o[0], o[1]);
    }
    __syncwarp();  // G = 32: every lane has read the old scale
    if (t == 0) *scale = now;
}

lowbit_status kv8_append_launch(const lowbit_kv8_cache &c, const lowbit_kv8_batch &b, const void *k, int64_t k_stride,
                                lowbit_dtype k_type, const void *v, int64_t v_stride, lowbit_dtype v_type,
                                cudaStream_t st)
{
    Kv8Append a;
    a.v = kv8_view(c, b);
    a.codes[0] = c.k; a.codes[1] = c.v;
    a.scales[0] = c.k_scales; a.scales[1] = c.v_scales;
    a.x[0] = k; a.x[1] = v;
    a.stride[0] = k_stride; a.stride[1] = v_stride;
    a.bf16[0] = k_type == LOWBIT_BF16; a.bf16[1] = v_type == LOWBIT_BF16;
    // touched pages, at most: see kv8_find_seq (n rows touch n / P + 2 or fewer)
    const int64_t items = b.row_start ? (int64_t)b.n_rows / c.page_tokens + 2 * (int64_t)b.n_seqs : b.n_seqs;
    if (items >= (int64_t(1) << 31)) return LOWBIT_ERR_UNSUPPORTED_SHAPE;
    a.items = (int)items;
    const int64_t tasks = items * 2 * c.n_heads;
    // one warp per page where a call brings few tokens per sequence
    const bool few = b.n_rows <= 4 * (int64_t)b.n_seqs;
    const int per = few ? kKvThreads / 32 : 1;
    const int64_t grid = (tasks + per - 1) / per;
    if (grid >= (int64_t(1) << 31)) return LOWBIT_ERR_UNSUPPORTED_SHAPE;
    const cudaError_t e = launch_pdl(few ? k_kv8_append<32> : k_kv8_append<kKvThreads>, dim3((unsigned)grid),
                                     dim3(kKvThreads), 0, st, a);
    return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

struct Kv8Read {
    Kv8View v;
    const int8_t *codes[2];
    const float *scales[2];
    void *out[2];
    int bf16;
};

// One thread per 16 values of a row and head; blockIdx.y: keys or values.
__global__ void __launch_bounds__(kKvThreads) k_kv8_read(const Kv8Read a)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    const Kv8View &v = a.v;
    const int which = blockIdx.y;
    void *out = which ? a.out[1] : a.out[0];
    if (!out) return;
    const int8_t *codes = which ? a.codes[1] : a.codes[0];
    const float *scales = which ? a.scales[1] : a.scales[0];
    const int D16 = v.D / 16, per_row = v.H * D16;
    const int64_t i = (int64_t)blockIdx.x * kKvThreads + threadIdx.x;
    if (i >= (int64_t)v.n_rows * per_row) return;
    const int r = (int)(i / per_row), c = (int)(i % per_row), h = c / D16;
    const int b = v.row_start ? kv8_find_seq(v, r, 1, 0) : r;
    if (b < 0) return;
    const Kv8Seq s = kv8_seq(v, b, &g_kv8_fault);
    if (r >= s.r0 + s.n) return;  // behind the last sequence
    const int pos = s.len - s.n + (r - s.r0);
    uint4 u = make_uint4(0, 0, 0, 0);
    float scale = 0.f;
    const int page = pos >= 0 ? kv8_page(v, b, pos / v.P, &g_kv8_fault) : -1;
    if (page >= 0) {
        const int64_t ph = (int64_t)page * v.H + h;
        u = *reinterpret_cast<const uint4 *>(codes + (ph * v.P + pos % v.P) * v.D + c % D16 * 16);
        scale = scales[ph];
    }
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    float f[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) f[k] = (float)(int8_t)(w[k / 4] >> (8 * (k % 4))) * scale;
    const int64_t at = i * 16;
    if (a.bf16) {
        uint32_t o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[k]) : "f"(f[2 * k + 1]), "f"(f[2 * k]));
        uint4 *p = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + at);
        p[0] = make_uint4(o[0], o[1], o[2], o[3]);
        p[1] = make_uint4(o[4], o[5], o[6], o[7]);
    } else {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(out) + at);
#pragma unroll
        for (int k = 0; k < 4; ++k) p[k] = make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
    }
}

lowbit_status kv8_read_launch(const lowbit_kv8_cache &c, const lowbit_kv8_batch &b, void *k_out, void *v_out,
                              lowbit_dtype out_type, cudaStream_t st)
{
    Kv8Read a;
    a.v = kv8_view(c, b);
    a.codes[0] = c.k; a.codes[1] = c.v;
    a.scales[0] = c.k_scales; a.scales[1] = c.v_scales;
    a.out[0] = k_out; a.out[1] = v_out;
    a.bf16 = out_type == LOWBIT_BF16;
    const int64_t threads = (int64_t)b.n_rows * c.n_heads * (c.head_dim / 16);
    const int64_t grid = (threads + kKvThreads - 1) / kKvThreads;
    if (grid >= (int64_t(1) << 31)) return LOWBIT_ERR_UNSUPPORTED_SHAPE;
    const cudaError_t e = launch_pdl(k_kv8_read, dim3((unsigned)grid, 2), dim3(kKvThreads), 0, st, a);
    return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

}  // namespace lowbit
