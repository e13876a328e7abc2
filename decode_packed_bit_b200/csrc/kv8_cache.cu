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
// for a decode step.  One CTA takes one (page, head, k or v).  For prompts it
// has a thread per 32 values, which stay in registers between the maximum and
// the codes (reading them twice took 66 us where this takes 33, 16384 rows of 2 x 8 heads of 128); for a decode
// step 128 threads, which one token leaves idle but a growing scale does not:
// the page's older codes are then rewritten.  (The prompts' write takes 34 us where its
// bytes take 12: a CTA has nothing of its next page under way while it rounds.)
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

constexpr int kKvThreads = 256;  // of the read

struct Kv8Append {
    Kv8View v;
    int8_t *codes[2];
    float *scales[2];
    const void *x[2];
    int64_t stride[2];
    int bf16[2];
};

// Eight consecutive values as floats.
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
}

// NaN becomes 0 and infinities the largest float.
__device__ __forceinline__ void kv8_finite8(float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] == v[i] ? fminf(fmaxf(v[i], -FLT_MAX), FLT_MAX) : 0.f;
}

// The largest magnitude's bits, which order like integers; from 0x7F800000 on
// something is not finite.
__device__ __forceinline__ uint32_t kv8_top8(const float (&v)[8], uint32_t top)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return top;
}

// Eight rint(x / s) as bytes, exactly; inv = 1 / s, or 0 where s = 0.  x * inv is off by
// 1.5 ulp at most, 2e-5 below 127, so only a quotient within 1e-4 of a tie may be
// rounded wrongly: it is taken again in double.  Adding 1.5 * 2^23
// rounds to an integer (ties to even) and leaves it in the low bits, in two's
// complement.  |x| <= 127 s (1 + 2^-23) where s is a normal number; a subnormal s
// may be up to a half off (190 units of 2^-149 give s = 1), so quotients are held
// to 127, in the branch that they all take: below 2^-128 inv is infinite.
__device__ __forceinline__ uint2 kv8_codes8(const float (&x)[8], float s, float inv)
{
    constexpr float kMagic = 12582912.f;
    uint32_t c[8], near = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float t = x[k] * inv, r = t + kMagic;
        c[k] = __float_as_uint(r);
        if (!(fabsf(t - (r - kMagic)) <= 0.4999f)) near |= 1u << k;
    }
    while (near) {  // one in 600 pieces
        const int k = __ffs(near) - 1;
        near &= near - 1;
        float v = x[0];
#pragma unroll
        for (int y = 1; y < 8; ++y) v = k == y ? x[y] : v;
        const uint32_t q = (uint32_t)(int)fmin(fmax(rint((double)v / (double)s), -127.0), 127.0);
#pragma unroll
        for (int y = 0; y < 8; ++y) c[y] = k == y ? q : c[y];
    }
    return make_uint2(__byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410));
}

// Four codes c as rint(c * was / now), exactly, the same way (ratio = was / now).
__device__ __forceinline__ uint32_t kv8_recode4(uint32_t w, float ratio, float was, float now)
{
    constexpr float kMagic = 12582912.f;
    uint32_t c[4], near = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float t = (float)(int8_t)(w >> (8 * e)) * ratio, r = t + kMagic;
        c[e] = __float_as_uint(r);
        if (!(fabsf(t - (r - kMagic)) <= 0.4999f)) near |= 1u << e;
    }
    while (near) {
        const int e = __ffs(near) - 1;
        near &= near - 1;
        const uint32_t q = (uint32_t)(int)rint((double)(int8_t)(w >> (8 * e)) * (double)was / (double)now);
#pragma unroll
        for (int y = 0; y < 4; ++y) c[y] = e == y ? q : c[y];
    }
    return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
}

// G threads; each keeps its first NC pieces of 8 values in registers and reads
// further ones again.
template <int G, int NC>
__global__ void __launch_bounds__(G, 768 / G) k_kv8_append(const Kv8Append a)
{
    __shared__ uint32_t red[G / 32];
    pdl_launch_dependents();
    pdl_wait_primary();
    const Kv8View &v = a.v;
    const int t = threadIdx.x;
    const int item = blockIdx.x, h = blockIdx.y, which = blockIdx.z;
    // the item's sequence, and which of its touched pages (all uniform in the CTA)
    const int b = v.row_start ? kv8_find_seq_warp(v, item, v.P, 2) : item;
    if (b < 0) return;
    const Kv8Seq s = kv8_seq(v, b, &g_kv8_fault);
    const int nth = v.row_start ? item - ((max(__ldg(v.row_start + b), 0) >> v.P_log2) + 2 * b) : 0;
    const int p0 = s.len - s.n, first = max(p0, 0);
    const int64_t j64 = (int64_t)(first >> v.P_log2) + nth;
    if (s.n == 0 || nth < 0 || j64 << v.P_log2 >= s.len) return;  // nth < 0: row_start falls
    const int j = (int)j64, start = j << v.P_log2;
    const int lo = max(first, start), hi = min(s.len, start + v.P);
    const int older = lo - start, d8 = v.D_log2 - 3, n8 = (hi - lo) << d8;
    auto place = [&](int i, int64_t at, int64_t stride) { return at + (i >> d8) * stride + ((i & ((1 << d8) - 1)) << 3); };
    const int64_t stride = which ? a.stride[1] : a.stride[0], at0 = (s.r0 + (int64_t)(lo - p0)) * stride + (int64_t)h * v.D;
    const void *x = which ? a.x[1] : a.x[0];
    const int bf16 = which ? a.bf16[1] : a.bf16[0];
    float f[NC][8];
    uint32_t most = 0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int i = t + c * G;
#pragma unroll
        for (int k = 0; k < 8; ++k) f[c][k] = 0.f;
        if (i < n8) kv8_load8(x, place(i, at0, stride), bf16, f[c]);
    }
    const int page = kv8_page(v, b, j, &g_kv8_fault);
    if (page < 0) return;
    int8_t *codes = (which ? a.codes[1] : a.codes[0]) + ((int64_t)page * v.H + h) * v.P * v.D;
    float *scale = (which ? a.scales[1] : a.scales[0]) + (int64_t)page * v.H + h;
    const float was = older ? fmaxf(*scale, 0.f) : 0.f;
    // the largest magnitude; where something is not finite (a CTA's decision),
    // again over the finite values that stand for it
    bool odd = false;
    while (true) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (odd) kv8_finite8(f[c]);
            most = kv8_top8(f[c], most);
        }
        for (int i = t + NC * G; i < n8; i += G) {
            float g[8];
            kv8_load8(x, place(i, at0, stride), bf16, g);
            if (odd) kv8_finite8(g);
            most = kv8_top8(g, most);
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if ((t & 31) == 0) red[t >> 5] = most;
        __syncthreads();  // also: every thread has read the old scale
#pragma unroll
        for (int i = 0; i < G / 32; ++i) most = max(most, red[i]);
        if (most < 0x7F800000u) break;
        odd = true;
        most = 0;
        __syncthreads();
    }
    const float top = __uint_as_float(most);
    const float now = fmaxf(was, __fdiv_rn(top, 127.f));
    const float inv = now > 0.f ? __frcp_rn(now) : 0.f;
    if (now > was) {
        const float ratio = __fdiv_rn(was, now);
#pragma unroll 4
        for (int i = t; i < older << (v.D_log2 - 4); i += G) {
            const uint4 u = reinterpret_cast<const uint4 *>(codes)[i];
            uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = kv8_recode4(w[k], ratio, was, now);
            reinterpret_cast<uint4 *>(codes)[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    uint2 *dst = reinterpret_cast<uint2 *>(codes) + (older << d8);
#pragma unroll
    for (int c = 0; c < NC; ++c)
        if (t + c * G < n8) dst[t + c * G] = kv8_codes8(f[c], now, inv);
    for (int i = t + NC * G; i < n8; i += G) {
        float g[8];
        kv8_load8(x, place(i, at0, stride), bf16, g);
        if (odd) kv8_finite8(g);
        dst[i] = kv8_codes8(g, now, inv);
    }
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
    // a decode step: about a token per sequence; else a thread per 32 values of a page
    const bool few = b.n_rows <= 4 * (int64_t)b.n_seqs;
    const int G = few ? 128 : c.page_tokens * c.head_dim / 32;
    void (*kern)(const Kv8Append) = few        ? k_kv8_append<128, 1>
                                    : G == 64  ? k_kv8_append<64, 4>
                                    : G == 128 ? k_kv8_append<128, 4>
                                    : G == 256 ? k_kv8_append<256, 4>
                                               : k_kv8_append<512, 4>;
    const cudaError_t e = launch_pdl(kern, dim3((unsigned)items, c.n_heads, 2), dim3(G), 0, st, a);
    return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

struct Kv8Read {
    Kv8View v;
    const int8_t *codes[2];
    const float *scales[2];
    void *out[2];
};

// One warp per row, of keys or of values (blockIdx.y): 4 values a lane, so that a
// head's codes are read and its values written in one piece each; NU heads at a
// time, so that as many loads are under way.
template <int D, bool BF16>
__global__ void __launch_bounds__(kKvThreads) k_kv8_read(const Kv8Read a)
{
    constexpr int PER = 128 / D, NU = 8;  // heads a warp takes at once; times unrolled
    pdl_launch_dependents();
    pdl_wait_primary();
    const Kv8View &v = a.v;
    const int which = blockIdx.y, lane = threadIdx.x & 31;
    void *out = which ? a.out[1] : a.out[0];
    const int r = blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5);
    if (!out || r >= v.n_rows) return;
    const int8_t *codes = which ? a.codes[1] : a.codes[0];
    const float *scales = which ? a.scales[1] : a.scales[0];
    const int b = v.row_start ? kv8_find_seq_warp(v, r, 1, 0) : r;
    if (b < 0) return;
    const Kv8Seq s = kv8_seq(v, b, &g_kv8_fault);
    if (r < s.r0 || r >= s.r0 + s.n) return;  // behind the last sequence
    const int pos = s.len - s.n + (r - s.r0);
    const int page = pos >= 0 ? kv8_page(v, b, pos >> v.P_log2, &g_kv8_fault) : -1;
    const int64_t ph = (int64_t)page * v.H;
    const int own = lane * 4 / D, e = lane * 4 % D;  // this lane's head of a group, and entry
    for (int h0 = own; h0 < v.H; h0 += PER * NU) {
        uint32_t w[NU];
        float sc[NU];
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const int h = h0 + PER * u;
            w[u] = 0;
            sc[u] = 0.f;
            if (page >= 0 && h < v.H) {
                w[u] = __ldg(reinterpret_cast<const uint32_t *>(codes + (((ph + h) << v.P_log2) + (pos & (v.P - 1))) * D + e));
                sc[u] = __ldg(scales + ph + h);
            }
        }
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const int h = h0 + PER * u;
            if (h >= v.H) break;
            float f[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = (float)(int8_t)(w[u] >> (8 * k)) * sc[u];
            const int64_t at = ((int64_t)r * v.H + h) * D + e;
            if (BF16) {
                uint2 o;
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o.x) : "f"(f[1]), "f"(f[0]));
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o.y) : "f"(f[3]), "f"(f[2]));
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + at) = o;
            } else {
                *reinterpret_cast<float4 *>(static_cast<float *>(out) + at) = make_float4(f[0], f[1], f[2], f[3]);
            }
        }
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
    const bool bf16 = out_type == LOWBIT_BF16;
    void (*kern)(const Kv8Read) = c.head_dim == 128 ? (bf16 ? k_kv8_read<128, true> : k_kv8_read<128, false>)
                                                    : (bf16 ? k_kv8_read<64, true> : k_kv8_read<64, false>);
    const int64_t grid = ((int64_t)b.n_rows + kKvThreads / 32 - 1) / (kKvThreads / 32);
    const cudaError_t e = launch_pdl(kern, dim3((unsigned)grid, 2), dim3(kKvThreads), 0, st, a);
    return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

}  // namespace lowbit
