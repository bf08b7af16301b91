// kv4_append.cu - new tokens into the 4-bit token cache, and its rows back as values.
//
// Format (include/pbsa.h): sixteen channels share scale = e4m3(amax / 6 / unit); a channel is
// the e2m1 code nearest to x / unit / scale.
//
// Every rounding is the format's own, ties included.  Inputs have at most 11 significant bits
// and the borders between codes (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5 times an e4m3 scale) at
// most 7, so an input that is not on a border is at least 2^-11 of it away.  x / scale is formed
// as x times the scale's reciprocal, off by at most 2^-22 of it, and rounded to a multiple of
// 2^-15 (by adding and subtracting 384): on a border, that gives the border again (a multiple
// of 1/4), beside one it stays at least 2^-14 away.  The conversion then decides as exact
// arithmetic would.  The same distances make one IEEE division exact enough for amax / 6 against
// the borders of e4m3.  (4680 tokens of 12 heads: 20.2 us with a division a channel, 13.8 with the
// largest magnitude and NaN found in fp32 and divisions for a thread's place, 11.8 so.)
//
// append_kernel and read_kernel are bound by HBM: one thread owns one block of sixteen
// channels, 32 bytes of a 16-bit type against 8 bytes of codes and one scale byte; neighbouring
// threads own neighbouring blocks, so a warp touches whole sectors on both sides.  4680 tokens
// of 12 heads of 128 channels, L2 cold: append 11.6 us (28.8 MB read, 8.1 MB written, to
// scattered rows), read 10.5 us; 18720 tokens 32.3 and 36.1 us, so 4 us are fixed (launch, the
// first look-ups) and the rest streams at 5.3 and 4.5 TB/s: a thread waits for its row's place
// before it can store (append) or load (read).  One token of 32 x 8 caches 2.7 and 2.5 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv4_device.cuh"
#include "pbsa_device.cuh"
#include "token_internal.cuh"

namespace pbsa {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float2 widen2(uint32_t u, __nv_bfloat16*) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ float2 widen2(uint32_t u, __half*) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
__device__ __forceinline__ uint32_t narrow2(float a, float b, __nv_bfloat16*) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t narrow2(float a, float b, __half*) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ constexpr uint32_t infinity_bits(__nv_bfloat16*) { return 0x7f80u; }
__device__ constexpr uint32_t infinity_bits(__half*) { return 0x7c00u; }

// The largest magnitude of sixteen values, as its bits: those order as the values do, and NaN
// comes above infinity.
__device__ __forceinline__ uint32_t top_bits(const uint32_t (&u)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = __vmaxu2(m, u[j] & 0x7fff7fffu);
    return max(m & 0xffffu, m >> 16);
}

// Quantises sixteen values x `inv` (a power of two, one over the unit): 8 bytes of codes and the
// scale byte.  `top`: the bits of the largest magnitude.  The unit goes into the scale's
// reciprocal, which it leaves exact.
template <typename T>
__device__ __forceinline__ uint2 quantise16(const uint32_t (&u)[8], uint32_t top, float inv, uint8_t* scale) {
    const float amax = widen2(top, static_cast<T*>(nullptr)).x * inv;
    const uint8_t sb = e4m3_from_float(__fdiv_rn(amax, 6.f));
    *scale = sb;
    const float s = e4m3_to_float(sb);
    uint32_t w[2] = {0, 0};
    if (s > 0.f) {
        const float r = __frcp_rn(s) * inv;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 x = widen2(u[i], static_cast<T*>(nullptr));
            const float lo = __fsub_rn(__fmaf_rn(x.x, r, 384.f), 384.f);
            const float hi = __fsub_rn(__fmaf_rn(x.y, r, 384.f), 384.f);
            w[i / 4] |= e2m1x2_from_float(lo, hi) << (8 * (i % 4));
        }
    }
    return make_uint2(w[0], w[1]);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 8) append_kernel(Kv4Args a, float inv_unit_k, float inv_unit_v) {
    const pbsa_kv4_config& c = a.c;
    const int log_gpr = c.D == 128 ? 3 : 2, gpr = 1 << log_gpr;   // blocks of a row
    // block -> (keys or values, sequence); thread -> (token, key head, block): the source's order
    const int is_v = blockIdx.z, b = blockIdx.y;
    const unsigned i = blockIdx.x * kThreads + threadIdx.x, th = i >> log_gpr, Hkv = c.Hkv;
    const int g = i & (gpr - 1), t = th / Hkv, h = th - t * Hkv;
    if (t >= a.T) return;
    // the source is on its way while the token's place is looked up
    const Strides& s = is_v ? a.sv : a.sk;
    const T* src = static_cast<const T*>(is_v ? a.v_new : a.k_new) + b * s.b + t * s.t + h * s.h + 16 * g;
    const uint4 lo = __ldg(reinterpret_cast<const uint4*>(src)), hi = __ldg(reinterpret_cast<const uint4*>(src) + 1);
    const size_t bh = (size_t)b * c.Hkv + h;
    const int pos = a.pos_new[(size_t)b * a.T + t];
    const int row = a.rows ? a.rows[bh * a.T + t] : pos;
    if (pos < 0) return;
    if (row < 0 || row >= c.capacity || pos == 0x7fffffff) {   // that position is kHidden
        set_status(a.status, PBSA_ERR_DEVICE_CHECK);
        return;
    }
    uint32_t u[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    constexpr uint32_t kInf = infinity_bits(static_cast<T*>(nullptr));
    uint32_t top = top_bits(u);
    if (top > kInf) {   // a NaN becomes 0
        set_status(a.status, PBSA_ERR_DEVICE_CHECK);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            u[j] &= ((u[j] & 0x7fffu) > kInf ? 0u : 0xffffu) | ((u[j] >> 16 & 0x7fffu) > kInf ? 0u : 0xffff0000u);
        top = top_bits(u);
    }
    const size_t at = ((bh * c.capacity + row) << log_gpr) + g;
    uint8_t scale;
    const uint2 codes = quantise16<T>(u, top, is_v ? inv_unit_v : inv_unit_k, &scale);
    reinterpret_cast<uint2*>(is_v ? a.cache.v_codes : a.cache.k_codes)[at] = codes;
    (is_v ? a.cache.v_scales : a.cache.k_scales)[at] = scale;
    if (g == 0 && !is_v) {
        a.cache.pos[bh * c.capacity + row] = pos;
        if (a.mass) a.mass[bh * c.capacity + row] = 0.f;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) read_kernel(Kv4Args a) {
    const pbsa_kv4_config& c = a.c;
    const int log_gpr = c.D == 128 ? 3 : 2, gpr = 1 << log_gpr;
    // block -> (keys or values, sequence and key head); thread -> (row, block)
    const unsigned per = (unsigned)((a.n * gpr + kThreads - 1) / kThreads), bh = blockIdx.x / per;
    const unsigned i = (blockIdx.x - bh * per) * kThreads + threadIdx.x;
    const int is_v = blockIdx.y, g = i & (gpr - 1), j = i >> log_gpr;
    if (j >= a.n) return;
    const int row = a.rows ? a.rows[(size_t)bh * a.n + j] : j;
    uint32_t out[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (row >= 0 && row < c.capacity) {
        const size_t at = ((size_t)bh * c.capacity + row) * gpr + g;
        const uint2 w = reinterpret_cast<const uint2*>(is_v ? a.cache.v_codes : a.cache.k_codes)[at];
        const float s = e4m3_to_float((is_v ? a.cache.v_scales : a.cache.k_scales)[at]) * (is_v ? c.v_unit : c.k_unit);
        uint32_t h[8];
        e2m1x8_to_half2x4(w.x, h[0], h[1], h[2], h[3]);
        e2m1x8_to_half2x4(w.y, h[4], h[5], h[6], h[7]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
            out[k] = narrow2(v.x * s, v.y * s, static_cast<T*>(nullptr));
        }
    } else if (row != -1) {
        set_status(a.status, PBSA_ERR_DEVICE_CHECK);
    }
    T* dst = static_cast<T*>(is_v ? a.v_out : a.k_out) + (((size_t)bh * a.n + j) * gpr + g) * 16;
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(out[0], out[1], out[2], out[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Args& a, cudaStream_t st) {
    const dim3 grid((unsigned)((a.T * a.c.Hkv * (a.c.D / 16) + kThreads - 1) / kThreads), (unsigned)a.c.B, 2);
    const float ik = 1.f / a.c.k_unit, iv = 1.f / a.c.v_unit;   // exact: powers of two
    if (a.c.dtype == PBSA_DTYPE_BF16) append_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a, ik, iv);
    else append_kernel<__half><<<grid, kThreads, 0, st>>>(a, ik, iv);
    return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4Args& a, cudaStream_t st) {
    const dim3 grid((unsigned)(a.c.B * a.c.Hkv * ((a.n * (a.c.D / 16) + kThreads - 1) / kThreads)), 2);
    if (a.c.dtype == PBSA_DTYPE_BF16) read_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a);
    else read_kernel<__half><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace pbsa
