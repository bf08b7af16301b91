// qk_norm_rope.cu - RMS norm of every query and key head with the position rotation in the
// same pass, and its gradients.
//
// Forward, for a head x of D channels:  r = (mean x^2 + eps)^(-1/2),  n_i = x_i r w_i, and every
// rotated pair (a, b) of n becomes (a cos - b sin, b cos + a sin).
// Backward, with the output's gradient turned back, g = Rot^T(dy), i.e. (a cos + b sin,
// b cos - a sin):  dw_i = sum over tokens and heads of g_i x_i r,
//   dx_i = r (g_i w_i - x_i r^2 / D sum_j g_j w_j x_j).
//
// Both are bound by HBM: the forward reads and writes every element once, the backward reads
// x and dy once and writes dx once; nothing is kept between them (r is a sum over a row that
// the backward has in registers anyway).  A warp owns a token and a range of its heads: D/8
// lanes hold one head, 8 channels (16 bytes of a 16-bit type) each, 32 / (D/8) heads per step.
// The token's cosines and sines are loaded once and kept in registers for all of its heads;
// three steps of loads are issued before the first is used, a token's first ones before its
// position is looked up (the position, the table and the heads are then two waits, not three).
// Partners of the half-split pairing sit rot_dim/16 lanes away and are exchanged by shuffles, so
// that memory is only touched with full-width accesses; interleaved partners are in one lane.
//
// The weights' gradients stay in registers over all tokens of a warp, are summed over the
// block in shared memory, and the blocks' sums are added by a second small kernel in a fixed
// order (no atomics), all in 32 bits.
//
// 32760 tokens of 12 + 12 heads of 128 channels, three axes, L2 cold; the backward with the weights'
// sums (3 us):
//   bf16, fp32 gradients   forward 73 us (403 MB, 5.5 TB/s), backward 137 (805 MB, 5.9 TB/s)
//   fp16, fp16 gradients   73, and 122 (604 MB, 5.0 TB/s)
//   fp32                   125 (805 MB, 6.4 TB/s), and 223 (1.21 GB, 5.4 TB/s)
// (a copy runs at 6.5).  In the backward 128 registers leave 16 warps an SM, and what they have in
// flight bounds it where the gradients are narrow: with two steps of loads in flight in place of
// three 147 us, with the weights in shared memory and the next step's loads behind this step's work
// 152.  A step of fp32 is twice the registers: one is in flight in the backward, two in the forward.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pbsa_device.cuh"
#include "token_internal.cuh"

namespace pbsa {

namespace {

constexpr int kWarps = 8;
constexpr int kFwdCtas = 4, kBwdCtas = 2;   // blocks an SM, by registers

// Eight consecutive channels of a lane, as loaded.
template <typename T>
struct Raw8 {
    uint4 v[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
    Raw8<T> r;
    const uint4* q = reinterpret_cast<const uint4*>(p);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.v[i] = q[i];
    return r;
}

__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16>& r, float (&f)[8]) {
    const uint32_t u[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ void unpack8(const Raw8<__half>& r, float (&f)[8]) {
    const uint32_t u[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
}

__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(r.v[i].x);
        f[4 * i + 1] = __uint_as_float(r.v[i].y);
        f[4 * i + 2] = __uint_as_float(r.v[i].z);
        f[4 * i + 3] = __uint_as_float(r.v[i].w);
    }
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ void store8(__half* p, const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    float4* q = reinterpret_cast<float4*>(p);
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// Sum over the LANES lanes that hold one head.
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One lane's share of a token's rotation: the factors of its own channels and, for the
// half-split pairing, of the partner's.
//   interleaved: pairs (2j, 2j+1) of the lane; c[j], s[j] for j < 4.
//   half-split:  out_i = v_i c[i] + partner_i s[i]; s carries the sign of the lane's half.
template <bool IL>
struct Turn {
    float c[IL ? 4 : 8], s[IL ? 4 : 8];
};

template <int D, bool IL>
struct Rotation {
    static constexpr int kLanes = D / 8;
    int chunk;     // this lane's 8 channels of the head: [8 chunk, 8 chunk + 8)
    int partner;   // lane of the partner channels (half-split)
    bool rotated;

    __device__ __forceinline__ Rotation(const pbsa_qk_config& c, int lane) {
        chunk = lane % kLanes;
        rotated = chunk < c.rot_dim / 8;
        partner = lane;
        if (!IL && rotated) partner = lane + (chunk < c.rot_dim / 16 ? c.rot_dim / 16 : -(c.rot_dim / 16));
    }

    // False when a component of the token's position is out of the table.
    __device__ __forceinline__ bool load(const QkArgs& a, long long token, Turn<IL>& t) const {
        const pbsa_qk_config& c = a.c;
        constexpr int n = IL ? 4 : 8;
#pragma unroll
        for (int j = 0; j < n; ++j) {
            t.c[j] = 1.f;
            t.s[j] = 0.f;
        }
        if (c.rot_dim == 0) return true;
        const int32_t* ps = a.pos + token * c.n_axes;
        const int pairs = c.rot_dim / 2;
        int p0 = ps[0], p1 = 0, p2 = 0;
        if (c.n_axes > 1) p1 = ps[1];
        if (c.n_axes > 2) p2 = ps[2];
        if (min(p0, min(p1, p2)) < 0 || max(p0, max(p1, p2)) >= c.table_len) return false;
        if (!rotated) return true;
        const int first = IL ? 4 * chunk : 8 * (chunk % (c.rot_dim / 16));
        const float sign = (IL || chunk >= c.rot_dim / 16) ? 1.f : -1.f;
        if (c.n_axes == 1) {   // consecutive pairs of one table row
            const long long at = (long long)p0 * pairs + first;
#pragma unroll
            for (int j = 0; j < n; j += 4) {
                const float4 cv = __ldg(reinterpret_cast<const float4*>(a.cos + at + j));
                const float4 sv = __ldg(reinterpret_cast<const float4*>(a.sin + at + j));
                t.c[j] = cv.x, t.c[j + 1] = cv.y, t.c[j + 2] = cv.z, t.c[j + 3] = cv.w;
                t.s[j] = sign * sv.x, t.s[j + 1] = sign * sv.y, t.s[j + 2] = sign * sv.z, t.s[j + 3] = sign * sv.w;
            }
            return true;
        }
        const int e0 = c.axis_pairs[0], e1 = e0 + c.axis_pairs[1];
#pragma unroll
        for (int j = 0; j < n; ++j) {
            const int i = first + j;
            const long long at = (long long)(i < e0 ? p0 : (i < e1 ? p1 : p2)) * pairs + i;
            t.c[j] = __ldg(a.cos + at);
            t.s[j] = sign * __ldg(a.sin + at);
        }
        return true;
    }

    // Turns v (dir = 1) or turns it back (dir = -1).  All lanes of the warp call it.
    __device__ __forceinline__ void apply(float (&v)[8], const Turn<IL>& t, float dir) const {
        if (IL) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = v[2 * j], y = v[2 * j + 1], s = dir * t.s[j];
                v[2 * j] = x * t.c[j] - y * s;
                v[2 * j + 1] = y * t.c[j] + x * s;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float o = __shfl_sync(0xffffffffu, v[j], partner);
                v[j] = v[j] * t.c[j] + o * (dir * t.s[j]);
            }
        }
    }
};

__device__ __forceinline__ void load_weights(const float* w, int chunk, float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 1.f;
    if (w) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(w + 8 * chunk));
        const float4 b = __ldg(reinterpret_cast<const float4*>(w + 8 * chunk) + 1);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
        f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
}

// Heads [lo, hi) of the token's Hq + Hkv heads that part `which` (0 queries, 1 keys) has.
__device__ __forceinline__ void part_range(const pbsa_qk_config& c, int which, int lo, int hi, int& h0, int& h1) {
    h0 = which ? max(lo - c.Hq, 0) : lo;
    h1 = which ? hi - c.Hq : min(hi, c.Hq);
}

template <typename T, int D, bool IL>
__global__ void __launch_bounds__(32 * kWarps, kFwdCtas) qk_fwd_kernel(QkArgs a, int heads_per_item, int items_per_token) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kUnroll = sizeof(T) == 2 ? 3 : 2;
    const pbsa_qk_config& c = a.c;
    const int lane = threadIdx.x & 31, row = lane / kLanes;
    const long long item = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const long long token = item / items_per_token;
    if (token >= (long long)c.B * c.T) return;
    const int lo = (int)(item % items_per_token) * heads_per_item;
    const int hi = min(lo + heads_per_item, c.Hq + c.Hkv);
    const long long b = token / c.T, t = token % c.T;
    const Rotation<D, IL> rot(c, lane);
    Raw8<T> raw[kUnroll];
    auto fetch = [&](int which, int h, int h1) {
        const T* x = static_cast<const T*>(a.x[which]) + b * a.sx[which].b + t * a.sx[which].t + 8 * rot.chunk;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) raw[u] = load8(x + min(h + u * kRows + row, h1 - 1) * a.sx[which].h);
    };
    // the first heads are on their way while the token's position is looked up
    const int first = lo >= c.Hq;
    int f0, f1;
    part_range(c, first, lo, hi, f0, f1);
    fetch(first, f0, f1);
    Turn<IL> turn;
    if (!rot.load(a, token, turn)) {
        if (lane == 0) set_status(a.status, PBSA_ERR_DEVICE_CHECK);
        return;
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        int h0, h1;
        part_range(c, which, lo, hi, h0, h1);
        if (h0 >= h1) continue;
        T* y = static_cast<T*>(a.y[which]) + b * a.sy[which].b + t * a.sy[which].t + 8 * rot.chunk;
        float w[8];
        load_weights(a.w[which], rot.chunk, w);
        for (int h = h0; h < h1; h += kRows * kUnroll) {
            if (which != first || h != h0) fetch(which, h, h1);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (h + u * kRows >= h1) break;
                float v[8];
                unpack8(raw[u], v);
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) ss += v[j] * v[j];
                const float r = rsqrtf(row_sum<kLanes>(ss) * (1.f / D) + c.eps);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = v[j] * r * w[j];
                rot.apply(v, turn, 1.f);
                const int hh = h + u * kRows + row;
                if (hh < h1) store8(y + hh * a.sy[which].h, v);
            }
        }
    }
}

template <typename T, typename G, int D, bool IL>
__global__ void __launch_bounds__(32 * kWarps, kBwdCtas) qk_bwd_kernel(QkArgs a, int heads_per_item, int items_per_token) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kUnroll = sizeof(T) == 2 ? 3 : 1;
    const pbsa_qk_config& c = a.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = lane / kLanes;
    const Rotation<D, IL> rot(c, lane);
    float acc[2][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[0][j] = acc[1][j] = 0.f;
    const long long items = (long long)c.B * c.T * items_per_token;
    for (long long item = (long long)blockIdx.x * kWarps + warp; item < items; item += (long long)gridDim.x * kWarps) {
        const long long token = item / items_per_token;
        const int lo = (int)(item % items_per_token) * heads_per_item;
        const int hi = min(lo + heads_per_item, c.Hq + c.Hkv);
        const long long b = token / c.T, t = token % c.T;
        Raw8<T> rx[kUnroll];
        Raw8<G> rg[kUnroll];
        auto fetch = [&](int which, int h, int h1) {
            const T* x = static_cast<const T*>(a.x[which]) + b * a.sx[which].b + t * a.sx[which].t + 8 * rot.chunk;
            const G* gy = static_cast<const G*>(a.gy[which]) + b * a.sg[which].b + t * a.sg[which].t + 8 * rot.chunk;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int hh = min(h + u * kRows + row, h1 - 1);
                rx[u] = load8(x + hh * a.sx[which].h);
                rg[u] = load8(gy + hh * a.sg[which].h);
            }
        };
        // the first heads are on their way while the token's position is looked up
        const int first = lo >= c.Hq;
        int f0, f1;
        part_range(c, first, lo, hi, f0, f1);
        fetch(first, f0, f1);
        Turn<IL> turn;
        if (!rot.load(a, token, turn)) {
            if (lane == 0) set_status(a.status, PBSA_ERR_DEVICE_CHECK);
            continue;
        }
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            int h0, h1;
            part_range(c, which, lo, hi, h0, h1);
            if (h0 >= h1) continue;
            T* dx = static_cast<T*>(a.y[which]) + b * a.sy[which].b + t * a.sy[which].t + 8 * rot.chunk;
            float w[8];
            load_weights(a.w[which], rot.chunk, w);
            for (int h = h0; h < h1; h += kRows * kUnroll) {
                if (which != first || h != h0) fetch(which, h, h1);
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    if (h + u * kRows >= h1) break;
                    float v[8], g[8];
                    unpack8(rx[u], v);
                    unpack8(rg[u], g);
                    rot.apply(g, turn, -1.f);
                    float ss = 0.f, gs = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        ss += v[j] * v[j];
                        gs += g[j] * w[j] * v[j];
                    }
                    const float r = rsqrtf(row_sum<kLanes>(ss) * (1.f / D) + c.eps);
                    const float k = row_sum<kLanes>(gs) * (1.f / D) * r * r;
                    const int hh = h + u * kRows + row;
                    if (hh < h1) {
                        float d[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            acc[which][j] += g[j] * v[j] * r;
                            d[j] = r * (g[j] * w[j] - v[j] * k);
                        }
                        store8(dx + hh * a.sy[which].h, d);
                    }
                }
            }
        }
    }
    if (!a.partial) return;
    // the block's sum: 8 warps x kRows lanes per channel, in a fixed order
    __shared__ float sm[kWarps * kRows][2][D];
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
        for (int j = 0; j < 8; ++j) sm[warp * kRows + row][which][8 * rot.chunk + j] = acc[which][j];
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += 32 * kWarps) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps * kRows; ++k) s += sm[k][i / D][i % D];
        a.partial[(size_t)blockIdx.x * 2 * D + i] = s;
    }
}

// Adds the blocks' sums: a block takes 32 of the 2 D channels, 32 threads deep each.
__global__ void __launch_bounds__(1024) qk_dw_kernel(const float* partial, int blocks, int D, float* dwq, float* dwk) {
    __shared__ float sm[32][33];
    const int i = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    for (int k = threadIdx.y; k < blocks; k += 32) s += partial[(size_t)k * 2 * D + i];
    sm[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) t += sm[k][threadIdx.x];
        float* dw = i < D ? dwq : dwk;
        if (dw) dw[i % D] = t;
    }
}

// Heads of one work item: all of a token's heads when the tokens alone fill the GPU (the
// rotation is then loaded once per token), else as few as still give every resident warp
// (`ctas` blocks an SM) an item of its own, down to the heads of one step.  Of at least one token.
int heads_per_item(const pbsa_qk_config& c, int ctas) {
    const int heads = c.Hq + c.Hkv, step = 32 / (c.D / 8);
    const long long tokens = (long long)c.B * c.T, warps = (long long)kSMs * kWarps * ctas;
    const long long items = tokens < warps ? warps / tokens : 1;
    const long long per = (heads + items - 1) / items;
    return (int)((per + step - 1) / step * step);
}

template <typename T, int D, bool IL>
cudaError_t run_fwd(const QkArgs& a, cudaStream_t st) {
    const int per = heads_per_item(a.c, kFwdCtas), ipt = (a.c.Hq + a.c.Hkv + per - 1) / per;
    const long long items = (long long)a.c.B * a.c.T * ipt;
    qk_fwd_kernel<T, D, IL><<<(unsigned)((items + kWarps - 1) / kWarps), 32 * kWarps, 0, st>>>(a, per, ipt);
    return cudaGetLastError();
}

template <typename T, typename G, int D, bool IL>
cudaError_t run_bwd(const QkArgs& a, cudaStream_t st) {
    const int blocks = qk_bwd_blocks(a.c);   // 0 without tokens: the weights' gradients are zeros then
    if (blocks > 0) {
        const int per = heads_per_item(a.c, kBwdCtas), ipt = (a.c.Hq + a.c.Hkv + per - 1) / per;
        qk_bwd_kernel<T, G, D, IL><<<blocks, 32 * kWarps, 0, st>>>(a, per, ipt);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (!a.dw[0] && !a.dw[1]) return cudaSuccess;
    qk_dw_kernel<<<2 * D / 32, dim3(32, 32), 0, st>>>(a.partial, blocks, D, a.dw[0], a.dw[1]);
    return cudaGetLastError();
}

template <typename T>
cudaError_t fwd_shape(const QkArgs& a, cudaStream_t st) {
    if (a.c.D == 64) return a.c.interleaved ? run_fwd<T, 64, true>(a, st) : run_fwd<T, 64, false>(a, st);
    return a.c.interleaved ? run_fwd<T, 128, true>(a, st) : run_fwd<T, 128, false>(a, st);
}

template <typename T, typename G>
cudaError_t bwd_shape(const QkArgs& a, cudaStream_t st) {
    if (a.c.D == 64) return a.c.interleaved ? run_bwd<T, G, 64, true>(a, st) : run_bwd<T, G, 64, false>(a, st);
    return a.c.interleaved ? run_bwd<T, G, 128, true>(a, st) : run_bwd<T, G, 128, false>(a, st);
}

}  // namespace

int qk_bwd_blocks(const pbsa_qk_config& c) {
    const long long tokens = (long long)c.B * c.T;
    if (tokens == 0) return 0;
    const int per = heads_per_item(c, kBwdCtas);
    const long long need = (tokens * ((c.Hq + c.Hkv + per - 1) / per) + kWarps - 1) / kWarps;
    return (int)(need < kSMs * kBwdCtas ? need : kSMs * kBwdCtas);
}

cudaError_t launch_qk_fwd(const QkArgs& a, cudaStream_t st) {
    switch (a.c.dtype) {
        case PBSA_DTYPE_BF16: return fwd_shape<__nv_bfloat16>(a, st);
        case PBSA_DTYPE_FP16: return fwd_shape<__half>(a, st);
        default: return fwd_shape<float>(a, st);
    }
}

cudaError_t launch_qk_bwd(const QkArgs& a, cudaStream_t st) {
    if (a.c.dtype == PBSA_DTYPE_FP32) return bwd_shape<float, float>(a, st);
    const bool f32 = a.c.grad_dtype == PBSA_DTYPE_FP32;
    if (a.c.dtype == PBSA_DTYPE_BF16)
        return f32 ? bwd_shape<__nv_bfloat16, float>(a, st) : bwd_shape<__nv_bfloat16, __nv_bfloat16>(a, st);
    return f32 ? bwd_shape<__half, float>(a, st) : bwd_shape<__half, __half>(a, st);
}

}  // namespace pbsa
