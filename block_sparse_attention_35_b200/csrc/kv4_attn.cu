// kv4_attn.cu - attention of query tokens over the 4-bit token cache.
//
//   s_rj = q_r . k_j / sqrt(D) over the rows j that query r sees,
//   out_r = sum_j e^(s_rj) v_j / sum_j e^(s_rj),   lse_r = log sum_j e^(s_rj),
//   mass_j += sum_r e^(s_rj - lse_r).
//
// The T tokens x G query heads of one key head are the R = T G rows that share its keys.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv4_device.cuh"
#include "pbsa_device.cuh"
#include "token_internal.cuh"

namespace pbsa {

namespace {

constexpr int kWarps = 4;
constexpr int kUnit = 16;          // keys of one tensor-core step
constexpr int kHidden = 0x7fffffff;   // position that no query sees
constexpr float kLog2e = 1.4426950408889634f;
// Probabilities are kept as 2^(s - m + kShift) in fp16, m the running maximum or up to
// kLag below it: at most 2^15, and what is lost below 2^-24 is under 2^-31 of the largest.
constexpr float kShift = 7.f;
constexpr float kLag = 8.f;

struct AttnArgs {
    Kv4Args k;
    int G, R, tiles8;      // query heads of a key head, rows, groups of 8 rows
    int n_splits;
    float* part_o;         // [B Hkv][n_splits][R][D]
    float2* part_ml;       // [B Hkv][n_splits][R]
    uint2* q_frag;         // [B Hkv][tiles8][D / 16][32] (mass pass)
    float* q_fac;          // [B Hkv][tiles8][8]
};

// What a lane reads of sixteen keys.  Lane 4 g + c holds, of keys g and g + 8, the c-th
// quarter of the key's channels (one load), and, of values 2c, 2c+1, 2c+8, 2c+9, the g-th
// eighth of the channels.
template <int D>
struct Unit {
    uint32_t k[2][D / 32], ks[2];
    uint32_t v[4][D / 64], vs[4];
    int pos[2];
};

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&d)[N], const uint8_t* p) {
    if (N == 4) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
        d[0] = v.x, d[1 % N] = v.y, d[2 % N] = v.z, d[3 % N] = v.w;
    } else if (N == 2) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
        d[0] = v.x, d[1 % N] = v.y;
    } else {
        d[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    }
}

template <int D>
__device__ __forceinline__ void load_keys(Unit<D>& x, const pbsa_kv4_cache& c, size_t row0, int len_left, int lane) {
    const int g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int j = g + 8 * r;
        const size_t row = row0 + j;
        load_words(x.k[r], c.k_codes + row * (D / 2) + q * (D / 8));
        if (D == 128) x.ks[r] = __ldg(reinterpret_cast<const uint16_t*>(c.k_scales + row * 8) + q);
        else x.ks[r] = __ldg(c.k_scales + row * 4 + q);
        const int p = __ldg(c.pos + row);
        x.pos[r] = (p < 0 || j >= len_left) ? kHidden : p;
    }
}

template <int D>
__device__ __forceinline__ void load_values(Unit<D>& x, const pbsa_kv4_cache& c, size_t row0, int lane) {
    const int g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const size_t row = row0 + 2 * q + (i & 1) + 8 * (i >> 1);
        load_words(x.v[i], c.v_codes + row * (D / 2) + g * (D / 16));
        x.vs[i] = __ldg(c.v_scales + row * (D / 16) + g * (D / 16) / 8);
    }
}

// s[n] += K Q^T of sixteen keys and rows 8 n .. 8 n + 7; `q` gives the lane's operands of
// step j and row group n.  Step j contracts channels 32c' + 4j .. + 3 of every quarter c'.
template <int D, int NT, typename QF>
__device__ __forceinline__ void scores(float (&s)[NT][4], const Unit<D>& x, QF q) {
    uint32_t sc[2][2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        if (D == 128) {
            const uint32_t h = e4m3x2_to_half2((uint16_t)x.ks[r]);
            sc[r][0] = __byte_perm(h, h, 0x1010);
            sc[r][1] = __byte_perm(h, h, 0x3232);
        } else {
            const uint32_t h = e4m3x2_to_half2((uint16_t)(x.ks[r] * 0x0101u));
            sc[r][0] = sc[r][1] = h;
        }
    }
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
        uint32_t h[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            e2m1x8_to_half2x4(x.k[r][w], h[r][0], h[r][1], h[r][2], h[r][3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[r][i] = hmul2_u32(h[r][i], sc[r][w / 2]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t a[4] = {h[0][2 * i], h[1][2 * i], h[0][2 * i + 1], h[1][2 * i + 1]};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint2 b = q(2 * w + i, n);
                mma_16816(s[n], a, b.x, b.y);
            }
        }
    }
}

// Reads eight query rows (rows of `tile`) into operand order: lane 4 g + c gets row g's
// channels 32c .. 32c+31 (D = 128), scaled by a power of two that brings the row's largest to
// [2^14, 2^15) - exact but for entries 2^-38 below it - and the factor that turns a product
// into a base-2 logit.
template <int D, typename T>
__device__ __forceinline__ void load_queries(const AttnArgs& a, int b, int hkv, int tile, int lane,
                                             uint2 (&frag)[D / 16], float& fac) {
    const int g = lane >> 2, c = lane & 3, r = tile * 8 + g;
    float v[D / 4];
#pragma unroll
    for (int i = 0; i < D / 4; ++i) v[i] = 0.f;
    if (r < a.R) {
        const int t = r / a.G, h = hkv * a.G + r % a.G;
        const T* p = static_cast<const T*>(a.k.q) + b * a.k.sq.b + t * a.k.sq.t + h * a.k.sq.h + c * (D / 4);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + i);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float2 f;
                if (sizeof(T) == 2 && __is_same(T, __half)) {
                    f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
                } else {
                    f = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
                }
                v[8 * i + 2 * k] = f.x;
                v[8 * i + 2 * k + 1] = f.y;
            }
        }
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < D / 4; ++i) amax = fmaxf(amax, fabsf(v[i]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int ex = (int)(__float_as_uint(amax) >> 23);   // biased; 255: inf
    int e = (ex == 0 || ex == 255) ? 0 : 14 - (ex - 127);
    e = min(e, 120);
    const float up = __uint_as_float((uint32_t)(127 + e) << 23);
    fac = rsqrtf((float)D) * kLog2e * a.k.c.k_unit * __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        const __half2 x = __floats2half2_rn(v[4 * j] * up, v[4 * j + 1] * up);
        const __half2 y = __floats2half2_rn(v[4 * j + 2] * up, v[4 * j + 3] * up);
        frag[j] = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    }
}

// Largest position row r sees (kHidden - 1: all of them; -1: none).
__device__ __forceinline__ int row_limit(const AttnArgs& a, int b, int r) {
    if (r >= a.R) return -1;
    return a.k.q_pos ? min(a.k.q_pos[(size_t)b * a.k.T + r / a.G], kHidden - 1) : kHidden - 1;
}

__device__ __forceinline__ int used_rows(const AttnArgs& a, int b, bool report) {
    const int n = a.k.kv_len[b];
    if (n < 0 || n > a.k.c.capacity) {
        if (report) set_status(a.k.status, PBSA_ERR_DEVICE_CHECK);
        return n < 0 ? 0 : a.k.c.capacity;
    }
    return n;
}

template <typename T>
__device__ __forceinline__ void store4(T* p, const float4& v, float k) {
    const T x[4] = {(T)(v.x * k), (T)(v.y * k), (T)(v.z * k), (T)(v.w * k)};
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(x);
}

// One CTA: 8 NT rows of a (sequence, key head) over one split of its keys.  Its warps take
// units of sixteen keys in turn, each with its own running maximum, sum and output, which are
// joined in shared memory at the end.  Keys and values are the row operand of the tensor-core
// steps (S^T = K Q^T, O^T = V^T P^T), so that rows come in groups of eight and a code is
// turned into fp16 once, in the register it is multiplied from.
template <int D, int NT, typename T>
__global__ void __launch_bounds__(32 * kWarps) attn_kernel(AttnArgs a) {
    constexpr int kSteps = D / 16, kRows = 8 * NT;
    extern __shared__ __align__(16) uint8_t sm[];
    uint2* q_sm = reinterpret_cast<uint2*>(sm);                       // [kSteps][NT][32]
    float* fac_sm = reinterpret_cast<float*>(q_sm + kSteps * NT * 32);   // [kRows]
    int* lim_sm = reinterpret_cast<int*>(fac_sm + kRows);                // [kRows]
    float* m_sm = reinterpret_cast<float*>(lim_sm + kRows);              // [kWarps][kRows]
    float* l_sm = m_sm + kWarps * kRows;                                 // [kWarps][kRows]
    float* o_sm = l_sm + kWarps * kRows;                                 // [kWarps][kRows][D]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int split = blockIdx.x % a.n_splits, bh = blockIdx.x / a.n_splits;
    const int b = bh / a.k.c.Hkv, hkv = bh % a.k.c.Hkv, tile0 = blockIdx.y * NT;
    const int N = a.k.c.capacity;

    for (int n = warp; n < NT; n += kWarps) {
        uint2 f[kSteps];
        float fac;
        load_queries<D, T>(a, b, hkv, tile0 + n, lane, f, fac);
#pragma unroll
        for (int j = 0; j < kSteps; ++j) q_sm[(j * NT + n) * 32 + lane] = f[j];
        if (c == 0) {
            fac_sm[8 * n + g] = fac;
            lim_sm[8 * n + g] = row_limit(a, b, (tile0 + n) * 8 + g);
        }
        if (a.q_frag && split == 0 && tile0 + n < a.tiles8) {
            const size_t tile = (size_t)bh * a.tiles8 + tile0 + n;
#pragma unroll
            for (int j = 0; j < kSteps; ++j) a.q_frag[(tile * kSteps + j) * 32 + lane] = f[j];
            if (c == 0) a.q_fac[tile * 8 + g] = fac;
        }
    }
    __syncthreads();

    float fac[NT][2];
    int lim[NT][2];
    uint2 qr[NT == 1 ? kSteps : 1];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            fac[n][i] = fac_sm[8 * n + 2 * c + i];
            lim[n][i] = lim_sm[8 * n + 2 * c + i];
        }
    if (NT == 1) {
#pragma unroll
        for (int j = 0; j < kSteps; ++j) qr[NT == 1 ? j : 0] = q_sm[j * 32 + lane];
    }
    auto qf = [&](int j, int n) -> uint2 { return NT == 1 ? qr[NT == 1 ? j : 0] : q_sm[(j * NT + n) * 32 + lane]; };

    float m[NT][2], mref[NT][2], l[NT][2], o[NT][kSteps][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            m[n][i] = -INFINITY;   // running maximum, common to the lanes of a row
            mref[n][i] = -kShift;  // m - kShift once there is one
            l[n][i] = 0.f;         // this lane's share of the sum
        }
#pragma unroll
        for (int j = 0; j < kSteps; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][j][i] = 0.f;
    }

    const int len = used_rows(a, b, threadIdx.x == 0 && split == 0 && blockIdx.y == 0);
    const int units = (len + kUnit - 1) / kUnit;
    const int per_split = (units + a.n_splits - 1) / a.n_splits;
    const int u_end = min(units, (split + 1) * per_split);
    const size_t row0 = (size_t)bh * N;
    Unit<D> nxt;
    int u = split * per_split + warp;
    if (u < u_end) {
        load_keys(nxt, a.k.cache, row0 + (size_t)u * kUnit, len - u * kUnit, lane);
        load_values(nxt, a.k.cache, row0 + (size_t)u * kUnit, lane);
    }
    for (; u < u_end; u += kWarps) {
        const Unit<D> x = nxt;
        if (u + kWarps < u_end) {
            const int v = u + kWarps;
            load_keys(nxt, a.k.cache, row0 + (size_t)v * kUnit, len - v * kUnit, lane);
            load_values(nxt, a.k.cache, row0 + (size_t)v * kUnit, lane);
        }
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
        scores<D, NT>(s, x, qf);
        // s[n][i]: key g + 8 (i >> 1), row 2c + (i & 1) of group n
        bool grow = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[n][i] = x.pos[i >> 1] <= lim[n][i & 1] ? s[n][i] * fac[n][i & 1] : -INFINITY;
                grow |= s[n][i] > m[n][i & 1] + kLag;
            }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float v = fmaxf(s[n][i], s[n][i + 2]);
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                    const float mn = fmaxf(m[n][i], v);
                    if (mn > m[n][i]) {
                        const float k = exp2f(m[n][i] - mn);   // 0 from the initial -inf
                        l[n][i] *= k;
#pragma unroll
                        for (int j = 0; j < kSteps; ++j) {
                            o[n][j][i] *= k;
                            o[n][j][i + 2] *= k;
                        }
                        m[n][i] = mn;
                        mref[n][i] = mn - kShift;
                    }
                }
        }
        uint32_t p[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[n][i] = exp2f(s[n][i] - mref[n][i & 1]);
                l[n][i & 1] += s[n][i];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const __half2 h = __floats2half2_rn(s[n][2 * i], s[n][2 * i + 1]);
                p[n][i] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&h));
            }
        }
        // rows that hold no token: their values may be anything, their scale becomes zero
        const unsigned live0 = __ballot_sync(0xffffffffu, x.pos[0] != kHidden);
        const unsigned live1 = __ballot_sync(0xffffffffu, x.pos[1] != kHidden);
        uint32_t vs[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const unsigned live = i ? live1 : live0;
            const uint32_t s0 = (live >> (8 * c)) & 1u ? x.vs[2 * i] : 0u;
            const uint32_t s1 = (live >> (8 * c + 4)) & 1u ? x.vs[2 * i + 1] : 0u;
            vs[i] = e4m3x2_to_half2((uint16_t)(s0 | (s1 << 8)));
        }
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {
            // even and odd channels of the lane's eighth, two keys to a byte
            uint32_t h[4][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t va = x.v[2 * i][w], vb = x.v[2 * i + 1][w];
                const uint32_t even = (va & 0x0f0f0f0fu) | ((vb << 4) & 0xf0f0f0f0u);
                const uint32_t odd = ((va >> 4) & 0x0f0f0f0fu) | (vb & 0xf0f0f0f0u);
                e2m1x8_to_half2x4(even, h[2 * i][0], h[2 * i][1], h[2 * i][2], h[2 * i][3]);
                e2m1x8_to_half2x4(odd, h[2 * i + 1][0], h[2 * i + 1][1], h[2 * i + 1][2], h[2 * i + 1][3]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t av[4] = {hmul2_u32(h[0][j], vs[0]), hmul2_u32(h[1][j], vs[0]),
                                        hmul2_u32(h[2][j], vs[1]), hmul2_u32(h[3][j], vs[1])};
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_16816(o[n][4 * w + j], av, p[n][0], p[n][1]);
            }
        }
    }

    // join the warps.  o[n][j][i]: channel (D/8) g + 2j + (i >> 1), row 2c + (i & 1) of group n
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float v = l[n][i];
            v += __shfl_xor_sync(0xffffffffu, v, 4);
            v += __shfl_xor_sync(0xffffffffu, v, 8);
            v += __shfl_xor_sync(0xffffffffu, v, 16);
            const int r = 8 * n + 2 * c + i;
            if (g == 0) {
                m_sm[warp * kRows + r] = m[n][i];
                l_sm[warp * kRows + r] = v;
            }
            float* dst = o_sm + ((size_t)warp * kRows + r) * D + g * (D / 8);
#pragma unroll
            for (int j = 0; j < kSteps; ++j)
                *reinterpret_cast<float2*>(dst + 2 * j) = make_float2(o[n][j][i], o[n][j][i + 2]);
        }
    __syncthreads();
    for (int e = threadIdx.x; e < kRows * (D / 4); e += 32 * kWarps) {
        const int r = e / (D / 4), d = (e % (D / 4)) * 4, row = blockIdx.y * kRows + r;
        if (row >= a.R) continue;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, m_sm[w * kRows + r]);
        const float base = mx == -INFINITY ? 0.f : mx;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float k = exp2f(m_sm[w * kRows + r] - base);
            const float4 x = *reinterpret_cast<const float4*>(o_sm + ((size_t)w * kRows + r) * D + d);
            v.x += k * x.x, v.y += k * x.y, v.z += k * x.z, v.w += k * x.w;
            sum += k * l_sm[w * kRows + r];
        }
        if (a.n_splits > 1) {
            const size_t at = ((size_t)bh * a.n_splits + split) * a.R + row;
            *reinterpret_cast<float4*>(a.part_o + at * D + d) = v;
            if (d == 0) a.part_ml[at] = make_float2(mx, sum);
            continue;
        }
        const int t = row / a.G, h = hkv * a.G + row % a.G;
        const float inv = sum == 0.f ? 0.f : a.k.c.v_unit / sum;
        store4(static_cast<T*>(a.k.out) + (((size_t)b * a.k.T + t) * a.k.c.Hq + h) * D + d, v, inv);
        if (d == 0)
            a.k.lse[((size_t)b * a.k.c.Hq + h) * a.k.T + t] =
                sum == 0.f ? -INFINITY : (mx - kShift + log2f(sum)) * 0.6931471805599453f;
    }
}

// Joins the splits: D / 4 lanes per row.
template <int D, typename T>
__global__ void __launch_bounds__(128) join_kernel(AttnArgs a) {
    constexpr int kLanes = D / 4;
    const long long r = ((long long)blockIdx.x * 128 + threadIdx.x) / kLanes;
    const int d = (threadIdx.x % kLanes) * 4;
    const long long rows = (long long)a.k.c.B * a.k.c.Hkv * a.R;
    if (r >= rows) return;
    const int bh = (int)(r / a.R), row = (int)(r % a.R), b = bh / a.k.c.Hkv, hkv = bh % a.k.c.Hkv;
    const size_t at0 = (size_t)bh * a.n_splits * a.R + row;
    float mx = -INFINITY;
    for (int s = 0; s < a.n_splits; ++s) mx = fmaxf(mx, a.part_ml[at0 + (size_t)s * a.R].x);
    const float base = mx == -INFINITY ? 0.f : mx;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
#pragma unroll 4
    for (int s = 0; s < a.n_splits; ++s) {
        const size_t at = at0 + (size_t)s * a.R;
        const float2 ml = a.part_ml[at];
        const float k = exp2f(ml.x - base);
        const float4 x = *reinterpret_cast<const float4*>(a.part_o + at * D + d);
        v.x += k * x.x, v.y += k * x.y, v.z += k * x.z, v.w += k * x.w;
        sum += k * ml.y;
    }
    const int t = row / a.G, h = hkv * a.G + row % a.G;
    const float inv = sum == 0.f ? 0.f : a.k.c.v_unit / sum;
    store4(static_cast<T*>(a.k.out) + (((size_t)b * a.k.T + t) * a.k.c.Hq + h) * D + d, v, inv);
    if (d == 0)
        a.k.lse[((size_t)b * a.k.c.Hq + h) * a.k.T + t] =
            sum == 0.f ? -INFINITY : (mx - kShift + log2f(sum)) * 0.6931471805599453f;
}

// Masses: the scores are formed again (half of the cache's bytes) once the rows' lse is known;
// a warp owns its keys and walks all rows, so that every sum has one order and one owner.
template <int D>
__global__ void __launch_bounds__(32 * kWarps) mass_kernel(AttnArgs a) {
    constexpr int kSteps = D / 16;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int N = a.k.c.capacity, per_bh = N / (kUnit * kWarps);
    const int bh = blockIdx.x / per_bh, b = bh / a.k.c.Hkv, hkv = bh % a.k.c.Hkv;
    const int u = (blockIdx.x % per_bh) * kWarps + warp;
    const int len = used_rows(a, b, false);
    if (u * kUnit >= len) return;
    Unit<D> x;
    load_keys(x, a.k.cache, (size_t)bh * N + (size_t)u * kUnit, len - u * kUnit, lane);
    float sum[2] = {0.f, 0.f};
    for (int tile = 0; tile < a.tiles8; ++tile) {
        const size_t at = (size_t)bh * a.tiles8 + tile;
        uint2 f[kSteps];
#pragma unroll
        for (int j = 0; j < kSteps; ++j) f[j] = a.q_frag[(at * kSteps + j) * 32 + lane];
        float s[1][4] = {{0.f, 0.f, 0.f, 0.f}};
        scores<D, 1>(s, x, [&](int j, int) { return f[j]; });
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = tile * 8 + 2 * c + i, rr = min(r, a.R - 1);
            const int lim = row_limit(a, b, r);
            const float fac = a.q_fac[at * 8 + 2 * c + i];
            const float lse = a.k.lse[((size_t)b * a.k.c.Hq + hkv * a.G + rr % a.G) * a.k.T + rr / a.G] * kLog2e;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (x.pos[k] <= lim) sum[k] += exp2f(s[0][i + 2 * k] * fac - lse);
        }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 1);
        sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 2);
        if (c == 0 && x.pos[k] != kHidden) a.k.mass[(size_t)bh * N + u * kUnit + g + 8 * k] += sum[k];
    }
}

int row_groups(int R) { return R <= 8 ? 1 : (R <= 16 ? 2 : 4); }

// Splits of the keys: enough CTAs for every SM to hold four, each with at least 256 keys.
int split_count(const pbsa_kv4_config& c, int R) {
    const long long base = (long long)c.B * c.Hkv * ((R + 8 * row_groups(R) - 1) / (8 * row_groups(R)));
    long long s = (4 * kSMs + base - 1) / base;
    const long long most = (c.capacity + 255) / 256;
    if (s > most) s = most;
    return (int)(s < 1 ? 1 : s);
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

template <int D, int NT, typename T>
cudaError_t run_attn(const AttnArgs& a, cudaStream_t st) {
    const size_t smem = (size_t)(D / 16) * NT * 32 * 8 + 8 * NT * 8 + kWarps * 8 * NT * 8 +
                        (size_t)kWarps * 8 * NT * D * 4;
    cudaError_t e = cudaFuncSetAttribute(attn_kernel<D, NT, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int bh = a.k.c.B * a.k.c.Hkv;
    const dim3 grid((unsigned)(bh * a.n_splits), (unsigned)((a.R + 8 * NT - 1) / (8 * NT)));
    attn_kernel<D, NT, T><<<grid, 32 * kWarps, smem, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (a.n_splits > 1) {
        const long long threads = (long long)bh * a.R * (D / 4);
        join_kernel<D, T><<<(unsigned)((threads + 127) / 128), 128, 0, st>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (a.k.mass) {
        mass_kernel<D><<<(unsigned)(bh * (a.k.c.capacity / (kUnit * kWarps))), 32 * kWarps, 0, st>>>(a);
        e = cudaGetLastError();
    }
    return e;
}

template <int D, typename T>
cudaError_t attn_rows(const AttnArgs& a, cudaStream_t st) {
    switch (row_groups(a.R)) {
        case 1: return run_attn<D, 1, T>(a, st);
        case 2: return run_attn<D, 2, T>(a, st);
        default: return run_attn<D, 4, T>(a, st);
    }
}

}  // namespace

size_t kv4_attn_workspace(const pbsa_kv4_config& c, int T) {
    const size_t R = (size_t)T * (c.Hq / c.Hkv), bh = (size_t)c.B * c.Hkv, t8 = (R + 7) / 8;
    const size_t ns = split_count(c, (int)R);
    size_t n = up256(bh * t8 * (c.D / 16) * 32 * 8) + up256(bh * t8 * 8 * 4);
    if (ns > 1) n += up256(bh * ns * R * c.D * 4) + up256(bh * ns * R * 8);
    return n;
}

cudaError_t launch_kv4_attn(const Kv4Args& k, cudaStream_t st) {
    AttnArgs a;
    a.k = k;
    a.G = k.c.Hq / k.c.Hkv;
    a.R = k.T * a.G;
    a.tiles8 = (a.R + 7) / 8;
    a.n_splits = split_count(k.c, a.R);
    const size_t bh = (size_t)k.c.B * k.c.Hkv;
    char* w = static_cast<char*>(k.workspace);
    a.q_frag = nullptr;
    a.q_fac = nullptr;
    if (k.mass) {
        a.q_frag = reinterpret_cast<uint2*>(w);
        a.q_fac = reinterpret_cast<float*>(w + up256(bh * a.tiles8 * (k.c.D / 16) * 32 * 8));
    }
    w += up256(bh * a.tiles8 * (k.c.D / 16) * 32 * 8) + up256(bh * a.tiles8 * 8 * 4);
    a.part_o = reinterpret_cast<float*>(w);
    a.part_ml = reinterpret_cast<float2*>(w + up256(bh * a.n_splits * a.R * k.c.D * 4));
    if (k.c.D == 64)
        return k.c.dtype == PBSA_DTYPE_BF16 ? attn_rows<64, __nv_bfloat16>(a, st) : attn_rows<64, __half>(a, st);
    return k.c.dtype == PBSA_DTYPE_BF16 ? attn_rows<128, __nv_bfloat16>(a, st) : attn_rows<128, __half>(a, st);
}

}  // namespace pbsa
