// kv4_attn.cuh - what the attention kernels over the 4-bit token cache share: their arguments,
// the list of work that CTAs split among themselves, and the end of a row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>

#include "kv4_device.cuh"
#include "pbsa_device.cuh"
#include "token_internal.cuh"

namespace pbsa {

constexpr int kHidden = 0x7fffffff;        // position that no query sees
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Probabilities are kept as 2^((s - m) fac + kShift) in fp16, s a product, fac its factor to a base-2
// logit and m the largest product of the row so far or one at most kLag / fac below it: at most
// 2^15, and what is lost below 2^-24 is under 2^-31 of the largest.  The difference is formed
// before it is scaled: near the largest it is exact, while a logit of 2^24 and more, rounded
// alone, would be off by whole powers of two, past fp16's range at 2^27.
constexpr float kShift = 7.f;
constexpr float kLag = 8.f;
// Where a row's largest base-2 logit is below this, the difference may as well be formed by the
// multiply-add that scales it: rounding the constant costs no more than 2^-24 of the logit, which
// its product has lost already, and it is one instruction less for every score (chunk_kernel; the
// other kernels have room for it and always subtract).
constexpr float kNear = 256.f;

// The T tokens x G query heads of one key head are the R = T G rows that share its keys; a CTA
// takes `rows` of them at a time.
struct AttnArgs {
    Kv4Args k;
    int G, R;
    int rows, groups, heads;   // rows of a group, groups of a key head, Hkv * groups
    int block;                 // keys of one piece of work
    int ctas;                  // CTAs that share the work
    float* part_o;             // [ctas][2][rows][D]
    float4* part_ml;           // [ctas][2][rows]: largest product, sum, factor of the row
    float4* row_ref;           // [B Hkv][R] (masses): a probability is 2^((s - x) y + z)
    float* logits;             // [B Hkv][R][N] products (mass of few rows)
    int tiles8;                // groups of 8 rows
    uint2* q_frag;             // [B Hkv][tiles8][D / 16][32] (mass of more rows)
    int tiles128;              // groups of 128 rows
    uint8_t* q_tile;           // [B Hkv][tiles128][128 rows x D fp16 as they lie in shared memory]
    float* q_scale;            // [B Hkv][tiles128][128]: factor from a product to a base-2 logit
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Programmatic launches: lets the next kernel of the stream start early; waits for the one
// before (all of it, with its writes).
__device__ __forceinline__ void grid_dependency_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// A power of two that brings a row's largest entry to [2^14, 2^15) in fp16 - entries keep an
// absolute error of at most 2^-39 of it, half of fp16's smallest step (2^-145 where it is below
// 2^-106 and not brought all the way); bf16 entries down to 2^-31 of it are exact - and the factor
// that turns a product of the row so scaled into a base-2 logit.
// The factor is at least the smallest normal number: where it would be less (a small unit, a tiny
// row) every logit is next to zero anyway, and -infinity for a hidden key times zero would be NaN.
// It is at most the largest: where it would be more, so are logits, but not their differences' signs.
__device__ __forceinline__ void query_scale(const AttnArgs& a, float amax, float& up, float& fac) {
    const int ex = (int)(__float_as_uint(amax) >> 23);   // biased; 255: inf
    const int e = (ex == 0 || ex == 255) ? 0 : min(14 - (ex - 127), 120);
    up = __uint_as_float((uint32_t)(127 + e) << 23);
    fac = rsqrtf((float)a.k.c.D) * kLog2e * a.k.c.k_unit * __uint_as_float((uint32_t)(127 - e) << 23);
    fac = fminf(fmaxf(fac, FLT_MIN), FLT_MAX);
}

// Four channels from ch on of query row r, zeros past the last row.
template <typename T>
__device__ __forceinline__ float4 load_query4(const AttnArgs& a, int b, int hkv, int r, int ch) {
    if (r >= a.R) return make_float4(0.f, 0.f, 0.f, 0.f);
    const int t = r / a.G, h = hkv * a.G + r - t * a.G;
    const T* p = static_cast<const T*>(a.k.q) + b * a.k.sq.b + t * a.k.sq.t + h * a.k.sq.h + ch;
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    if (__is_same(T, __half)) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
        return make_float4(x.x, x.y, y.x, y.y);
    }
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}

// D / 4 lanes hold a query row, four channels each: the row in fp16, scaled, and its factor.
template <int D>
__device__ __forceinline__ uint2 scale_query4(const AttnArgs& a, const float4& v, float& fac) {
    float amax = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
#pragma unroll
    for (int o = D / 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    float up;
    query_scale(a, amax, up, fac);
    const __half2 x = __floats2half2_rn(v.x * up, v.y * up), y = __floats2half2_rn(v.z * up, v.w * up);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

// Largest position row r sees (kHidden - 1: all of them; -1: none).
__device__ __forceinline__ int row_limit(const AttnArgs& a, int b, int r) {
    if (r >= a.R) return -1;
    return a.k.q_pos ? min(a.k.q_pos[(size_t)b * a.k.T + r / a.G], kHidden - 1) : kHidden - 1;
}

__device__ __forceinline__ int used_rows(const AttnArgs& a, int b) {
    return max(0, min(a.k.kv_len[b], a.k.c.capacity));
}

__device__ __forceinline__ int blocks_of(const AttnArgs& a, int len) { return (len + a.block - 1) / a.block; }

// The work of a call is the list of all blocks of keys, by sequence, head and block (below
// 2^31 of them), a head here being one of `groups` groups of rows of a key head (one, up to
// kFewRows): the groups follow one another, so that CTAs side by side read the same keys.
// n = min(ctas, total) CTAs share it in runs of `each` blocks or, the first `more` of them, one
// more.  A warp makes and asks it together: every lane adds up the blocks of its share of the
// sequences.
struct WorkList {
    int total, n, each, more;
    int per, upto, mine;   // sequences of a lane, blocks of the lanes up to this one, and its own

    __device__ __forceinline__ WorkList(const AttnArgs& a, int lane) {
        const int B = a.k.c.B;
        per = (B + 31) / 32;
        mine = 0;
        for (int b = lane * per; b < min(B, (lane + 1) * per); ++b) mine += blocks_of(a, used_rows(a, b));
        mine *= a.heads;
        upto = mine;
        if (B > 1) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
        }
        total = __shfl_sync(0xffffffffu, upto, B > 1 ? 31 : 0);
        n = min(a.ctas, total);
        each = n > 0 ? total / n : 0;
        more = total - each * n;
    }

    __device__ __forceinline__ int first_of(int cta) const { return cta * each + min(cta, more); }
    __device__ __forceinline__ int cta_of(int w) const {
        const int wide = more * (each + 1);
        return w < wide ? w / (each + 1) : more + (w - wide) / each;
    }

    // Blocks before sequence b.
    __device__ __forceinline__ int before(const AttnArgs& a, int lane, int b) const {
        const int src = b / per;
        int at = upto - mine;
        if (lane == src)
            for (int x = src * per; x < b; ++x) at += blocks_of(a, used_rows(a, x)) * a.heads;
        return __shfl_sync(0xffffffffu, at, src);
    }

    // The sequence of block w, and the blocks before that sequence.
    __device__ __forceinline__ void find(const AttnArgs& a, int lane, int w, int& b, int& before) const {
        const bool here = upto > w && upto - mine <= w && (lane == 0 || a.k.c.B > 1);
        const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
        int at = upto - mine, bb = lane * per;
        if (here) {
            while (true) {
                const int k = blocks_of(a, used_rows(a, bb)) * a.heads;
                if (w < at + k) break;
                at += k;
                ++bb;
            }
        }
        b = __shfl_sync(0xffffffffu, bb, src);
        before = __shfl_sync(0xffffffffu, at, src);
    }
};

// A walk over the work list, block by block.
struct Cursor {
    int b, h, blk, len;

    __device__ __forceinline__ void start(const AttnArgs& a, int b_, int in_seq) {
        b = b_;
        len = used_rows(a, b);
        const int n = blocks_of(a, len);
        h = in_seq / n;
        blk = in_seq - h * n;
    }

    // To the next block, when there are `left` of them.
    __device__ __forceinline__ void next(const AttnArgs& a, int left) {
        if (++blk * a.block < len) return;
        blk = 0;
        if (++h < a.heads) return;
        h = 0;
        if (left <= 0) return;
        do len = used_rows(a, ++b);
        while (len == 0);
    }
};

template <typename T>
__device__ __forceinline__ void store4(T* p, const float4& v, float k) {
    const T x[4] = {(T)(v.x * k), (T)(v.y * k), (T)(v.z * k), (T)(v.w * k)};
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(x);
}

// A finished row's lse and, where masses follow, its probabilities' reference.
__device__ __forceinline__ void finish_sum(const AttnArgs& a, int b, int hkv, int row, int t, int h, float mx, float fac,
                                           float sum) {
    const float l2 = log2f(sum);
    a.k.lse[((size_t)b * a.k.c.Hq + h) * a.k.T + t] = sum == 0.f ? -INFINITY : (fmaf(mx, fac, -kShift) + l2) * kLn2;
    if (a.row_ref)   // a row that sees nothing: 2^-inf
        a.row_ref[((size_t)b * a.k.c.Hkv + hkv) * a.R + row] =
            sum == 0.f ? make_float4(0.f, 0.f, -INFINITY, 0.f) : make_float4(mx, fac, kShift - l2, 0.f);
}

// Four channels of a finished row: v = sum of probabilities times values, relative to the
// product mx.
template <int D, typename T>
__device__ __forceinline__ void finish_row(const AttnArgs& a, int b, int hkv, int row, int d, const float4& v, float mx,
                                           float fac, float sum) {
    const int t = row / a.G, h = hkv * a.G + row % a.G;
    store4(static_cast<T*>(a.k.out) + (((size_t)b * a.k.T + t) * a.k.c.Hq + h) * D + d, v,
           sum == 0.f ? 0.f : a.k.c.v_unit / sum);
    if (d == 0) finish_sum(a, b, hkv, row, t, h, mx, fac, sum);
}

// Launches a kernel that may start while the one before it in the stream still runs; every
// thread of it waits for that one (grid_dependency_wait) before it reads its results.
template <typename... More>
cudaError_t launch_after(void (*kernel)(AttnArgs, More...), dim3 grid, int threads, size_t smem, cudaStream_t st, const AttnArgs& a,
                         More... more) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, more...);
}

// Up to so many rows of a key head go to attn_kernel, more to the kernels of kv4_chunk.cu.  With 32
// rows (4 sequences x 8 heads, 8192 cached rows) attn_kernel takes 40.4 us and chunk_kernel 39.7
// (54.4 against 79.8 with masses; D = 64: 28.6 against 34.5, 38.6 against 72.0); with 40 rows, of
// which attn_kernel would need two groups, 56.6 against 40.3 (85 against 80.3).
constexpr int kFewRows = 32;
inline bool chunk_takes(int R) { return R > kFewRows; }

// Many rows (kv4_chunk.cu).
cudaError_t launch_chunk_attn(const AttnArgs& a, cudaStream_t st);
cudaError_t launch_chunk_mass(const AttnArgs& a, cudaStream_t st);
constexpr int kChunkRows = 256, kChunkKeys = 128;

}  // namespace pbsa
