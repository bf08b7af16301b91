// kv4_evict.cu - the rows of the 4-bit token cache that the next tokens take.
//
// Every row gets a 32-bit key: 0 when it is empty, all ones when it is protected (a first
// token of the sequence or a recent one), else one more than the bits of its accumulated mass
// (non-negative floats order as their bits do).  The n rows with the smallest (key, row) are
// wanted, in row order: the n-th smallest key is found by a radix select, 8 bits a round, then
// one ordered sweep writes the rows below it and the first of those that equal it.
//
// Bound: the masses and positions are read once from HBM (8 bytes a row); later rounds find
// them in L2.
#include "pbsa_device.cuh"
#include "token_internal.cuh"

namespace pbsa {

namespace {

constexpr int kThreads = 1024;
constexpr uint32_t kProtected = 0xffffffffu;

__device__ __forceinline__ uint32_t row_key(int pos, float mass, int n_sink, int keep_from) {
    if (pos < 0) return 0u;
    if (pos < n_sink || pos >= keep_from) return kProtected;
    if (mass != mass) return 0x7f800002u;      // NaN: above infinity
    return __float_as_uint(fmaxf(mass, 0.f) + 0.f) + 1u;   // + 0: no negative zero
}

__global__ void __launch_bounds__(kThreads) evict_kernel(EvictArgs a) {
    __shared__ unsigned hist[256];
    __shared__ uint32_t s_prefix;
    __shared__ int s_rank, s_warp_lt[32], s_warp_eq[32];
    const int bh = blockIdx.x, b = bh / a.Hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t* pos = a.pos + (size_t)bh * a.N;
    const float* mass = a.mass + (size_t)bh * a.N;
    const int keep_from = a.keep_from ? a.keep_from[b] : 0x7fffffff;
    int32_t* rows = a.rows + (size_t)bh * a.n;

    // radix select: the n-th smallest key, and its rank among the keys equal to it
    uint32_t prefix = 0;
    int rank = a.n;   // 1-based rank within the keys that match the prefix so far
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int i = tid; i < a.N; i += kThreads) {
            const uint32_t k = row_key(pos[i], mass[i], a.n_sink, keep_from);
            if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (warp == 0) {
            unsigned c[8], sum = 0;
            for (int j = 0; j < 8; ++j) sum += (c[j] = hist[lane * 8 + j]);
            unsigned incl = sum;
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            unsigned before = incl - sum;
            if (before < (unsigned)rank && (unsigned)rank <= incl) {
                for (int j = 0; j < 8; ++j) {
                    if ((unsigned)rank <= before + c[j]) {
                        s_prefix = prefix | ((uint32_t)(lane * 8 + j) << shift);
                        s_rank = rank - (int)before;
                        break;
                    }
                    before += c[j];
                }
            }
        }
        __syncthreads();
        prefix = s_prefix;
        rank = s_rank;
    }
    const uint32_t tau = prefix;
    const int quota = tau == kProtected ? 0 : rank;   // rows equal to tau that are taken

    // ordered sweep
    int out = 0, eq_seen = 0;
    for (int i0 = 0; i0 < a.N; i0 += kThreads) {
        const int i = i0 + tid;
        const uint32_t k = i < a.N ? row_key(pos[i], mass[i], a.n_sink, keep_from) : kProtected;
        const bool lt = k < tau, eq = k == tau && i < a.N;
        const unsigned mlt = __ballot_sync(0xffffffffu, lt), meq = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) {
            s_warp_lt[warp] = __popc(mlt);
            s_warp_eq[warp] = __popc(meq);
        }
        __syncthreads();
        int lt_before = 0, eq_before = eq_seen, lt_all = 0, eq_all = 0;
        for (int w = 0; w < 32; ++w) {
            const int l = s_warp_lt[w], e = s_warp_eq[w];
            if (w < warp) {
                lt_before += l;
                eq_before += e;
            }
            lt_all += l;
            eq_all += e;
        }
        const unsigned below = (1u << lane) - 1u;
        lt_before += __popc(mlt & below);
        eq_before += __popc(meq & below);
        // rows written before this one: smaller keys, and equal ones within the quota
        const int at = out + lt_before + (min(eq_before, quota) - min(eq_seen, quota));
        if (lt || (eq && eq_before < quota)) rows[at] = i;
        out += lt_all + min(eq_seen + eq_all, quota) - min(eq_seen, quota);
        eq_seen += eq_all;
        __syncthreads();
    }
    if (out < a.n) {
        for (int i = out + tid; i < a.n; i += kThreads) rows[i] = -1;
        if (tid == 0) set_status(a.status, PBSA_ERR_DEVICE_CHECK);
    }
}

}  // namespace

cudaError_t launch_kv4_evict(const EvictArgs& a, cudaStream_t st) {
    evict_kernel<<<a.BH, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace pbsa
