// kv4_evict.cu - the rows of the 4-bit token cache that the next tokens take.
//
// Every row gets a 32-bit key: 0 when it is empty, all ones when it is protected (a first
// token of the sequence or a recent one), else one more than the bits of its accumulated mass
// (non-negative floats order as their bits do).  The n rows with the smallest (key, row) are
// wanted, in row order.
//
// Bound: the masses and positions are read once from HBM, 8 bytes a row.  A cluster of one to
// eight CTAs holds all keys of a (sequence, key head) in registers; a warp owns consecutive
// rows.  The n-th smallest key is found by a radix select in three rounds (11, 11 and 10 bits)
// with histograms in shared memory: only the keys that share the digits found so far take part
// in a round, so nearly all of the work is the first, and 11 bits of a float tell octaves and
// quarters apart, which keeps the histogram's adds off each other.  Two sweeps over the
// registers then count and write the rows in order: the counts of a warp need no barrier, and
// one exchange between the warps and CTAs places them.  A single row (n = 1) is one reduction.
//
// L2 cold: 1 row of each of 32 x 8 caches of 8192 rows 5.7 us (16.8 MB, 2.9 TB/s; launch, one
// round trip to memory and the reduction), all 256 CTAs at once: with 4-byte loads and one CTA an
// SM 7.7.  1560 rows of each of 12 caches of 18752 9.7 us with eight CTAs a cache, 12.8 with four,
// 16.5 with one, which holds 19 keys a thread.
#include <cooperative_groups.h>

#include "pbsa_device.cuh"
#include "token_internal.cuh"

namespace pbsa {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr uint32_t kProtected = 0xffffffffu;

__device__ __forceinline__ uint32_t row_key(int pos, float mass, int n_sink, int keep_from) {
    if (pos < 0) return 0u;
    if (pos < n_sink || pos >= keep_from) return kProtected;
    if (mass != mass) return 0x7f800002u;      // NaN: above infinity
    return __float_as_uint(fmaxf(mass, 0.f) + 0.f) + 1u;   // + 0: no negative zero
}

// Inclusive sum over the block of one value a thread; `sums` is shared scratch of kWarps.
__device__ __forceinline__ unsigned block_scan(unsigned v, unsigned* sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    unsigned before = lane < warp ? sums[lane] : 0u;
    before = __reduce_add_sync(0xffffffffu, before);
    return v + before;
}

// K > 0: a thread keeps K keys, a multiple of 4; K = 0: `tiles` of them, read again in every round (a cache of
// more than kMaxCluster x 24576 rows).
template <int K>
__global__ void __launch_bounds__(kThreads, K > 8 ? 1 : 2) evict_kernel(EvictArgs a, int tiles) {
    __shared__ unsigned hist[kBins];
    __shared__ unsigned sums[kWarps];
    __shared__ unsigned s_lt[kWarps], s_eq[kWarps];
    __shared__ unsigned s_cta[kMaxCluster][2];   // every CTA's counts below and equal to the threshold
    __shared__ unsigned s_found[2];              // prefix and rank, from the first CTA
    __shared__ unsigned long long s_min[kMaxCluster][kWarps];
    const cg::cluster_group cluster = cg::this_cluster();
    const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int bh = blockIdx.x / ctas, b = bh / a.Hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t* pos = a.pos + (size_t)bh * a.N;
    const float* mass = a.mass + (size_t)bh * a.N;
    const int keep_from = a.keep_from ? a.keep_from[b] : 0x7fffffff;
    int32_t* rows = a.rows + (size_t)bh * a.n;
    const int per = K > 0 ? K : tiles;
    // a warp's rows are consecutive, four in a row a thread: one 16-byte load for each array
    const int row0 = (rank * kWarps + warp) * per * 32 + 4 * lane;
    auto row = [&](int j) { return row0 + 128 * (j / 4) + j % 4; };

    uint32_t keys[K > 0 ? K : 1];
    if (K > 0) {
#pragma unroll
        for (int j0 = 0; j0 < K; j0 += 8) {   // loads in flight: of eight keys
            int4 p[2];
            float4 m[2];
#pragma unroll
            for (int v = 0; v < 2 && j0 + 4 * v < K; ++v) {
                const int i = row(j0 + 4 * v);   // a multiple of 4, as N is
                p[v] = i < a.N ? *reinterpret_cast<const int4*>(pos + i) : make_int4(-1, -1, -1, -1);
                m[v] = i < a.N ? *reinterpret_cast<const float4*>(mass + i) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int v = 0; v < 2 && j0 + 4 * v < K; ++v) {
                const int j = j0 + 4 * v;
                const bool in = row(j) < a.N;
                keys[j] = in ? row_key(p[v].x, m[v].x, a.n_sink, keep_from) : kProtected;
                keys[j + 1] = in ? row_key(p[v].y, m[v].y, a.n_sink, keep_from) : kProtected;
                keys[j + 2] = in ? row_key(p[v].z, m[v].z, a.n_sink, keep_from) : kProtected;
                keys[j + 3] = in ? row_key(p[v].w, m[v].w, a.n_sink, keep_from) : kProtected;
            }
        }
    }
    auto key = [&](int j) -> uint32_t {
        if (K > 0) return keys[K > 0 ? j : 0];
        const int i = row(j);
        return i < a.N ? row_key(pos[i], mass[i], a.n_sink, keep_from) : kProtected;
    };

    if (a.n == 1) {   // the smallest (key, row) alone: no select
        unsigned long long best = ~0ull;
#pragma unroll
        for (int j = 0; j < per; ++j) best = min(best, ((unsigned long long)key(j) << 32) | (unsigned)row(j));
        const unsigned hi = __reduce_min_sync(0xffffffffu, (unsigned)(best >> 32));
        const unsigned lo = __reduce_min_sync(0xffffffffu, (unsigned)(best >> 32) == hi ? (unsigned)best : 0xffffffffu);
        if (ctas > 1) cluster.sync();   // the first CTA runs before its memory is written
        if (lane == 0) cluster.map_shared_rank(&s_min[rank][warp], 0)[0] = ((unsigned long long)hi << 32) | lo;
        if (ctas > 1) cluster.sync();
        else __syncthreads();
        if (rank == 0 && warp == 0) {
            best = ~0ull;
            for (int r = 0; r < ctas; ++r) best = min(best, s_min[r][lane]);
            const unsigned h = __reduce_min_sync(0xffffffffu, (unsigned)(best >> 32));
            const unsigned l = __reduce_min_sync(0xffffffffu, (unsigned)(best >> 32) == h ? (unsigned)best : 0xffffffffu);
            if (lane == 0) {
                rows[0] = h == kProtected ? -1 : (int)l;
                if (h == kProtected) set_status(a.status, PBSA_ERR_DEVICE_CHECK);
            }
        }
        return;
    }

    // radix select: the n-th smallest key, and its rank among the keys equal to it
    uint32_t prefix = 0, known = 0;   // digits found so far, and their mask
    unsigned want = a.n;              // 1-based rank among the keys with these digits
    for (int round = 0; round < 3; ++round) {
        const int shift = round == 0 ? 21 : (round == 1 ? 10 : 0), bits = round == 2 ? 10 : 11;
        const uint32_t mask = (1u << bits) - 1u;
        for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
        if (ctas > 1) cluster.sync();
        else __syncthreads();
#pragma unroll
        for (int j = 0; j < per; ++j) {
            const uint32_t k = key(j);
            const bool in = (k & known) == prefix && row(j) < a.N;
            const unsigned who = __ballot_sync(0xffffffffu, in);
            if (who == 0) continue;
            const unsigned digit = (k >> shift) & mask;
            // a warp of one digit (new rows' zero masses, protected rows) adds once
            const unsigned lead = __shfl_sync(0xffffffffu, digit, __ffs(who) - 1);
            if (__ballot_sync(0xffffffffu, in && digit != lead) == 0) {
                if (lane == 0) atomicAdd(&hist[lead], (unsigned)__popc(who));
            } else if (in) {
                atomicAdd(&hist[digit], 1u);
            }
        }
        __syncthreads();
        if (ctas > 1) {
            if (rank > 0) {
                unsigned* h0 = cluster.map_shared_rank(hist, 0);
                for (int i = tid; i < kBins; i += kThreads)
                    if (hist[i]) atomicAdd(&h0[i], hist[i]);
            }
            cluster.sync();
        }
        if (rank == 0) {
            const unsigned c0 = hist[2 * tid], c1 = hist[2 * tid + 1];
            const unsigned upto = block_scan(c0 + c1, sums), before = upto - c0 - c1;
            if (before < want && want <= upto) {
                const bool second = want > before + c0;
                const unsigned found[2] = {prefix | ((unsigned)(2 * tid + second) << shift),
                                           want - before - (second ? c0 : 0u)};
                for (int r = 0; r < ctas; ++r) {
                    unsigned* f = cluster.map_shared_rank(s_found, r);
                    f[0] = found[0];
                    f[1] = found[1];
                }
            }
        }
        if (ctas > 1) cluster.sync();
        else __syncthreads();
        prefix = s_found[0];
        want = s_found[1];
        known |= mask << shift;
    }
    const uint32_t tau = prefix;
    const unsigned quota = tau == kProtected ? 0u : want;   // rows equal to tau that are taken

    // counts of every warp, then the rows below tau and the first of those equal to it
    unsigned lt = 0, eq = 0;
#pragma unroll
    for (int j = 0; j < per; ++j) {
        const uint32_t k = key(j);
        lt += __popc(__ballot_sync(0xffffffffu, k < tau));
        eq += __popc(__ballot_sync(0xffffffffu, k == tau));
    }
    if (lane == 0) {
        s_lt[warp] = lt;
        s_eq[warp] = eq;
    }
    __syncthreads();
    if (warp == 0) {
        const unsigned l = __reduce_add_sync(0xffffffffu, s_lt[lane]), e = __reduce_add_sync(0xffffffffu, s_eq[lane]);
        if (lane < ctas) {
            unsigned* d = cluster.map_shared_rank(&s_cta[rank][0], lane);
            d[0] = l;
            d[1] = e;
        }
    }
    if (ctas > 1) cluster.sync();
    else __syncthreads();
    unsigned lt_at = __reduce_add_sync(0xffffffffu, (lane < warp ? s_lt[lane] : 0u) + (lane < rank ? s_cta[lane][0] : 0u));
    unsigned eq_at = __reduce_add_sync(0xffffffffu, (lane < warp ? s_eq[lane] : 0u) + (lane < rank ? s_cta[lane][1] : 0u));
    const unsigned below = (1u << lane) - 1u;
#pragma unroll
    for (int j0 = 0; j0 < per; j0 += 4) {   // 128 consecutive rows
        uint32_t k[4];
        unsigned l = 0, e = 0, lts = 0, eqs = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            k[i] = key(j0 + i);
            const unsigned ml = __ballot_sync(0xffffffffu, k[i] < tau), me = __ballot_sync(0xffffffffu, k[i] == tau);
            l += __popc(ml & below);
            e += __popc(me & below);
            lts += __popc(ml);
            eqs += __popc(me);
        }
        l += lt_at;
        e += eq_at;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (k[i] < tau || (k[i] == tau && e < quota)) rows[l + min(e, quota)] = row(j0 + i);
            l += k[i] < tau;
            e += k[i] == tau;
        }
        lt_at += lts;
        eq_at += eqs;
    }
    if (tau == kProtected && rank == 0) {   // fewer than n rows may go
        unsigned all = __reduce_add_sync(0xffffffffu, lane < ctas ? s_cta[lane][0] : 0u);
        for (int i = all + tid; i < a.n; i += kThreads) rows[i] = -1;
        if (tid == 0) set_status(a.status, PBSA_ERR_DEVICE_CHECK);
    }
}

template <int K>
cudaError_t run(const EvictArgs& a, int ctas, int tiles, cudaStream_t st) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.BH * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_kernel<K>, a, tiles);
}

}  // namespace

cudaError_t launch_kv4_evict(const EvictArgs& a, cudaStream_t st) {
    const int tiles = (a.N + kThreads - 1) / kThreads;   // keys of a thread, with one CTA
    auto cluster = [&](int keys) {
        int ctas = 1;
        while (keys * ctas < tiles) ctas *= 2;
        return ctas;
    };
    // few heads: more CTAs for each, four or eight keys a thread
    if (tiles <= 4 * kMaxCluster && (tiles <= 4 || a.BH * cluster(4) <= kSMs)) return run<4>(a, cluster(4), 0, st);
    if (tiles <= 8 * kMaxCluster && (tiles <= 8 || a.BH * cluster(8) <= kSMs)) return run<8>(a, cluster(8), 0, st);
    if (tiles <= 24 * kMaxCluster) return run<24>(a, cluster(24), 0, st);
    const int per = (tiles + kMaxCluster - 1) / kMaxCluster;
    return run<0>(a, kMaxCluster, (per + 3) / 4 * 4, st);
}

}  // namespace pbsa
