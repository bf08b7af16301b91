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

constexpr int kWarps = 7;                  // warps that compute; an eighth loads
constexpr int kUnit = 16;                  // keys of one tensor-core step: a warp's share of a block
constexpr int kBlock = kWarps * kUnit;     // keys a CTA handles per round: the unit of work
constexpr int kStages = 4;                 // blocks in the ring
constexpr int kMassWarps = 4;
constexpr int kHidden = 0x7fffffff;        // position that no query sees
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Probabilities are kept as 2^(s - m + kShift) in fp16, m the running maximum or up to
// kLag below it: at most 2^15, and what is lost below 2^-24 is under 2^-31 of the largest.
constexpr float kShift = 7.f;
constexpr float kLag = 8.f;

struct AttnArgs {
    Kv4Args k;
    int G, R, tiles8;      // query heads of a key head, rows, groups of 8 rows
    int ctas;              // CTAs that share the keys of one group of rows
    float* part_o;         // [row groups][ctas][2][8 NT][D]
    float2* part_ml;       // [row groups][ctas][2][8 NT]
    float* logits;         // [B Hkv][R][N] base-2 logits (mass of few rows)
    uint2* q_frag;         // [B Hkv][tiles8][D / 16][32] (mass of many rows)
    float* q_fac;          // [B Hkv][tiles8][8]
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

// A block of keys in shared memory, as it lies in the cache.
template <int D>
struct Block {
    uint8_t kc[kBlock][D / 2], vc[kBlock][D / 2], ks[kBlock][D / 16], vs[kBlock][D / 16];
    int32_t pos[kBlock];
};

// What a lane reads of sixteen keys.  Lane 4 g + c holds, of keys g and g + 8, the c-th
// quarter of the key's channels (one load), and, of values 2c, 2c+1, 2c+8, 2c+9, the g-th
// eighth of the channels.
template <int D>
struct Keys {
    uint32_t k[2][D / 32], ks[2];
    int pos[2];
};

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&d)[N], const uint8_t* p) {
    if (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        d[0] = v.x, d[1 % N] = v.y, d[2 % N] = v.z, d[3 % N] = v.w;
    } else if (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        d[0] = v.x, d[1 % N] = v.y;
    } else {
        d[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

template <int D>
__device__ __forceinline__ void load_keys(Keys<D>& x, const uint8_t* kc, const uint8_t* ks, const int32_t* pos, int lane) {
    const int g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int j = g + 8 * r;
        load_words(x.k[r], kc + j * (D / 2) + q * (D / 8));
        if (D == 128) x.ks[r] = *reinterpret_cast<const uint16_t*>(ks + j * 8 + 2 * q);
        else x.ks[r] = ks[j * 4 + q];
        x.pos[r] = pos[j];
    }
}

// Of sixteen keys the first `left` are in use.  A row that holds no token may be anything: its
// position becomes kHidden and its scale zero.
template <int D>
__device__ __forceinline__ void hide_keys(Keys<D>& x, int left, int lane) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
        if (x.pos[r] < 0 || (lane >> 2) + 8 * r >= left) {
            x.pos[r] = kHidden;
            x.ks[r] = 0;
        }
}

// s[n] += K Q^T of sixteen keys and rows 8 n .. 8 n + 7; `q` gives the lane's operands of
// step j and row group n.  Step j contracts channels 32c' + 4j .. + 3 of every quarter c'.
template <int D, int NT, typename QF>
__device__ __forceinline__ void scores(float (&s)[NT][4], const Keys<D>& x, QF q) {
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

__device__ __forceinline__ int used_rows(const AttnArgs& a, int b) {
    return max(0, min(a.k.kv_len[b], a.k.c.capacity));
}

__device__ __forceinline__ int blocks_of(int len) { return (len + kBlock - 1) / kBlock; }

// The work of a group of rows is the list of all blocks of keys, by sequence, key head and
// block (below 2^31 of them).  n = min(ctas, total) CTAs share it in runs of `each` blocks or,
// the first `more` of them, one more.  A warp makes and asks it together: every lane adds up
// the blocks of its share of the sequences.
struct WorkList {
    int total, n, each, more;
    int per, upto, mine;   // sequences of a lane, blocks of the lanes up to this one, and its own

    __device__ __forceinline__ WorkList(const AttnArgs& a, int lane) {
        const int B = a.k.c.B;
        per = (B + 31) / 32;
        mine = 0;
        for (int b = lane * per; b < min(B, (lane + 1) * per); ++b) mine += blocks_of(used_rows(a, b));
        mine *= a.k.c.Hkv;
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
            for (int x = src * per; x < b; ++x) at += blocks_of(used_rows(a, x)) * a.k.c.Hkv;
        return __shfl_sync(0xffffffffu, at, src);
    }

    // The sequence of block w, and the blocks before that sequence.
    __device__ __forceinline__ void find(const AttnArgs& a, int lane, int w, int& b, int& before) const {
        const bool here = upto > w && upto - mine <= w && (lane == 0 || a.k.c.B > 1);
        const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
        int at = upto - mine, bb = lane * per;
        if (here) {
            while (true) {
                const int k = blocks_of(used_rows(a, bb)) * a.k.c.Hkv;
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
        const int n = blocks_of(len);
        h = in_seq / n;
        blk = in_seq - h * n;
    }

    // To the next block, when there are `left` of them.
    __device__ __forceinline__ void next(const AttnArgs& a, int left) {
        if (++blk * kBlock < len) return;
        blk = 0;
        if (++h < a.k.c.Hkv) return;
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

// Four channels of a finished row: v = sum of probabilities times values, relative to 2^mx.
template <int D, typename T>
__device__ __forceinline__ void finish_row(const AttnArgs& a, int b, int hkv, int row, int d, const float4& v, float mx,
                                           float sum) {
    const int t = row / a.G, h = hkv * a.G + row % a.G;
    store4(static_cast<T*>(a.k.out) + (((size_t)b * a.k.T + t) * a.k.c.Hq + h) * D + d, v,
           sum == 0.f ? 0.f : a.k.c.v_unit / sum);
    if (d == 0)
        a.k.lse[((size_t)b * a.k.c.Hq + h) * a.k.T + t] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
}

// A CTA takes a run of the work list for one group of 8 NT rows and goes through it segment by
// segment, a segment being the blocks of one (sequence, key head).  One warp loads: it asks for
// block after block, across segment borders, into a ring in shared memory (bulk copies).  The
// other warps take sixteen of a block's keys each; each has its own running maximum, sum and
// output, which are joined in shared memory at the end of a segment.  A segment that covers
// its head's keys goes straight to the output, the others to the workspace, for join_kernel.
//
// Keys and values are the row operand of the tensor-core steps (S^T = K Q^T, O^T = V^T P^T),
// so that rows come in groups of eight and a code is turned into fp16 once, in the register
// that it is multiplied from.
template <int D, int NT, typename T, bool kLogits>
__global__ void __launch_bounds__(32 * (kWarps + 1), NT == 1 ? 2 : 1) attn_kernel(AttnArgs a) {
    constexpr int kSteps = D / 16, kRows = 8 * NT, kComputing = 32 * kWarps;
    constexpr int kPair = 1;
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ __align__(8) uint64_t s_full[kStages], s_free[kStages];
    __shared__ int s_abort;
    Block<D>* ring = reinterpret_cast<Block<D>*>(sm);
    uint2* q_sm = reinterpret_cast<uint2*>(ring + kStages);          // [kSteps][NT][32], NT > 1
    float* o_sm = reinterpret_cast<float*>(q_sm + (NT == 1 ? 0 : kSteps * NT * 32));   // [kWarps][kRows][D]
    float* m_sm = o_sm + kWarps * kRows * D;                         // [kWarps][kRows]
    float* l_sm = m_sm + kWarps * kRows;                             // [kWarps][kRows]
    float* fac_sm = l_sm + kWarps * kRows;                           // [kRows]
    int* lim_sm = reinterpret_cast<int*>(fac_sm + kRows);            // [kRows]
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), g = lane >> 2, c = lane & 3;
    const int N = a.k.c.capacity, tile0 = blockIdx.y * NT;
    if (threadIdx.x == 32 * kWarps) {
        s_abort = 0;
#pragma unroll
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_free[i], kWarps);
        }
        fence_barrier_init();
    }
    grid_dependency_launch();
    const WorkList list(a, lane);
    if (blockIdx.x >= list.n) return;
    const int w0 = list.first_of(blockIdx.x), total = list.first_of(blockIdx.x + 1) - w0;   // blocks of this CTA
    int b0, before;
    list.find(a, lane, w0, b0, before);
    Cursor at;
    at.start(a, b0, w0 - before);

    if (warp == kWarps) {
        uint32_t stage = 0, phase = 0;
        int n = 0;
        auto load = [&]() {
            const int row = at.blk * kBlock;
            const uint32_t rows = min(kBlock, N - row);
            Block<D>& s = ring[stage];
            const uint32_t bar = smem_u32(&s_full[stage]);
            const size_t first = ((size_t)at.b * a.k.c.Hkv + at.h) * N + row;
            const pbsa_kv4_cache& k = a.k.cache;
            mbar_arrive_expect_tx(&s_full[stage], rows * (D + D / 8 + 4));
            bulk_load(smem_u32(s.kc), k.k_codes + first * (D / 2), rows * (D / 2), bar);
            bulk_load(smem_u32(s.ks), k.k_scales + first * (D / 16), rows * (D / 16), bar);
            bulk_load(smem_u32(s.pos), k.pos + first, rows * 4, bar);
            bulk_load(smem_u32(s.vc), k.v_codes + first * (D / 2), rows * (D / 2), bar);
            bulk_load(smem_u32(s.vs), k.v_scales + first * (D / 16), rows * (D / 16), bar);
            ++n;
            at.next(a, total - n);
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1u;
            }
        };
        // the ring is filled before the other warps are let in
        if (lane == 0)
            while (n < min(kStages, total)) load();
        __syncwarp();
        __syncthreads();
        if (lane == 0) {
            while (n < total && mbar_wait(&s_free[stage], phase ^ 1u, &s_abort, a.k.status)) load();
            // after a wait that ran out: no copy may still be on its way into this CTA's memory
            if (n < total)
                for (int i = max(0, n - kStages); i < n; ++i)
                    mbar_wait_drain(&s_full[i % kStages], (i / kStages) & 1, kWaitLimitNs);
        }
        return;
    }
    __syncthreads();

    bool ok = true;
    uint32_t stage = 0, phase = 0;
    int left = total;   // blocks to go
    // this lane's places in a block
    const uint8_t* my_kc = ring->kc[warp * kUnit];
    const uint8_t* my_ks = ring->ks[warp * kUnit];
    const int32_t* my_pos = ring->pos + warp * kUnit;
    const uint8_t* my_vc = ring->vc[warp * kUnit + 2 * c] + g * (D / 16);
    const uint8_t* my_vs = ring->vs[warp * kUnit + 2 * c] + g * (D / 16) / 8;
    while (left > 0) {
        const int b = at.b, hkv = at.h, len = at.len, blk0 = at.blk, bh = b * a.k.c.Hkv + hkv;
        const int nblk = blocks_of(len), blk1 = min(nblk, blk0 + left);
        float fac1[2];
        int lim1[2];
        uint2 qr[kSteps];
        if (NT == 1) {
            float f;
            load_queries<D, T>(a, b, hkv, tile0, lane, qr, f);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fac1[i] = __shfl_sync(0xffffffffu, f, 4 * (2 * c + i));
                lim1[i] = row_limit(a, b, tile0 * 8 + 2 * c + i);
            }
        } else {
            for (int n = warp; n < NT; n += kWarps) {
                float f;
                load_queries<D, T>(a, b, hkv, tile0 + n, lane, qr, f);
#pragma unroll
                for (int j = 0; j < kSteps; ++j) q_sm[(j * NT + n) * 32 + lane] = qr[j];
                if (c == 0) {
                    fac_sm[8 * n + g] = f;
                    lim_sm[8 * n + g] = row_limit(a, b, (tile0 + n) * 8 + g);
                }
                if (a.q_frag && blk0 == 0 && tile0 + n < a.tiles8) {
                    const size_t tile = (size_t)bh * a.tiles8 + tile0 + n;
#pragma unroll
                    for (int j = 0; j < kSteps; ++j) a.q_frag[(tile * kSteps + j) * 32 + lane] = qr[j];
                    if (c == 0) a.q_fac[tile * 8 + g] = f;
                }
            }
            named_bar_sync(1, kComputing);
        }
        // of row 2c + i of group n: factor from a product to a base-2 logit, largest position seen
        auto fac = [&](int n, int i) -> float { return NT == 1 ? fac1[i] : fac_sm[8 * n + 2 * c + i]; };
        auto lim = [&](int n, int i) -> int { return NT == 1 ? lim1[i] : lim_sm[8 * n + 2 * c + i]; };
        auto qf = [&](int j, int n) -> uint2 { return NT == 1 ? qr[j] : q_sm[(j * NT + n) * 32 + lane]; };
        float* lg = kLogits ? a.logits + ((size_t)bh * a.R + 2 * c) * N + g : nullptr;

        float mref[NT][2], thr[NT][2], l[NT][2], o[NT][kSteps][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mref[n][i] = -INFINITY;   // running maximum - kShift, common to the lanes of a row
                thr[n][i] = -INFINITY;    // products above it raise the maximum: (maximum + kLag) / fac
                l[n][i] = 0.f;            // this lane's share of the sum
            }
#pragma unroll
            for (int j = 0; j < kSteps; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][j][i] = 0.f;
        }

        // kPair blocks at a time: their chains of dependent steps overlap
        for (int blk = blk0; blk < blk1; blk += kPair) {
            const int row = blk * kBlock + warp * kUnit;
            const bool more = kPair == 2 && blk + 1 < blk1;
            const uint32_t stage1 = stage + 1 == kStages ? 0 : stage + 1, phase1 = stage + 1 == kStages ? phase ^ 1u : phase;
            ok = ok && mbar_wait(&s_full[stage], phase, &s_abort, a.k.status);
            if (more) ok = ok && mbar_wait(&s_full[stage1], phase1, &s_abort, a.k.status);
            if (ok && row < len) {
                Keys<D> x[kPair];
                uint32_t at_stage[kPair];
                bool odd = a.k.q_pos || kRows > a.R;   // some row may not see some key
#pragma unroll
                for (int u = 0; u < kPair; ++u) {
                    at_stage[u] = (u ? stage1 : stage) * (uint32_t)sizeof(Block<D>);
                    load_keys(x[u], my_kc + at_stage[u], my_ks + at_stage[u], my_pos + at_stage[u] / 4, lane);
                    odd |= (x[u].pos[0] | x[u].pos[1]) < 0 || row + u * kBlock + kUnit > len || (u && !more);
                }
                // s[u][n][i]: key g + 8 (i >> 1) of block u, row 2c + (i & 1) of group n
                float s[kPair][NT][4];
                uint32_t vmask[kPair][2];   // of the scales of values 2c, 2c+1 and 2c+8, 2c+9
#pragma unroll
                for (int u = 0; u < kPair; ++u) {
                    vmask[u][0] = vmask[u][1] = 0xffffu;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[u][n][i] = 0.f;
                }
                if (__any_sync(0xffffffffu, odd)) {
#pragma unroll
                    for (int u = 0; u < kPair; ++u) {
                        hide_keys(x[u], u && !more ? 0 : len - row - u * kBlock, lane);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (x[u].pos[i >> 1] > lim(n, i & 1)) s[u][n][i] = -INFINITY;
                        // values of rows without a token: scale zero
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const unsigned live = __ballot_sync(0xffffffffu, x[u].pos[i] != kHidden) >> (8 * c);
                            vmask[u][i] = (live & 1u ? 0xffu : 0u) | (live & 16u ? 0xff00u : 0u);
                        }
                    }
                }
                bool grow = false;
#pragma unroll
                for (int u = 0; u < kPair; ++u) scores<D, NT>(s[u], x[u], qf);
#pragma unroll
                for (int u = 0; u < kPair; ++u)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) grow |= fmaxf(s[u][n][i], s[u][n][i + 2]) > thr[n][i];
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float t = fmaxf(s[0][n][i], s[0][n][i + 2]);
                            if (kPair == 2) t = fmaxf(t, fmaxf(s[kPair - 1][n][i], s[kPair - 1][n][i + 2]));
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                            const float mn = t * fac(n, i) - kShift;
                            if (mn > mref[n][i]) {
                                const float k = ex2(mref[n][i] - mn);   // 0 from the initial -inf
                                l[n][i] *= k;
#pragma unroll
                                for (int j = 0; j < kSteps; ++j) {
                                    o[n][j][i] *= k;
                                    o[n][j][i + 2] *= k;
                                }
                                mref[n][i] = mn;
                                thr[n][i] = (mn + kShift + kLag) / fac(n, i);
                            }
                        }
                }
                uint32_t p[kPair][NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float f[2], ref[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        f[i] = fac(n, i);
                        ref[i] = mref[n][i] == -INFINITY ? 0.f : -mref[n][i];   // none seen so far: 2^-inf
                    }
#pragma unroll
                    for (int u = 0; u < kPair; ++u) {
                        if (kLogits && (u == 0 || more)) {   // NT == 1
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                if (2 * c + i < a.R && row + u * kBlock < N) {
                                    float* dst = lg + (size_t)i * N + row + u * kBlock;
                                    dst[0] = s[u][0][i] * f[i];
                                    dst[8] = s[u][0][i + 2] * f[i];
                                }
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            s[u][n][i] = ex2(fmaf(s[u][n][i], f[i & 1], ref[i & 1]));
                            l[n][i & 1] += s[u][n][i];
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const __half2 h = __floats2half2_rn(s[u][n][2 * i], s[u][n][2 * i + 1]);
                            p[u][n][i] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&h));
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < kPair; ++u) {
                    uint32_t v[4][D / 64], vs[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = (i & 1) + 8 * (i >> 1);
                        load_words(v[i], my_vc + at_stage[u] + j * (D / 2));
                        vs[i] = my_vs[at_stage[u] + j * (D / 16)];
                    }
                    const uint32_t vs0 = e4m3x2_to_half2((uint16_t)(__byte_perm(vs[0], vs[1], 0x0040) & vmask[u][0]));
                    const uint32_t vs1 = e4m3x2_to_half2((uint16_t)(__byte_perm(vs[2], vs[3], 0x0040) & vmask[u][1]));
#pragma unroll
                    for (int q = 0; q < D / 64; ++q) {
                        // even and odd channels of the lane's eighth, two keys to a byte
                        uint32_t h[4][4];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t va = v[2 * i][q], vb = v[2 * i + 1][q];
                            const uint32_t even = (va & 0x0f0f0f0fu) | ((vb << 4) & 0xf0f0f0f0u);
                            const uint32_t odds = ((va >> 4) & 0x0f0f0f0fu) | (vb & 0xf0f0f0f0u);
                            e2m1x8_to_half2x4(even, h[2 * i][0], h[2 * i][1], h[2 * i][2], h[2 * i][3]);
                            e2m1x8_to_half2x4(odds, h[2 * i + 1][0], h[2 * i + 1][1], h[2 * i + 1][2], h[2 * i + 1][3]);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t av[4] = {hmul2_u32(h[0][j], vs0), hmul2_u32(h[1][j], vs0),
                                                    hmul2_u32(h[2][j], vs1), hmul2_u32(h[3][j], vs1)};
#pragma unroll
                            for (int n = 0; n < NT; ++n) mma_16816(o[n][4 * q + j], av, p[u][n][0], p[u][n][1]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&s_free[stage]);
                if (more) mbar_arrive(&s_free[stage1]);
            }
            const uint32_t step = more ? 2 : 1;
            stage += step;
            if (stage >= kStages) {
                stage -= kStages;
                phase ^= 1u;
            }
        }

        // join the warps.  o[n][j][i]: channel (D/8) g + 2j + (i >> 1), row 2c + (i & 1) of group n
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float t = l[n][i];
                t += __shfl_xor_sync(0xffffffffu, t, 4);
                t += __shfl_xor_sync(0xffffffffu, t, 8);
                t += __shfl_xor_sync(0xffffffffu, t, 16);
                const int r = 8 * n + 2 * c + i;
                if (g == 0) {
                    m_sm[warp * kRows + r] = mref[n][i];
                    l_sm[warp * kRows + r] = t;
                }
                float* dst = o_sm + ((size_t)warp * kRows + r) * D + g * (D / 8);
#pragma unroll
                for (int j = 0; j < kSteps; ++j)
                    *reinterpret_cast<float2*>(dst + 2 * j) = make_float2(o[n][j][i], o[n][j][i + 2]);
            }
        named_bar_sync(1, kComputing);
        const bool whole = blk0 == 0 && blk1 == nblk;
        const size_t slot = (((size_t)blockIdx.y * a.ctas + blockIdx.x) * 2 + (blk0 == 0)) * kRows;
        for (int e = threadIdx.x; e < kRows * (D / 4); e += kComputing) {
            const int r = e / (D / 4), d = (e % (D / 4)) * 4, qrow = blockIdx.y * kRows + r;
            if (qrow >= a.R) break;
            float mx = -INFINITY;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) mx = fmaxf(mx, m_sm[k * kRows + r]);
            const float base = mx == -INFINITY ? 0.f : mx;
            float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float f = ex2(m_sm[k * kRows + r] - base);
                const float4 y = *reinterpret_cast<const float4*>(o_sm + ((size_t)k * kRows + r) * D + d);
                t.x += f * y.x, t.y += f * y.y, t.z += f * y.z, t.w += f * y.w;
                sum += f * l_sm[k * kRows + r];
            }
            if (whole) {
                finish_row<D, T>(a, b, hkv, qrow, d, t, mx, sum);
            } else {
                *reinterpret_cast<float4*>(a.part_o + (slot + r) * D + d) = t;
                if (d == 0) a.part_ml[slot + r] = make_float2(mx, sum);
            }
        }
        left -= blk1 - blk0;
        if (left > 0) {
            at.blk = blk1 - 1;
            at.next(a, left);
            named_bar_sync(1, kComputing);   // the join has read o_sm
        }
    }
}

// Joins the segments of heads whose keys were shared by several CTAs, and writes the heads
// that have no keys.  One CTA per row: D / 4 lanes hold its channels, PARTS of them in
// parallel take the parts in turn (a long cache of one head has a part per CTA of the GPU).
// It is launched while attn_kernel still runs and waits for it before it reads its parts.
template <int D, int NT, int PARTS, typename T>
__global__ void __launch_bounds__(PARTS * D / 4) join_kernel(AttnArgs a) {
    constexpr int kRows = 8 * NT, kLanes = D / 4;
    __shared__ float4 s_v[PARTS][kLanes];
    __shared__ float s_m[PARTS], s_l[PARTS];
    const int lane = threadIdx.x & 31, bh = blockIdx.x / a.R, qrow = blockIdx.x % a.R;
    const int b = bh / a.k.c.Hkv, hkv = bh % a.k.c.Hkv;
    const int d = (threadIdx.x % kLanes) * 4, part = threadIdx.x / kLanes;
    const WorkList list(a, lane);
    const int n = blocks_of(used_rows(a, b));
    int first = 0, last = 0;
    if (n > 0) {
        const int w0 = list.before(a, lane, b) + hkv * n;
        first = list.cta_of(w0);
        last = list.cta_of(w0 + n - 1);
    }
    if (blockIdx.x == 0)
        for (int x = threadIdx.x; x < a.k.c.B; x += PARTS * kLanes)
            if (a.k.kv_len[x] != used_rows(a, x)) set_status(a.k.status, PBSA_ERR_DEVICE_CHECK);
    grid_dependency_wait();
    grid_dependency_launch();
    if (n > 0 && first == last) return;   // written by its CTA
    // the first CTA's part is its last segment (slot 1), the others' their first (slot 0)
    const size_t base = (size_t)(qrow / kRows) * a.ctas * 2 * kRows + qrow % kRows;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    float mx = -INFINITY, sum = 0.f;
    if (n > 0) {
#pragma unroll 4
        for (int i = first + part; i <= last; i += PARTS) {
            const size_t at = base + ((size_t)2 * i + (i == first)) * kRows;
            const float2 ml = a.part_ml[at];
            const float4 x = *reinterpret_cast<const float4*>(a.part_o + at * D + d);
            const float mn = fmaxf(mx, ml.x), ref = mn == -INFINITY ? 0.f : mn;
            const float f = ex2(mx - ref), k = ex2(ml.x - ref);
            v.x = f * v.x + k * x.x, v.y = f * v.y + k * x.y, v.z = f * v.z + k * x.z, v.w = f * v.w + k * x.w;
            sum = f * sum + k * ml.y;
            mx = mn;
        }
    }
    s_v[part][threadIdx.x % kLanes] = v;
    if (d == 0) {
        s_m[part] = mx;
        s_l[part] = sum;
    }
    __syncthreads();
    if (part > 0) return;
    for (int i = 1; i < PARTS; ++i) mx = fmaxf(mx, s_m[i]);
    const float ref = mx == -INFINITY ? 0.f : mx;
    v = make_float4(0.f, 0.f, 0.f, 0.f);
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        const float k = ex2(s_m[i] - ref);
        const float4 x = s_v[i][threadIdx.x];
        v.x += k * x.x, v.y += k * x.y, v.z += k * x.z, v.w += k * x.w;
        sum += k * s_l[i];
    }
    finish_row<D, T>(a, b, hkv, qrow, d, v, mx, sum);
}

// Masses from the kept logits of at most eight rows: a thread takes four cached rows.
constexpr int kMassThreads = 128;

__global__ void __launch_bounds__(kMassThreads) mass_logits_kernel(AttnArgs a) {
    const int N = a.k.c.capacity, bh = blockIdx.x, b = bh / a.k.c.Hkv, hkv = bh % a.k.c.Hkv;
    const int j = (blockIdx.y * kMassThreads + threadIdx.x) * 4, len = used_rows(a, b);
    grid_dependency_wait();
    if (j >= len) return;
    const float* s = a.logits + (size_t)bh * a.R * N + j;
    const size_t at = (size_t)bh * N + j;
    const int4 pos = *reinterpret_cast<const int4*>(a.k.cache.pos + at);
    float4 mass = *reinterpret_cast<const float4*>(a.k.mass + at);
    float4 v[8];
    float lse[8];
#pragma unroll
    for (int r = 0; r < 8; ++r)
        if (r < a.R) {
            v[r] = *reinterpret_cast<const float4*>(s + (size_t)r * N);
            lse[r] = a.k.lse[((size_t)b * a.k.c.Hq + hkv * a.G + r % a.G) * a.k.T + r / a.G] * kLog2e;
        }
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < 8; ++r)
        if (r < a.R && lse[r] != -INFINITY) {   // a hidden row's logit is -inf: it adds 0
            sum.x += ex2(v[r].x - lse[r]);
            sum.y += ex2(v[r].y - lse[r]);
            sum.z += ex2(v[r].z - lse[r]);
            sum.w += ex2(v[r].w - lse[r]);
        }
    if (j < len && pos.x >= 0) mass.x += sum.x;
    if (j + 1 < len && pos.y >= 0) mass.y += sum.y;
    if (j + 2 < len && pos.z >= 0) mass.z += sum.z;
    if (j + 3 < len && pos.w >= 0) mass.w += sum.w;
    *reinterpret_cast<float4*>(a.k.mass + at) = mass;
}

// Masses of many rows: the scores are formed again (half of the cache's bytes) once the rows'
// lse is known; a warp owns its keys and walks all rows, so that every sum has one order and
// one owner.
template <int D>
__global__ void __launch_bounds__(32 * kMassWarps) mass_kernel(AttnArgs a) {
    constexpr int kSteps = D / 16;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int N = a.k.c.capacity, per_bh = N / (kUnit * kMassWarps);
    const int bh = blockIdx.x / per_bh, b = bh / a.k.c.Hkv, hkv = bh % a.k.c.Hkv;
    grid_dependency_wait();
    const int u = (blockIdx.x % per_bh) * kMassWarps + warp;
    const int len = used_rows(a, b);
    if (u * kUnit >= len) return;
    Keys<D> x;
    const size_t row0 = (size_t)bh * N + (size_t)u * kUnit;
    load_keys(x, a.k.cache.k_codes + row0 * (D / 2), a.k.cache.k_scales + row0 * (D / 16), a.k.cache.pos + row0, lane);
    hide_keys(x, len - u * kUnit, lane);
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
                if (x.pos[k] <= lim) sum[k] += ex2(s[0][i + 2 * k] * fac - lse);
        }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 1);
        sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 2);
        if (c == 0 && x.pos[k] != kHidden) a.k.mass[row0 + g + 8 * k] += sum[k];
    }
}

int row_groups(int R) { return R <= 8 ? 1 : (R <= 16 ? 2 : 4); }

// CTAs per group of rows: together they fill every SM once, and none has less than a block.
int cta_count(const pbsa_kv4_config& c, int R) {
    const int nt = row_groups(R), per_sm = nt == 1 ? 2 : 1;
    const long long groups = (R + 8 * nt - 1) / (8 * nt);
    const long long blocks = (long long)c.B * c.Hkv * ((c.capacity + kBlock - 1) / kBlock);
    long long n = (long long)kSMs * per_sm / groups;
    if (n > blocks) n = blocks;
    return n < 1 ? 1 : (int)n;
}

bool keeps_logits(int R) { return R <= 8; }

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// Workspace: parts of outputs and statistics, then what the masses need.
struct Layout {
    size_t part_o, part_ml, logits, q_frag, q_fac, bytes;

    Layout(const pbsa_kv4_config& c, int R) {
        const size_t bh = (size_t)c.B * c.Hkv, t8 = (R + 7) / 8, nt = row_groups(R);
        const size_t slots = (t8 + nt - 1) / nt * cta_count(c, R) * 2 * 8 * nt;
        size_t at = 0;
        auto take = [&](size_t n) {
            const size_t r = at;
            at += up256(n);
            return r;
        };
        part_o = take(slots * c.D * sizeof(float));
        part_ml = take(slots * sizeof(float2));
        logits = q_frag = q_fac = at;
        if (keeps_logits(R)) {
            logits = take(bh * c.capacity * R * sizeof(float));
        } else {
            q_frag = take(bh * t8 * (c.D / 16) * 32 * sizeof(uint2));
            q_fac = take(bh * t8 * 8 * sizeof(float));
        }
        bytes = at;
    }
};

// Launches a kernel that may start while the one before it in the stream still runs; every
// thread of it waits for that one (grid_dependency_wait) before it reads its results.
cudaError_t launch_after(void (*kernel)(AttnArgs), dim3 grid, int threads, cudaStream_t st, const AttnArgs& a) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int D, int NT, typename T, bool kLogits>
cudaError_t run_attn(const AttnArgs& a, cudaStream_t st) {
    const size_t smem = sizeof(Block<D>) * kStages + (NT == 1 ? 0 : (size_t)(D / 16) * NT * 32 * 8) +
                        (size_t)kWarps * 8 * NT * (D + 2) * 4 + 8 * NT * 8;
    cudaError_t e = cudaFuncSetAttribute(attn_kernel<D, NT, T, kLogits>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int bh = a.k.c.B * a.k.c.Hkv;
    const unsigned groups = (unsigned)((a.R + 8 * NT - 1) / (8 * NT));
    attn_kernel<D, NT, T, kLogits><<<dim3((unsigned)a.ctas, groups), 32 * (kWarps + 1), smem, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // few heads have many parts each
    if (a.ctas >= 8 * bh) e = launch_after(join_kernel<D, NT, 16, T>, dim3((unsigned)(bh * a.R)), 16 * D / 4, st, a);
    else e = launch_after(join_kernel<D, NT, 4, T>, dim3((unsigned)(bh * a.R)), 4 * D / 4, st, a);
    if (e != cudaSuccess || !a.k.mass) return e;
    if (kLogits) {
        const unsigned runs = (unsigned)((a.k.c.capacity + 4 * kMassThreads - 1) / (4 * kMassThreads));
        return launch_after(mass_logits_kernel, dim3((unsigned)bh, runs), kMassThreads, st, a);
    }
    return launch_after(mass_kernel<D>, dim3((unsigned)(bh * (a.k.c.capacity / (kUnit * kMassWarps)))),
                        32 * kMassWarps, st, a);
}

template <int D, typename T>
cudaError_t attn_rows(const AttnArgs& a, cudaStream_t st) {
    switch (row_groups(a.R)) {
        case 1: return a.k.mass ? run_attn<D, 1, T, true>(a, st) : run_attn<D, 1, T, false>(a, st);
        case 2: return run_attn<D, 2, T, false>(a, st);
        default: return run_attn<D, 4, T, false>(a, st);
    }
}

}  // namespace

size_t kv4_attn_workspace(const pbsa_kv4_config& c, int T) { return Layout(c, T * (c.Hq / c.Hkv)).bytes; }

cudaError_t launch_kv4_attn(const Kv4Args& k, cudaStream_t st) {
    AttnArgs a{};
    a.k = k;
    a.G = k.c.Hq / k.c.Hkv;
    a.R = k.T * a.G;
    a.tiles8 = (a.R + 7) / 8;
    a.ctas = cta_count(k.c, a.R);
    const Layout lay(k.c, a.R);
    char* w = static_cast<char*>(k.workspace);
    a.part_o = reinterpret_cast<float*>(w + lay.part_o);
    a.part_ml = reinterpret_cast<float2*>(w + lay.part_ml);
    if (k.mass && keeps_logits(a.R)) {
        a.logits = reinterpret_cast<float*>(w + lay.logits);
    } else if (k.mass) {
        a.q_frag = reinterpret_cast<uint2*>(w + lay.q_frag);
        a.q_fac = reinterpret_cast<float*>(w + lay.q_fac);
    }
    if (k.c.D == 64)
        return k.c.dtype == PBSA_DTYPE_BF16 ? attn_rows<64, __nv_bfloat16>(a, st) : attn_rows<64, __half>(a, st);
    return k.c.dtype == PBSA_DTYPE_BF16 ? attn_rows<128, __nv_bfloat16>(a, st) : attn_rows<128, __half>(a, st);
}

}  // namespace pbsa
