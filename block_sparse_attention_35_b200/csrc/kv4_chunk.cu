// kv4_chunk.cu - attention of many query rows over the 4-bit token cache, on the tcgen05
// tensor cores: a chunk of tokens at once, where the products and not the cache's bytes bound.
//
// Three kernels share the cache-side step: a 128-key tile of codes is turned into fp16 (exact:
// a value has six significant bits) and written to shared memory as a 128-byte-swizzled
// operand tile, once for 256 query rows (attention) or for all rows (masses).
//
//  prep_kernel   the queries in fp16, every row scaled by a power of two, as operand tiles of
//                128 rows, ready for one bulk copy each.
//  chunk_kernel  S = Q K^T, online softmax, O += P V for 256 rows a CTA (two sides of 128);
//                CTAs split the work list as attn_kernel's do and join_kernel joins them.
//  chunk_mass_kernel  S^T = K Q^T with the rows' final sums: a lane of tensor memory is a key, so
//                a key's mass is a sum along four threads' columns, with one owner and one order.
#include "kv4_attn.cuh"

namespace pbsa {

namespace {

constexpr int kHalf = 16384;   // bytes of 128 rows x 64 channels in fp16: one half of a tile

// Instruction descriptor of kind::f16 with fp16 A/B and fp32 accumulate.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
    return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

// Two floats in a 64-bit register: one instruction for both.
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 split(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 32 channels (16 bytes of codes, two scales) of row `row` as four 16-byte chunks of a tile;
// quarter q of 32 channels each.
__device__ __forceinline__ void expand32(uint8_t* tile, int row, int q, const uint4& codes, uint32_t scales) {
    const uint32_t h = e4m3x2_to_half2((uint16_t)scales);
    const uint32_t sc[2] = {__byte_perm(h, h, 0x1010), __byte_perm(h, h, 0x3232)};
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
    uint8_t* half = tile + (q >> 1) * kHalf;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint4 v;
        e2m1x8_to_half2x4(w[i], v.x, v.y, v.z, v.w);
        v.x = hmul2_u32(v.x, sc[i >> 1]), v.y = hmul2_u32(v.y, sc[i >> 1]);
        v.z = hmul2_u32(v.z, sc[i >> 1]), v.w = hmul2_u32(v.w, sc[i >> 1]);
        *reinterpret_cast<uint4*>(half + sw128_offset(row, (q & 1) * 4 + i)) = v;
    }
}

// 16 lanes x 32 columns of tensor memory, as products of mma.sync lie: lane 4 g + c gets, of
// columns 8 j + 2 c and the next one, rows g (d[4 j], d[4 j + 1]) and g + 8 (d[4 j + 2], ..).
__device__ __forceinline__ void tmem_ld_rows16(uint32_t addr, uint32_t (&d)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]), "=r"(d[4]), "=r"(d[5]), "=r"(d[6]), "=r"(d[7]), "=r"(d[8]),
          "=r"(d[9]), "=r"(d[10]), "=r"(d[11]), "=r"(d[12]), "=r"(d[13]), "=r"(d[14]), "=r"(d[15])
        : "r"(addr));
}

// One warp per query row; D / 4 lanes hold it, four channels each.
template <int D, typename T>
__global__ void __launch_bounds__(256) prep_kernel(AttnArgs a) {
    constexpr int kLanes = D / 4;
    const long long row = ((long long)blockIdx.x * 256 + threadIdx.x) / kLanes;
    const int ch4 = threadIdx.x % kLanes, rows = a.tiles128 * 128;
    grid_dependency_launch();
    const int bh = (int)(row / rows), r = (int)(row % rows);
    if (bh >= a.k.c.B * a.k.c.Hkv) return;
    const int b = bh / a.k.c.Hkv, hkv = bh % a.k.c.Hkv;
    float f;
    const uint2 v = scale_query4<D>(a, load_query4<T>(a, b, hkv, r, 4 * ch4), f);
    uint8_t* tile = a.q_tile + ((size_t)bh * a.tiles128 + r / 128) * (128 * D * 2) + (ch4 / 16) * kHalf;
    *reinterpret_cast<uint2*>(tile + sw128_offset(r % 128, (ch4 % 16) / 2) + (ch4 & 1) * 8) = v;
    if (ch4 == 0) a.q_scale[(size_t)bh * rows + r] = f;
}

// ------------------------------------------------------------------------------ masses
// A CTA owns 128 keys of a (sequence, key head) and walks all rows, 128 at a time, through two
// buffers in shared and tensor memory; two groups of four warps take the row tiles in turn.
// Tensor memory is read as products of mma.sync lie, four keys and a quarter of the columns a
// lane: the columns' constants cost a quarter of the shared-memory loads that a lane per key would
// take (141 against 138 us, before the references were products).
// Bound by the exponentials (one a key and row, 16 a clock and SM: 80 us for 1560 rows x 12
// heads x 18752 keys); it takes 135 us: 8.5 us for each 128 rows (three quarters of that rate) and
// 25 for the starts of six rounds of CTAs (expanding the keys).  A quarter of the exponentials as
// polynomials on the FMA pipe changed nothing, here and in chunk_kernel; half of them cost 17 us
// here and 13 there.  The mma.sync form that preceded it took 630 us.
constexpr int kMassGroupThreads = 320;   // 8 warps that compute, one that loads, one that issues

template <int D>
__global__ void __launch_bounds__(kMassGroupThreads, 2) chunk_mass_kernel(AttnArgs a) {
    constexpr int kTile = 128 * D * 2;
    extern __shared__ uint8_t raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* sK = sm;
    uint8_t* sQ = sm + kTile;   // [2][kTile]
    __shared__ __align__(8) uint64_t s_qfull[2], s_qfree[2], s_full[2], s_free[2], s_drain;
    // by group of warps and tile, of two rows: factors, exponents of the products that they are
    // relative to, and these with their sign turned; and limits
    __shared__ __align__(16) float s_col[2][2][64][4];
    __shared__ __align__(8) float s_ref[2][2][128];
    __shared__ int s_lim[2][2][128];
    __shared__ float s_sum[128];
    __shared__ int s_pos[128];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    const int N = a.k.c.capacity, per = (N + 127) / 128, bh = blockIdx.x / per, key0 = (blockIdx.x % per) * 128;
    const int b = bh / a.k.c.Hkv, len = used_rows(a, b);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (key0 >= len) {
        grid_dependency_wait();
        return;
    }
    const int tiles = a.tiles128;
    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_qfull[i], 1);
            mbar_init(&s_qfree[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&s_free[i], 128);
        }
        mbar_init(&s_drain, 1);
        fence_barrier_init();
    }
    if (warp == 9) tmem_alloc(&s_tmem, 256);
    if (warp < 8) {
        int pos = kHidden;
        // two threads to a key, each half of its channels
        const int key = tid & 127, part = tid >> 7;
        const size_t row = (size_t)bh * N + key0 + key;
        const bool here = key0 + key < len;
        if (here) pos = a.k.cache.pos[row];
        if (pos < 0) pos = kHidden;
#pragma unroll
        for (int q = part * (D / 64); q < (part + 1) * (D / 64); ++q) {
            uint4 codes = make_uint4(0, 0, 0, 0);
            uint32_t sc = 0;
            if (pos != kHidden) {
                codes = __ldg(reinterpret_cast<const uint4*>(a.k.cache.k_codes + row * (D / 2)) + q);
                sc = __ldg(reinterpret_cast<const uint16_t*>(a.k.cache.k_scales + row * (D / 16)) + q);
            }
            expand32(sK, key, q, codes, sc);
        }
        if (part == 0) s_pos[key] = pos;
        fence_proxy_async_smem();
    }
    grid_dependency_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const size_t tile0 = (size_t)bh * tiles;

    if (warp == 8) {
        if (lane == 0) {
            int t = 0;
            for (; t < tiles; ++t) {
                const int s = t & 1;
                if (t >= 2 && !mbar_wait(&s_qfree[s], ((t >> 1) - 1) & 1, &s_abort, a.k.status)) break;
                mbar_arrive_expect_tx(&s_qfull[s], kTile);
                bulk_load(smem_u32(sQ + s * kTile), a.q_tile + (tile0 + t) * kTile, kTile, smem_u32(&s_qfull[s]));
            }
            // after a wait that ran out: no copy may still be on its way
            if (t < tiles)
                for (int i = max(0, t - 2); i < t; ++i) mbar_wait_drain(&s_qfull[i & 1], (i >> 1) & 1, kWaitLimitNs);
        }
        __syncwarp();
    } else if (warp == 9) {
        constexpr uint32_t idesc = idesc_f16(128, 128, false);
        const uint32_t k_lo = sdesc_lo(smem_u32(sK), 16);
        bool ok = true;
        for (int t = 0; ok && t < tiles; ++t) {
            const int s = t & 1;
            ok = mbar_wait_warp(&s_qfull[s], (t >> 1) & 1, &s_abort, a.k.status);
            if (ok && t >= 2) ok = mbar_wait_warp(&s_free[s], ((t >> 1) - 1) & 1, &s_abort, a.k.status);
            if (!ok) break;
            tc_fence_after();
            const uint32_t q_lo = sdesc_lo(smem_u32(sQ + s * kTile), 16);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                if (elect_one()) umma_ss(tmem + 128 * s, sdesc_make(k_lo + off), sdesc_make(q_lo + off), idesc, kk > 0);
                __syncwarp();
            }
            if (elect_one()) {
                umma_commit(&s_full[s]);
                umma_commit(&s_qfree[s]);
            }
            __syncwarp();
        }
    } else {
        const int group = warp >> 2, key = tid & 127;
        const uint32_t addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 128 * group;
        // this thread's keys: k0 + 16 h + 8 i, of which it takes every fourth pair of columns
        const int k0 = (warp & 3) * 32 + (lane >> 2), c4 = lane & 3;
        int pos[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) pos[h][i] = s_pos[k0 + 16 * h + 8 * i];
        float sum[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
        bool ok = true;
        // a row's column: its reference and limit; thread i prepares column i of the next tile
        auto column = [&](int t) -> float4 {
            const int r = t * 128 + key;
            float4 c = make_float4(0.f, 0.f, -INFINITY, 0.f);   // past the last row: 2^-inf
            if (t < tiles && r < a.R) c = a.row_ref[(size_t)bh * a.R + r];
            c.w = __int_as_float(row_limit(a, b, r));
            return c;
        };
        float4 next = column(group);
        for (int t = group; t < tiles; t += 2) {
            const int buf = (t >> 1) & 1;
            s_col[group][buf][key >> 1][key & 1] = next.y;
            s_col[group][buf][key >> 1][2 + (key & 1)] = next.z;
            s_ref[group][buf][key] = -next.x;
            s_lim[group][buf][key] = __float_as_int(next.w);
            named_bar_sync(1 + group, 128);   // and the columns two tiles back have been read
            next = column(t + 2);
            ok = ok && mbar_wait_warp(&s_full[group], (t >> 1) & 1, &s_abort, a.k.status);
            if (ok) {
                tc_fence_after();
                uint64_t part[2][2] = {{0, 0}, {0, 0}};
                uint32_t u[2][16];
                float4 col[4];
                uint64_t ref[4];
                int2 lim[4];
                tmem_ld_rows16(addr, u[0]);
#pragma unroll
                for (int k = 0; k < 8; ++k) {   // 32 columns, 16 keys
                    const int h = k & 1, c0 = (k >> 1) * 32;
                    tmem_ld_wait();
                    if (k < 7) {
                        tmem_ld_rows16(addr + ((k + 1) >> 1) * 32 + (static_cast<uint32_t>(((k + 1) & 1) * 16) << 16), u[(k + 1) & 1]);
                    } else {
                        tc_fence_before();
                        mbar_arrive(&s_free[group]);
                    }
                    if (h == 0) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            col[j] = *reinterpret_cast<const float4*>(s_col[group][buf][c0 / 2 + 4 * j + c4]);
                            ref[j] = *reinterpret_cast<const uint64_t*>(&s_ref[group][buf][c0 + 8 * j + 2 * c4]);
                            if (a.k.q_pos) lim[j] = *reinterpret_cast<const int2*>(&s_lim[group][buf][c0 + 8 * j + 2 * c4]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint64_t s2 = pair(__uint_as_float(u[k & 1][4 * j + 2 * i]), __uint_as_float(u[k & 1][4 * j + 2 * i + 1]));
                            float2 x = split(fma2(add2(s2, ref[j]), pair(col[j].x, col[j].y), pair(col[j].z, col[j].w)));
                            x.x = ex2(x.x), x.y = ex2(x.y);
                            if (a.k.q_pos) {
                                x.x = pos[h][i] <= lim[j].x ? x.x : 0.f;
                                x.y = pos[h][i] <= lim[j].y ? x.y : 0.f;
                            }
                            part[h][i] = add2(part[h][i], pair(x.x, x.y));
                        }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 sums = split(part[h][i]);
                        sum[h][i] += sums.x + sums.y;
                    }
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                sum[h][i] += __shfl_xor_sync(0xffffffffu, sum[h][i], 1);
                sum[h][i] += __shfl_xor_sync(0xffffffffu, sum[h][i], 2);
                if (group == 1 && c4 == 0) s_sum[k0 + 16 * h + 8 * i] = sum[h][i];
            }
        named_bar_sync(3, 256);
        if (group == 0 && c4 == 0 && ok) {
            float* mass = a.k.mass + (size_t)bh * N + key0;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int kk = k0 + 16 * h + 8 * i;
                    if (pos[h][i] != kHidden) mass[kk] += sum[h][i] + s_sum[kk];
                }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        // after a wait that gave up, in whichever warp: the products already issued end before
        // tensor memory is released
        if (s_abort) {
            if (elect_one()) umma_commit(&s_drain);
            __syncwarp();
            mbar_wait_drain(&s_drain, 0, 100000000ull);
        }
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

// --------------------------------------------------------------------------- attention
// A CTA (one per SM) goes through its run of the work list in segments of one (sequence, key
// head, group of 256 rows).  Warps 0-3 and 4-7 are the softmax of the two sides (one row a
// thread), 8-11 expand the cache (one key a thread, 128 at a time), 12 and 13 issue the products
// of a side each, 64 keys at a time: QK of step u + 2 follows PV of step u into the same columns,
// so that a side's softmax finds its next scores ready when it is done with the last ones.  Tensor
// memory: two S of 64 columns for each side, O_A, O_B; P (fp16) goes over the first half of its
// own S and is the A operand of PV.  (Products of different shapes may overlap: QK waits until
// PV is done.)
//
// 1560 rows x 12 heads over 18752 rows, D = 128: 230 us for 180 GFLOP (0.78 PFLOP/s).  The
// softmax sets the pace: of the 2300 cycles of a step (at 237 us) its warps waited 200 to 500 for
// scores; the rest was reading them (140), hiding rows without a token (400), the maximum (220)
// and the exponentials (1100, two warps to a scheduler).  With 128 keys a step and one S (and a
// second sweep over it) the kernel took 307 us, with one warp issuing both sides 243, without
// pairs 236.  A last group of at most 128 rows takes nearly as long as a whole one (30 us each).
// Near rows (kNear) keep one multiply-add a score: 239.7 us for such a call without masses, 250.0
// where every warp takes its rows for far ones.
constexpr int kChunkThreads = 14 * 32;
constexpr int kInfo = 4;   // tiles whose key info is kept: a softmax is at most two tiles behind

struct TileInfo {
    float bias[128];     // 0, or -infinity for a row that holds no token
    int pos[128];        // position, or kHidden
    uint32_t live[4];    // by 32 keys: which hold a token
    int newest[4];       // by 32 keys: largest position
};

template <int D, typename T>
__global__ void __launch_bounds__(kChunkThreads, 1) chunk_kernel(AttnArgs a) {
    constexpr int kTile = 128 * D * 2, kQuarters = D / 32;
    extern __shared__ uint8_t raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* sQ = sm;                  // [2 sides][kTile]
    uint8_t* sK = sQ + 2 * kTile;      // [2][kTile]
    uint8_t* sV = sK + 2 * kTile;      // [2][kTile]
    TileInfo* info = reinterpret_cast<TileInfo*>(sV + 2 * kTile);   // [kInfo]
    __shared__ __align__(8) uint64_t s_q[2], s_kfull[2], s_kfree[2], s_vfull[2], s_vfree[2];
    __shared__ __align__(8) uint64_t s_sfull[2][2], s_pfull[2][2], s_pv[2][2], s_drain[2];   // by side, S
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int N = a.k.c.capacity;
    grid_dependency_launch();
    const WorkList list(a, lane);
    if (blockIdx.x >= list.n) {
        grid_dependency_wait();
        return;
    }
    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_kfull[i], 128);
            mbar_init(&s_vfull[i], 128);
            mbar_init(&s_kfree[i], 2);   // an arrival for each side
            mbar_init(&s_vfree[i], 2);
            mbar_init(&s_q[i], 1);
            mbar_init(&s_drain[i], 1);
            for (int j = 0; j < 2; ++j) {
                mbar_init(&s_sfull[i][j], 1);
                mbar_init(&s_pfull[i][j], 128);
                mbar_init(&s_pv[i][j], 1);
            }
        }
        fence_barrier_init();
    }
    if (warp == 12) tmem_alloc(&s_tmem, 512);
    const int w0 = list.first_of(blockIdx.x), total = list.first_of(blockIdx.x + 1) - w0;
    int b0, before;
    list.find(a, lane, w0, b0, before);
    Cursor at;
    at.start(a, b0, w0 - before);
    grid_dependency_wait();   // the queries' tiles
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return mbar_wait_warp(bar, parity, &s_abort, a.k.status);
    };

    // A segment: what every role needs of it; and the step to the next one.
    struct Segment {
        int b, hkv, len, blk0, bh, row0, nblk, tiles, sides;
    };
    int left = total;
    uint32_t tile = 0;             // tiles so far
    auto segment = [&]() -> Segment {
        Segment s;
        s.b = at.b, s.len = at.len, s.blk0 = at.blk;
        s.hkv = at.h / a.groups;
        s.bh = s.b * a.k.c.Hkv + s.hkv;
        s.row0 = (at.h - s.hkv * a.groups) * kChunkRows;
        s.nblk = blocks_of(a, s.len);
        s.tiles = min(s.nblk - s.blk0, left);
        s.sides = s.row0 + 128 < a.R ? 2 : 1;
        return s;
    };
    auto finish = [&](const Segment& s) {
        tile += s.tiles;
        left -= s.tiles;
        if (left > 0) {
            at.blk = s.blk0 + s.tiles - 1;
            at.next(a, left);
        }
        tc_fence_before();
        __syncthreads();   // the segment's operands and sums have been read
        tc_fence_after();
    };

    if (warp >= 8) {
        if (warp >= 12) {
            // ------------------------------------------------- queries, and the products
            const int x = warp - 12;
            constexpr uint32_t idesc_qk = idesc_f16(128, 64, false), idesc_pv = idesc_f16(128, D, true);
            uint32_t n_mine = 0;   // tiles so far of this side (the second rests in a group of at most 128 rows)
            int n_seg = 0;
            while (left > 0) {
                const Segment s = segment();
                if (x < s.sides) {
                    const int steps = 2 * s.tiles, ends = 3 - s.sides;   // arrivals that free a tile
                    if (ok) {
                        if (elect_one()) {
                            mbar_arrive_expect_tx(&s_q[x], kTile);
                            bulk_load(smem_u32(sQ + x * kTile), a.q_tile + ((size_t)s.bh * a.tiles128 + s.row0 / 128 + x) * kTile,
                                      kTile, smem_u32(&s_q[x]));
                        }
                        __syncwarp();
                        ok = wait(&s_q[x], n_seg & 1);
                        // after a wait that gave up: the copy may still be on its way
                        if (!ok) mbar_wait_drain(&s_q[x], n_seg & 1, kWaitLimitNs);
                    }
                    const uint32_t q_lo = sdesc_lo(smem_u32(sQ + x * kTile), 16);
                    auto qk = [&](int u) {   // S of step u
                        const uint32_t t = tile + u / 2, st = t & 1;
                        ok = ok && wait(&s_kfull[st], (t >> 1) & 1);
                        if (!ok) return;
                        tc_fence_after();
                        const uint32_t k_lo = sdesc_lo(smem_u32(sK + st * kTile + (u & 1) * (kHalf / 2)), 16);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                            if (elect_one())
                                umma_ss(tmem + 128 * x + 64 * (u & 1), sdesc_make(q_lo + off), sdesc_make(k_lo + off), idesc_qk, kk > 0);
                            __syncwarp();
                        }
                        if (elect_one()) {
                            umma_commit(&s_sfull[x][u & 1]);
                            if (u & 1)
                                for (int i = 0; i < ends; ++i) umma_commit(&s_kfree[st]);
                        }
                        __syncwarp();
                    };
                    qk(0);
                    qk(1);
                    for (int u = 0; ok && u < steps; ++u) {
                        // O += P V of step u
                        const uint32_t t = tile + u / 2, st = t & 1, parity = (n_mine + u / 2) & 1;
                        ok = wait(&s_pfull[x][u & 1], parity) && wait(&s_vfull[st], (t >> 1) & 1);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t v_lo = sdesc_lo(smem_u32(sV + st * kTile), kHalf) + (u & 1) * 4 * 128;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            if (elect_one())
                                umma_ts(tmem + 256 + 128 * x, tmem + 128 * x + 64 * (u & 1) + kk * 8, sdesc_make(v_lo + kk * 128),
                                        idesc_pv, (u > 0 || kk > 0) ? 1u : 0u);
                            __syncwarp();
                        }
                        if (elect_one()) {
                            umma_commit(&s_pv[x][u & 1]);
                            if (u & 1)
                                for (int i = 0; i < ends; ++i) umma_commit(&s_vfree[st]);
                        }
                        __syncwarp();
                        // S of step u + 2 takes the columns of P of step u: only once PV has read them
                        if (u + 2 < steps) {
                            ok = wait(&s_pv[x][u & 1], parity);
                            qk(u + 2);
                        }
                    }
                    n_mine += s.tiles;
                    ++n_seg;
                }
                finish(s);
            }
        } else {
            // -------------------------------------------------- the cache, into operands
            while (left > 0) {
                const Segment s = segment();
                const int key = tid - 256;
                uint4 kc[kQuarters], vc[kQuarters];
                uint32_t ks[kQuarters], vs[kQuarters];
                int pos;
                auto load = [&](int blk) {
                    const int j = blk * 128 + key;
                    const size_t row = (size_t)s.bh * N + j;
                    pos = j < s.len ? __ldg(a.k.cache.pos + row) : -1;
#pragma unroll
                    for (int q = 0; q < kQuarters; ++q) {
                        kc[q] = vc[q] = make_uint4(0, 0, 0, 0);
                        ks[q] = vs[q] = 0;
                    }
                    if (j < s.len) {
#pragma unroll
                        for (int q = 0; q < kQuarters; ++q) {
                            kc[q] = __ldg(reinterpret_cast<const uint4*>(a.k.cache.k_codes + row * (D / 2)) + q);
                            vc[q] = __ldg(reinterpret_cast<const uint4*>(a.k.cache.v_codes + row * (D / 2)) + q);
                            ks[q] = __ldg(reinterpret_cast<const uint16_t*>(a.k.cache.k_scales + row * (D / 16)) + q);
                            vs[q] = __ldg(reinterpret_cast<const uint16_t*>(a.k.cache.v_scales + row * (D / 16)) + q);
                        }
                    }
                };
                load(s.blk0);
                for (int i = 0; i < s.tiles; ++i) {
                    const uint32_t t = tile + i;
                    const int st = t & 1;
                    const bool here = pos >= 0;
                    if (ok && t >= 2) ok = wait(&s_kfree[st], ((t >> 1) - 1) & 1);
                    if (!ok) break;
                    TileInfo& inf = info[t % kInfo];
                    inf.bias[key] = here ? 0.f : -INFINITY;
                    inf.pos[key] = here ? pos : kHidden;
                    const unsigned live = __ballot_sync(0xffffffffu, here);
                    const int newest = __reduce_max_sync(0xffffffffu, here ? pos : -1);
                    if (lane == 0) {
                        inf.live[key >> 5] = live;
                        inf.newest[key >> 5] = newest;
                    }
#pragma unroll
                    for (int q = 0; q < kQuarters; ++q) expand32(sK + st * kTile, key, q, kc[q], here ? ks[q] : 0u);
                    fence_proxy_async_smem();
                    mbar_arrive(&s_kfull[st]);
                    if (t >= 2) ok = wait(&s_vfree[st], ((t >> 1) - 1) & 1);
                    if (!ok) break;
#pragma unroll
                    for (int q = 0; q < kQuarters; ++q) expand32(sV + st * kTile, key, q, vc[q], here ? vs[q] : 0u);
                    fence_proxy_async_smem();
                    mbar_arrive(&s_vfull[st]);
                    if (i + 1 < s.tiles) load(s.blk0 + i + 1);
                }
                finish(s);
            }
        }
    } else {
        // ------------------------------------------------------------------- softmax
        const int x = warp >> 2;
        uint32_t n_mine = 0;   // tiles so far of this side
        while (left > 0) {
            const Segment s = segment();
            if (x < s.sides) {
                const int r = s.row0 + tid;
                const uint32_t lane_at = static_cast<uint32_t>((warp & 3) * 32) << 16;
                const uint32_t o_at = tmem + lane_at + 256 + 128 * x;
                const float fac = a.q_scale[((size_t)s.bh * a.tiles128) * 128 + r];
                const int lim = row_limit(a, s.b, r);
                const float lag = kLag / fac;
                float ref = 0.f, thr = -INFINITY, l = 0.f;   // ref, thr: as in attn_kernel
                float c0 = kShift;                           // near rows: the exponent of a product of 0
                bool far = false;                            // some row of the warp is not near (kNear)
                for (int u = 0; ok && u < 2 * s.tiles; ++u) {
                    const int j = u & 1;
                    ok = wait(&s_sfull[x][j], (n_mine + u / 2) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t s_at = tmem + lane_at + 128 * x + 64 * j;
                    uint32_t raw_s[2][32];
                    tmem_ld32(s_at, raw_s[0]);
                    tmem_ld32(s_at + 32, raw_s[1]);
                    const TileInfo& inf = info[(tile + u / 2) % kInfo];
                    const int newest = max(inf.newest[2 * j], inf.newest[2 * j + 1]);
                    // some row of this warp may not see some token of the step, or none has one (rows
                    // past the last are never read back).  Elsewhere every row sees a token, and
                    // adding -infinity to what a NaN query made of an empty row costs nothing more.
                    const bool causal = __any_sync(0xffffffffu, r < a.R && (newest > lim || newest < 0));
                    tmem_ld_wait();
                    float v[64];
#pragma unroll
                    for (int e = 0; e < 64; ++e) v[e] = __uint_as_float(raw_s[e >> 5][e & 31]);
                    // -infinity for what the row does not see
                    if (causal) {
#pragma unroll
                        for (int e = 0; e < 64; e += 4) {
                            const int4 q = *reinterpret_cast<const int4*>(&inf.pos[64 * j + e]);
                            v[e] = q.x <= lim ? v[e] : -INFINITY;
                            v[e + 1] = q.y <= lim ? v[e + 1] : -INFINITY;
                            v[e + 2] = q.z <= lim ? v[e + 2] : -INFINITY;
                            v[e + 3] = q.w <= lim ? v[e + 3] : -INFINITY;
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            if (inf.live[2 * j + c] != 0xffffffffu) {
#pragma unroll
                                for (int e = 32 * c; e < 32 * c + 32; e += 4) {
                                    const float4 q = *reinterpret_cast<const float4*>(&inf.bias[64 * j + e]);
                                    const float2 y = split(add2(pair(v[e], v[e + 1]), pair(q.x, q.y)));
                                    const float2 z = split(add2(pair(v[e + 2], v[e + 3]), pair(q.z, q.w)));
                                    v[e] = y.x, v[e + 1] = y.y, v[e + 2] = z.x, v[e + 3] = z.y;
                                }
                            }
                    }
                    float top[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                    for (int e = 4; e < 64; e += 8) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) top[k] = fmaxf(top[k], e + 4 + k < 64 ? fmaxf(v[e + k], v[e + 4 + k]) : v[e + k]);
                    }
                    const float t = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                    const bool grow = t > thr;
                    if (__any_sync(0xffffffffu, grow)) {
                        const float k = !grow ? 1.f : (thr == -INFINITY ? 0.f : ex2((ref - t) * fac));
                        if (u > 0) {
                            ok = wait(&s_pv[x][(u - 1) & 1], (n_mine + (u - 1) / 2) & 1);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D / 16; ++c) {
                                uint32_t y[16];
                                tmem_ld16(o_at + 16 * c, y);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * k);
                                tmem_st16(o_at + 16 * c, y);
                            }
                            tmem_st_wait();
                        }
                        if (grow) {
                            l *= k;
                            ref = t;
                            thr = __fadd_rd(t, lag);
                        }
                        far = __any_sync(0xffffffffu, fabsf(ref * fac) >= kNear);
                        c0 = far ? kShift : fmaf(-ref, fac, kShift);
                    }
                    if (far) {
                        const uint64_t m2 = pair(-ref, -ref);
#pragma unroll
                        for (int e = 0; e < 64; e += 2) {
                            const float2 y = split(add2(pair(v[e], v[e + 1]), m2));
                            v[e] = y.x, v[e + 1] = y.y;
                        }
                    }
                    const uint64_t fac2 = pair(fac, fac), c2 = pair(c0, c0);
                    uint64_t part[2] = {0, 0};
                    uint32_t p[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        float2 y = split(fma2(pair(v[2 * e], v[2 * e + 1]), fac2, c2));
                        y.x = ex2(y.x), y.y = ex2(y.y);
                        part[e & 1] = add2(part[e & 1], pair(y.x, y.y));
                        const __half2 h = __floats2half2_rn(y.x, y.y);
                        p[e] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                    tmem_st32(s_at, p);   // over products that have been read
                    const float2 sums = split(add2(part[0], part[1]));
                    l += sums.x + sums.y;
                    tmem_st_wait();
                    tc_fence_before();
                    mbar_arrive(&s_pfull[x][j]);
                }
                if (ok) ok = wait(&s_pv[x][1], (n_mine + s.tiles - 1) & 1);   // an even number of steps
                if (ok) {
                    tc_fence_after();
                    const bool whole = s.blk0 == 0 && s.tiles == s.nblk;
                    const size_t slot = ((size_t)blockIdx.x * 2 + (s.blk0 == 0)) * kChunkRows + tid;
                    const int tt = r / a.G, h = s.hkv * a.G + r - tt * a.G;
                    T* out = static_cast<T*>(a.k.out) + (((size_t)s.b * a.k.T + tt) * a.k.c.Hq + h) * D;
                    const float inv = l == 0.f ? 0.f : a.k.c.v_unit / l;
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t v[32];
                        tmem_ld32(o_at + 32 * c, v);
                        tmem_ld_wait();
                        if (r < a.R) {
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                float4 y = make_float4(__uint_as_float(v[e]), __uint_as_float(v[e + 1]),
                                                       __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
                                if (l == 0.f) y = make_float4(0.f, 0.f, 0.f, 0.f);
                                if (whole) store4(out + 32 * c + e, y, inv);
                                else *reinterpret_cast<float4*>(a.part_o + slot * D + 32 * c + e) = y;
                            }
                        }
                    }
                    if (r < a.R) {
                        if (whole) finish_sum(a, s.b, s.hkv, r, tt, h, ref, fac, l);
                        else a.part_ml[slot] = make_float4(thr == -INFINITY ? -INFINITY : ref, l, fac, 0.f);
                    }
                }
                n_mine += s.tiles;
            }
            finish(s);
        }
    }
    tc_fence_before();
    __syncthreads();
    // after a wait that gave up, in whichever warp: the products already issued, by either of the
    // two warps that issue, end before tensor memory is released
    if (s_abort) {
        if (warp >= 12) {
            if (elect_one()) umma_commit(&s_drain[warp - 12]);
            __syncwarp();
            mbar_wait_drain(&s_drain[warp - 12], 0, 100000000ull);
        }
        __syncthreads();
    }
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

cudaError_t launch_chunk_attn(const AttnArgs& a, cudaStream_t st) {
    auto run = [&](auto prep, auto kernel, int D) -> cudaError_t {
        const long long threads = (long long)a.k.c.B * a.k.c.Hkv * a.tiles128 * 128 * (D / 4);
        prep<<<(unsigned)((threads + 255) / 256), 256, 0, st>>>(a);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        const size_t smem = 6 * 128 * D * 2 + kInfo * sizeof(TileInfo) + 1024;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        return launch_after(kernel, dim3((unsigned)a.ctas), kChunkThreads, smem, st, a);
    };
    const bool bf16 = a.k.c.dtype == PBSA_DTYPE_BF16;
    if (a.k.c.D == 64)
        return bf16 ? run(prep_kernel<64, __nv_bfloat16>, chunk_kernel<64, __nv_bfloat16>, 64)
                    : run(prep_kernel<64, __half>, chunk_kernel<64, __half>, 64);
    return bf16 ? run(prep_kernel<128, __nv_bfloat16>, chunk_kernel<128, __nv_bfloat16>, 128)
                : run(prep_kernel<128, __half>, chunk_kernel<128, __half>, 128);
}

cudaError_t launch_chunk_mass(const AttnArgs& a, cudaStream_t st) {
    auto run = [&](auto kernel, int D) -> cudaError_t {
        const int smem = 3 * 128 * D * 2 + 1024;
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        const dim3 grid((unsigned)(a.k.c.B * a.k.c.Hkv * ((a.k.c.capacity + 127) / 128)));
        return launch_after(kernel, grid, kMassGroupThreads, (size_t)smem, st, a);
    };
    return a.k.c.D == 64 ? run(chunk_mass_kernel<64>, 64) : run(chunk_mass_kernel<128>, 128);
}

}  // namespace pbsa
