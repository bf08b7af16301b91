// kv4_attn.cu - attention of query tokens over the 4-bit token cache.
//
//   s_rj = q_r . k_j / sqrt(D) over the rows j that query r sees,
//   out_r = sum_j e^(s_rj) v_j / sum_j e^(s_rj),   lse_r = log sum_j e^(s_rj),
//   mass_j += sum_r e^(s_rj - lse_r).
#include "kv4_attn.cuh"

namespace pbsa {

namespace {

constexpr int kWarps = 7;      // warps that compute; an eighth loads
constexpr int kUnit = 16;      // keys of one tensor-core step: a warp's share of a block
constexpr int kBlock = kWarps * kUnit;
constexpr int kStages = 4;     // blocks in the ring
constexpr int kMassWarps = 4;
constexpr int kMassRun = 4, kMassFull = 16 * kSMs * kMassWarps;   // see run_attn

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

// A CTA takes a run of the work list and goes through it segment by segment, a segment being
// the blocks of one (sequence, key head) and all of its rows, at most 8 NT: there is one group of
// rows, and the cursor's head is the key head.  One warp asks for block after
// block, across segment borders, into a ring in shared memory (bulk copies).  The others take
// sixteen of a block's keys each; each has its own running maximum, sum and output, which are
// joined in shared memory at the end of a segment.  A segment that covers its head's keys goes
// straight to the output, the others to the workspace, for join_kernel.
//
// Keys and values are the row operand of the tensor-core steps (S^T = K Q^T, O^T = V^T P^T),
// so that rows come in groups of eight and a code is turned into fp16 once, in the register
// that it is multiplied from.
//
// What bounds it (D = 128, L2 cold).  A step of sixteen keys is 2.4 KB and 338 instructions of a
// warp, 163 of them on the ALU pipe that takes one every other cycle (64 conversions of code
// pairs): with fourteen computing warps an SM, long caches stream at 4.7 TB/s, three quarters of
// the copy rate.  Without any arithmetic the same ring streams at 7.4 TB/s, so the ring does not
// bound it.  Short calls are latency.
//   131072 rows x 4 heads, 8 query rows: 30 us a call (77.6 MB).  4.0 of them without a key (two
//   launches), 6.8 more for the first block of every CTA and the join of 74 parts, 1.0 to 1.2 for
//   each of the 15 blocks after it.
//   32 sequences x 8 heads of 4224 rows, 4 query rows: 50 us (160 MB); of ragged lengths (4200 on
//   average) 58, as CTAs on the short ones end a segment every few blocks, with its join in shared
//   memory and new queries, 2 to 3 us each.  One query row in place of four: the same.  Masses
//   add 8 (kept products and the pass over them).
//   4096 rows x 12 heads, 1 row: 11.8 us.
// Measured and left: eight computing warps that issue the loads in turn, 33.7 against 30.7 us for
// each further 155 MB; two steps a warp at a time, whose chains overlap, and nine computing warps
// with the queries in shared memory, neither faster.
template <int D, int NT, typename T, bool kLogits>
__global__ void __launch_bounds__(32 * (kWarps + 1), NT == 1 ? 2 : 1) attn_kernel(AttnArgs a) {
    constexpr int kSteps = D / 16, kRows = 8 * NT, kThreads = 32 * kWarps;
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ __align__(8) uint64_t s_full[kStages], s_free[kStages];
    __shared__ int s_abort;
    Block<D>* ring = reinterpret_cast<Block<D>*>(sm);
    uint2* q_sm = reinterpret_cast<uint2*>(ring + kStages);               // [kSteps][NT][32]
    float* o_sm = reinterpret_cast<float*>(q_sm + kSteps * NT * 32);      // [kWarps][kRows][D]
    float* m_sm = o_sm + kWarps * kRows * D;                              // [kWarps][kRows]
    float* l_sm = m_sm + kWarps * kRows;                                  // [kWarps][kRows]
    float* join_fac = l_sm + kWarps * kRows;                              // [kRows]: the segment's, for its end
    float* fac_sm = join_fac + kRows;                                     // [kRows]
    int* lim_sm = reinterpret_cast<int*>(fac_sm + kRows);                 // [kRows]
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), g = lane >> 2, c = lane & 3;
    const int N = a.k.c.capacity;
    if (threadIdx.x == kThreads) {
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

    uint32_t stage = 0, phase = 0;
    if (warp == kWarps) {
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
        // it made the barriers and fills the ring before the other warps are let in
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

    bool ok = true;
    int n_use = 0;   // blocks so far
    // this lane's places in a block
    const uint8_t* my_kc = ring->kc[warp * kUnit];
    const uint8_t* my_ks = ring->ks[warp * kUnit];
    const int32_t* my_pos = ring->pos + warp * kUnit;
    const uint8_t* my_vc = ring->vc[warp * kUnit + 2 * c] + g * (D / 16);
    const uint8_t* my_vs = ring->vs[warp * kUnit + 2 * c] + g * (D / 16) / 8;
    for (bool first = true; n_use < total; first = false) {
        const int b = at.b, hkv = at.h, len = at.len, blk0 = at.blk;
        const int bh = b * a.k.c.Hkv + hkv;
        const int nblk = blocks_of(a, len), blk1 = min(nblk, blk0 + total - n_use);
        // queries into operand order, D / 4 lanes to a row: lane 4 g + c of step j and row group
        // n holds row 8 n + g's channels c D / 4 + 4 j .. + 3
#pragma unroll
        for (int r0 = 0; r0 < kRows; r0 += kThreads / (D / 4)) {
            const int r = r0 + (int)threadIdx.x / (D / 4), ch4 = threadIdx.x % (D / 4);
            float f;
            const uint2 v = scale_query4<D>(a, load_query4<T>(a, b, hkv, r, 4 * ch4), f);
            const int j = ch4 % kSteps, slot = (r & 7) * 4 + ch4 / kSteps;
            if (r < kRows) {
                q_sm[(j * NT + r / 8) * 32 + slot] = v;
                if (ch4 == 0) {
                    fac_sm[r] = f;
                    lim_sm[r] = row_limit(a, b, r);
                }
                if (a.q_frag && blk0 == 0 && r / 8 < a.tiles8) {
                    const size_t to = (size_t)bh * a.tiles8 + r / 8;
                    a.q_frag[(to * kSteps + j) * 32 + slot] = v;
                }
            }
        }
        if (first) __syncthreads();   // with the loading warp: the barriers are made
        else named_bar_sync(1, kThreads);
        uint2 qr[NT == 1 ? kSteps : 1];
        float fac1[2];
        int lim1[2];
        if (NT == 1) {
#pragma unroll
            for (int j = 0; j < kSteps; ++j) qr[NT == 1 ? j : 0] = q_sm[j * 32 + lane];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fac1[i] = fac_sm[2 * c + i];
                lim1[i] = lim_sm[2 * c + i];
            }
        }
        // of row 2c + i of group n: factor from a product to a base-2 logit, largest position seen
        auto fac = [&](int n, int i) -> float { return NT == 1 ? fac1[i] : fac_sm[8 * n + 2 * c + i]; };
        auto lim = [&](int n, int i) -> int { return NT == 1 ? lim1[i] : lim_sm[8 * n + 2 * c + i]; };
        auto qf = [&](int j, int n) -> uint2 { return NT == 1 ? qr[NT == 1 ? j : 0] : q_sm[(j * NT + n) * 32 + lane]; };
        const bool choosy = a.k.q_pos;   // some row may not see some key (rows past the last, zeros, may see all)
        float* lg = kLogits ? a.logits + ((size_t)bh * a.R + 2 * c) * N + g : nullptr;

        float ref[NT][2], thr[NT][2], l[NT][2], o[NT][kSteps][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                ref[n][i] = 0.f;          // largest product (with the lag), common to the lanes of a row
                thr[n][i] = -INFINITY;    // products above it raise it: ref + kLag / fac; -inf: none seen so far
                l[n][i] = 0.f;            // this lane's share of the sum
            }
#pragma unroll
            for (int j = 0; j < kSteps; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][j][i] = 0.f;
        }

        for (int blk = blk0; blk < blk1; ++blk) {
            const int row = blk * kBlock + warp * kUnit;
            ok = ok && mbar_wait_warp(&s_full[stage], phase, &s_abort, a.k.status);
            if (ok && row < len) {
                const uint32_t at_stage = stage * (uint32_t)sizeof(Block<D>);
                Keys<D> x;
                load_keys(x, my_kc + at_stage, my_ks + at_stage, my_pos + at_stage / 4, lane);
                uint32_t v[4][D / 64], vs[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = (i & 1) + 8 * (i >> 1);
                    load_words(v[i], my_vc + at_stage + j * (D / 2));
                    vs[i] = my_vs[at_stage + j * (D / 16)];
                }
                // s[n][i]: key g + 8 (i >> 1), row 2c + (i & 1) of group n
                float s[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
                uint32_t vmask[2] = {0xffffu, 0xffffu};   // of the scales of values 2c, 2c+1 and 2c+8, 2c+9
                const bool hide = __any_sync(0xffffffffu, (x.pos[0] | x.pos[1]) < 0) || row + kUnit > len || choosy;
                if (hide) {
                    hide_keys(x, len - row, lane);
                    // values of rows without a token: scale zero
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const unsigned live = __ballot_sync(0xffffffffu, x.pos[i] != kHidden) >> (8 * c);
                        vmask[i] = (live & 1u ? 0xffu : 0u) | (live & 16u ? 0xff00u : 0u);
                    }
                }
                scores<D, NT>(s, x, qf);
                // over the products, not under them: those of a padded query may be NaN
                if (hide) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (x.pos[i >> 1] > lim(n, i & 1)) s[n][i] = -INFINITY;
                }
                bool grow = false;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) grow |= fmaxf(s[n][i], s[n][i + 2]) > thr[n][i];
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float t = fmaxf(s[n][i], s[n][i + 2]);
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                            const bool none = thr[n][i] == -INFINITY;
                            if (t > (none ? -INFINITY : ref[n][i])) {
                                const float k = none ? 0.f : ex2((ref[n][i] - t) * fac(n, i));
                                l[n][i] *= k;
#pragma unroll
                                for (int j = 0; j < kSteps; ++j) {
                                    o[n][j][i] *= k;
                                    o[n][j][i + 2] *= k;
                                }
                                ref[n][i] = t;
                                thr[n][i] = __fadd_rd(t, kLag / fac(n, i));
                            }
                        }
                }
                uint32_t p[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float f[2] = {fac(n, 0), fac(n, 1)};
                    if (kLogits) {   // NT == 1
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (2 * c + i < a.R) {
                                float* dst = lg + (size_t)i * N + row;
                                dst[0] = s[0][i];
                                dst[8] = s[0][i + 2];
                            }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s[n][i] = ex2(fmaf(s[n][i] - ref[n][i & 1], f[i & 1], kShift));
                        l[n][i & 1] += s[n][i];
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const __half2 h = __floats2half2_rn(s[n][2 * i], s[n][2 * i + 1]);
                        p[n][i] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&h));
                    }
                }
                const uint32_t vs0 = e4m3x2_to_half2((uint16_t)(__byte_perm(vs[0], vs[1], 0x0040) & vmask[0]));
                const uint32_t vs1 = e4m3x2_to_half2((uint16_t)(__byte_perm(vs[2], vs[3], 0x0040) & vmask[1]));
#pragma unroll
                for (int q = 0; q < D / 64; ++q) {
                    // even and odd channels of the lane's eighth, two keys to a byte
                    uint32_t h[4][4];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t va = v[2 * i][q], vb = v[2 * i + 1][q];
                        const uint32_t even = (va & 0x0f0f0f0fu) | ((vb << 4) & 0xf0f0f0f0u);
                        const uint32_t odd = ((va >> 4) & 0x0f0f0f0fu) | (vb & 0xf0f0f0f0u);
                        e2m1x8_to_half2x4(even, h[2 * i][0], h[2 * i][1], h[2 * i][2], h[2 * i][3]);
                        e2m1x8_to_half2x4(odd, h[2 * i + 1][0], h[2 * i + 1][1], h[2 * i + 1][2], h[2 * i + 1][3]);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t av[4] = {hmul2_u32(h[0][j], vs0), hmul2_u32(h[1][j], vs0),
                                                hmul2_u32(h[2][j], vs1), hmul2_u32(h[3][j], vs1)};
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_16816(o[n][4 * q + j], av, p[n][0], p[n][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_free[stage]);
            ++n_use;
            if (++stage == kStages) {
                stage = 0;
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
                    m_sm[warp * kRows + r] = thr[n][i] == -INFINITY ? -INFINITY : ref[n][i];
                    l_sm[warp * kRows + r] = t;
                    if (warp == 0) join_fac[r] = fac(n, i);
                }
                float* dst = o_sm + ((size_t)warp * kRows + r) * D + g * (D / 8);
#pragma unroll
                for (int j = 0; j < kSteps; ++j)
                    *reinterpret_cast<float2*>(dst + 2 * j) = make_float2(o[n][j][i], o[n][j][i + 2]);
            }
        named_bar_sync(1, kThreads);
        const bool whole = blk0 == 0 && blk1 == nblk;
        const size_t slot = ((size_t)blockIdx.x * 2 + (blk0 == 0)) * kRows;
        for (int e = threadIdx.x; e < kRows * (D / 4); e += kThreads) {
            const int r = e / (D / 4), d = (e % (D / 4)) * 4;
            if (r >= a.R) break;
            float mx = -INFINITY;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) mx = fmaxf(mx, m_sm[k * kRows + r]);
            const float base = mx == -INFINITY ? 0.f : mx, fr = join_fac[r];
            float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float f = ex2((m_sm[k * kRows + r] - base) * fr);
                const float4 y = *reinterpret_cast<const float4*>(o_sm + ((size_t)k * kRows + r) * D + d);
                t.x += f * y.x, t.y += f * y.y, t.z += f * y.z, t.w += f * y.w;
                sum += f * l_sm[k * kRows + r];
            }
            if (whole) {
                finish_row<D, T>(a, b, hkv, r, d, t, mx, fr, sum);
            } else {
                *reinterpret_cast<float4*>(a.part_o + (slot + r) * D + d) = t;
                if (d == 0) a.part_ml[slot + r] = make_float4(mx, sum, fr, 0.f);
            }
        }
        if (n_use < total) {
            at.blk = blk1 - 1;
            at.next(a, total - n_use);   // o_sm is written again only behind the next segment's barrier
        }
    }
}

// Joins the segments of heads whose keys were shared by several CTAs, and writes the heads
// that have no keys.  D / 4 lanes hold a row's channels, PARTS of them in parallel take its
// parts in turn (a long cache of one head has a part per CTA of the GPU).  It is launched while
// the kernel before it still runs and waits for that one before it reads its parts.
template <int D, int PARTS>
constexpr int kJoinThreads = PARTS * D / 4 > 256 ? PARTS * D / 4 : 256;

template <int D, int PARTS, typename T>
__global__ void __launch_bounds__(kJoinThreads<D, PARTS>) join_kernel(AttnArgs a) {
    constexpr int kLanes = D / 4, kRows = kJoinThreads<D, PARTS> / (PARTS * kLanes);
    __shared__ float4 s_v[kRows][PARTS][kLanes];
    __shared__ float s_m[kRows][PARTS], s_l[kRows][PARTS];
    const int lane = threadIdx.x & 31, mine = threadIdx.x / (PARTS * kLanes);
    const long long row = (long long)blockIdx.x * kRows + mine;
    const bool valid = row < (long long)a.k.c.B * a.k.c.Hkv * a.R;
    const int bh = valid ? (int)(row / a.R) : 0, qrow = valid ? (int)(row % a.R) : 0;
    const int b = bh / a.k.c.Hkv, hkv = bh % a.k.c.Hkv;
    const int d = (threadIdx.x % kLanes) * 4, part = threadIdx.x / kLanes % PARTS;
    const WorkList list(a, lane);
    const int n = valid ? blocks_of(a, used_rows(a, b)) : 0;
    int first = 0, last = 0;
    // rows of one warp may be of two sequences (D = 64): the lanes ask together, for each
    const int before_lo = list.before(a, lane, __shfl_sync(0xffffffffu, b, 0));
    const int before_hi = list.before(a, lane, __shfl_sync(0xffffffffu, b, 31));
    if (n > 0) {
        const int w0 = (lane < kLanes ? before_lo : before_hi) + (hkv * a.groups + qrow / a.rows) * n;
        first = list.cta_of(w0);
        last = list.cta_of(w0 + n - 1);
    }
    if (blockIdx.x == 0)
        for (int x = threadIdx.x; x < a.k.c.B; x += kJoinThreads<D, PARTS>)
            if (a.k.kv_len[x] != used_rows(a, x)) set_status(a.k.status, PBSA_ERR_DEVICE_CHECK);
    grid_dependency_wait();
    grid_dependency_launch();
    const bool split = valid && !(n > 0 && first == last);   // else written by its CTA, or no row
    // the first CTA's part is its last segment (slot 1), the others' their first (slot 0)
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    float mx = -INFINITY, sum = 0.f, fac = 1.f;   // every part has the row's factor
    if (split && n > 0) {
        const size_t base = qrow % a.rows;
#pragma unroll 4
        for (int i = first + part; i <= last; i += PARTS) {
            const size_t at = base + ((size_t)2 * i + (i == first)) * a.rows;
            const float4 ml = a.part_ml[at];
            const float4 x = *reinterpret_cast<const float4*>(a.part_o + at * D + d);
            const float mn = fmaxf(mx, ml.x), ref = mn == -INFINITY ? 0.f : mn;
            fac = ml.z;
            const float f = ex2((mx - ref) * fac), k = ex2((ml.x - ref) * fac);
            v.x = f * v.x + k * x.x, v.y = f * v.y + k * x.y, v.z = f * v.z + k * x.z, v.w = f * v.w + k * x.w;
            sum = f * sum + k * ml.y;
            mx = mn;
        }
    }
    if (PARTS > 1) {
        s_v[mine][part][threadIdx.x % kLanes] = v;
        if (d == 0) {
            s_m[mine][part] = mx;
            s_l[mine][part] = sum;
        }
        __syncthreads();
        if (part == 0) {
            for (int i = 1; i < PARTS; ++i) mx = fmaxf(mx, s_m[mine][i]);
            const float ref = mx == -INFINITY ? 0.f : mx;
            v = make_float4(0.f, 0.f, 0.f, 0.f);
            sum = 0.f;
#pragma unroll
            for (int i = 0; i < PARTS; ++i) {
                const float k = ex2((s_m[mine][i] - ref) * fac);   // the first part's lanes have it
                const float4 x = s_v[mine][i][threadIdx.x % kLanes];
                v.x += k * x.x, v.y += k * x.y, v.z += k * x.z, v.w += k * x.w;
                sum += k * s_l[mine][i];
            }
        }
    }
    if (split && part == 0) finish_row<D, T>(a, b, hkv, qrow, d, v, mx, fac, sum);
}

// Masses from the kept products of at most eight rows: a thread takes four cached rows.
constexpr int kMassThreads = 128;

__global__ void __launch_bounds__(kMassThreads) mass_logits_kernel(AttnArgs a) {
    const int N = a.k.c.capacity, bh = blockIdx.x, b = bh / a.k.c.Hkv;
    const int j = (blockIdx.y * kMassThreads + threadIdx.x) * 4, len = used_rows(a, b);
    grid_dependency_wait();
    if (j >= len) return;
    const float* s = a.logits + (size_t)bh * a.R * N + j;
    const size_t at = (size_t)bh * N + j;
    const int4 pos = *reinterpret_cast<const int4*>(a.k.cache.pos + at);
    float4 mass = *reinterpret_cast<const float4*>(a.k.mass + at);
    float4 v[8], ref[8];
#pragma unroll
    for (int r = 0; r < 8; ++r)
        if (r < a.R) {
            v[r] = *reinterpret_cast<const float4*>(s + (size_t)r * N);
            ref[r] = a.row_ref[(size_t)bh * a.R + r];
        }
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < 8; ++r)
        if (r < a.R) {   // a hidden row's product is -inf: it adds 0, whatever the reference
            auto p = [&](float x) { return x == -INFINITY ? 0.f : ex2(fmaf(x - ref[r].x, ref[r].y, ref[r].z)); };
            sum.x += p(v[r].x);
            sum.y += p(v[r].y);
            sum.z += p(v[r].z);
            sum.w += p(v[r].w);
        }
    if (j < len && pos.x >= 0) mass.x += sum.x;
    if (j + 1 < len && pos.y >= 0) mass.y += sum.y;
    if (j + 2 < len && pos.z >= 0) mass.z += sum.z;
    if (j + 3 < len && pos.w >= 0) mass.w += sum.w;
    *reinterpret_cast<float4*>(a.k.mass + at) = mass;
}

// Masses of up to 8 NT rows: the scores are formed again (half of the cache's bytes) once the
// rows' sums are known; a warp owns its keys and takes all rows, so that every sum has one order
// and one owner, and a code is turned into fp16 once.  Latency bounds it, so a warp of a large
// call takes `run` units of keys with the next on its way (figures in run_attn), and the first is
// read before the wait.  The rows' constants lie in shared memory: in registers they took 104 to
// 138 of them and 3 us more a call (20 and 32 rows x 32 heads over 8192 cached rows).
template <int D, int NT>
__global__ void __launch_bounds__(32 * kMassWarps) mass_kernel(AttnArgs a, int run) {
    constexpr int kSteps = D / 16;
    __shared__ float4 s_row[8 * NT];   // a row's reference, factor, exponent of the reference; its limit
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int N = a.k.c.capacity, units = N / kUnit, per_bh = (units + kMassWarps * run - 1) / (kMassWarps * run);
    const int bh = blockIdx.x / per_bh, b = bh / a.k.c.Hkv;
    const int len = used_rows(a, b), used = (len + kUnit - 1) / kUnit;
    int u = (blockIdx.x % per_bh) * kMassWarps * run + warp;
    const int end = min(used, u + kMassWarps * run);
    const size_t row0 = (size_t)bh * N;
    auto load = [&](Keys<D>& x, int unit) {
        const size_t row = row0 + (size_t)unit * kUnit;
        load_keys(x, a.k.cache.k_codes + row * (D / 2), a.k.cache.k_scales + row * (D / 16), a.k.cache.pos + row, lane);
    };
    Keys<D> x;   // the first is read while the kernels before still run
    if (u < end) load(x, u);
    grid_dependency_wait();
    if (threadIdx.x < 8 * NT) {
        const float4 rf = a.row_ref[(size_t)bh * a.R + min((int)threadIdx.x, a.R - 1)];
        s_row[threadIdx.x] = make_float4(rf.x, rf.y, rf.z, __int_as_float(row_limit(a, b, threadIdx.x)));
    }
    __syncthreads();
    const uint2* q = a.q_frag + (size_t)bh * NT * kSteps * 32 + lane;
    for (; u < end; u += kMassWarps) {
        const int unit = u;
        Keys<D> y = x;
        if (u + kMassWarps < end) load(x, u + kMassWarps);
        hide_keys(y, len - unit * kUnit, lane);
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
        scores<D, NT>(s, y, [&](int j, int n) { return q[(n * kSteps + j) * 32]; });
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 rf = s_row[8 * n + 2 * c + i];
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (y.pos[k] <= __float_as_int(rf.w)) sum[k] += ex2(fmaf(s[n][i + 2 * k] - rf.x, rf.y, rf.z));
            }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 1);
            sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 2);
            if (c == 0 && y.pos[k] != kHidden) a.k.mass[row0 + (size_t)unit * kUnit + g + 8 * k] += sum[k];
        }
    }
}

// Groups of eight rows that a CTA of attn_kernel takes: all rows of a key head.  (20 rows x 8 heads
// of 4 sequences over 8192 cached rows: 34.0 us with three, 37.6 with four.)
int row_groups(int R) { return (R + 7) / 8; }
static_assert(kFewRows == 32, "attn_kernel is built for one to four groups of eight rows");

bool keeps_logits(int R) { return R <= 8; }

// The split of a call: rows of a group, groups, and CTAs - they fill every SM once, and none
// has less than a block.  Returns the blocks of a full cache.
long long plan(const pbsa_kv4_config& c, int R, AttnArgs& a) {
    const bool chunk = chunk_takes(R);
    const int per_sm = !chunk && row_groups(R) == 1 ? 2 : 1;
    a.rows = chunk ? kChunkRows : 8 * row_groups(R);
    a.groups = (R + a.rows - 1) / a.rows;
    a.heads = c.Hkv * a.groups;
    a.block = chunk ? kChunkKeys : kBlock;
    a.tiles8 = (R + 7) / 8;
    a.tiles128 = (R + 127) / 128;
    const long long blocks = (long long)c.B * a.heads * ((c.capacity + a.block - 1) / a.block);
    a.ctas = (int)(blocks < kSMs * per_sm ? blocks : kSMs * per_sm);
    return blocks;
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// Workspace: parts of outputs and statistics, then what the masses and the many-row kernels need.
struct Layout {
    size_t part_o, part_ml, row_ref, logits, q_frag, q_tile, q_scale, bytes;

    Layout(const pbsa_kv4_config& c, int R) {
        AttnArgs a{};
        plan(c, R, a);
        const size_t bh = (size_t)c.B * c.Hkv, slots = (size_t)a.ctas * 2 * a.rows;
        size_t at = 0;
        auto take = [&](size_t n) {
            const size_t r = at;
            at += up256(n);
            return r;
        };
        part_o = take(slots * c.D * sizeof(float));
        part_ml = take(slots * sizeof(float4));
        row_ref = take(bh * R * sizeof(float4));
        logits = q_frag = q_tile = q_scale = at;
        if (chunk_takes(R)) {
            q_tile = take(bh * a.tiles128 * 128 * c.D * 2);
            q_scale = take(bh * a.tiles128 * 128 * sizeof(float));
        } else if (keeps_logits(R)) {
            logits = take(bh * c.capacity * R * sizeof(float));
        } else {
            q_frag = take(bh * a.tiles8 * (c.D / 16) * 32 * sizeof(uint2));
        }
        bytes = at;
    }
};

template <int D, int NT, typename T, bool kLogits>
cudaError_t run_rows(const AttnArgs& a, cudaStream_t st) {
    const size_t smem = sizeof(Block<D>) * kStages + (size_t)(D / 16) * NT * 32 * 8 +
                        (size_t)kWarps * 8 * NT * (D + 2) * 4 + 8 * NT * 12;
    cudaError_t e = cudaFuncSetAttribute(attn_kernel<D, NT, T, kLogits>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    attn_kernel<D, NT, T, kLogits><<<(unsigned)a.ctas, 32 * (kWarps + 1), smem, st>>>(a);
    return cudaGetLastError();
}

template <int D, typename T>
cudaError_t run_attn(const AttnArgs& a, cudaStream_t st) {
    const bool chunk = chunk_takes(a.R);
    cudaError_t e;
    if (chunk) e = launch_chunk_attn(a, st);
    else if (a.groups != 1) return cudaErrorInvalidValue;   // attn_kernel knows no others
    else if (a.rows == 8) e = a.k.mass ? run_rows<D, 1, T, true>(a, st) : run_rows<D, 1, T, false>(a, st);
    else if (a.rows == 16) e = run_rows<D, 2, T, false>(a, st);
    else if (a.rows == 24) e = run_rows<D, 3, T, false>(a, st);
    else e = run_rows<D, 4, T, false>(a, st);   // 32: kFewRows
    if (e != cudaSuccess) return e;
    const int bh = a.k.c.B * a.k.c.Hkv;
    const long long rows = (long long)bh * a.R;
    auto join = [&](auto kernel, int threads, int parts) {
        const int per = threads / (parts * D / 4);
        return launch_after(kernel, dim3((unsigned)((rows + per - 1) / per)), threads, 0, st, a);
    };
    // Few heads have many parts each.  Whole calls, with 1, 4 and 16 parts of a row at a time: 296
    // parts a head 82.4, 43.9, 18.4 us; 9 parts of 8 rows 23.0, 21.3, 20.8; 4 parts of 8 rows 30.9,
    // 29.8, 33.6; 2 of 8 48.2, 48.2, 57.3; 1 of 8 82.1, 85.1, 101.2.
    const int parts = a.ctas / (a.k.c.B * a.heads);
    if (parts >= 8) e = join(join_kernel<D, 16, T>, kJoinThreads<D, 16>, 16);
    else if (parts >= 2) e = join(join_kernel<D, 4, T>, kJoinThreads<D, 4>, 4);
    else e = join(join_kernel<D, 1, T>, kJoinThreads<D, 1>, 1);
    if (e != cudaSuccess || !a.k.mass) return e;
    if (chunk) return launch_chunk_mass(a, st);
    if (keeps_logits(a.R)) {
        const unsigned runs = (unsigned)((a.k.c.capacity + 4 * kMassThreads - 1) / (4 * kMassThreads));
        return launch_after(mass_logits_kernel, dim3((unsigned)bh, runs), kMassThreads, 0, st, a);
    }
    // Units of sixteen keys that a warp takes: several where all of them fill the GPU (kMassFull).
    // Whole calls of 20 rows, with one unit and with four: 8192 units in all 33.4 and 35.6 us, 10240
    // 38.3 and 37.6, 16384 48.2 and 45.1, 65536 141.6 and 125.1 (eight: 123.9, but 50.5 at 16384).
    const int units = a.k.c.capacity / kUnit, run = (long long)bh * units >= kMassFull ? kMassRun : 1;
    const dim3 grid((unsigned)(bh * ((units + kMassWarps * run - 1) / (kMassWarps * run))));
    auto mass = [&](auto kernel) { return launch_after(kernel, grid, 32 * kMassWarps, 0, st, a, run); };
    if (a.tiles8 == 2) return mass(mass_kernel<D, 2>);
    if (a.tiles8 == 3) return mass(mass_kernel<D, 3>);
    return mass(mass_kernel<D, 4>);
}

}  // namespace

bool kv4_attn_fits(const pbsa_kv4_config& c, int T) {
    AttnArgs a{};
    return plan(c, T * (c.Hq / c.Hkv), a) < (1ll << 31);
}

size_t kv4_attn_workspace(const pbsa_kv4_config& c, int T) { return Layout(c, T * (c.Hq / c.Hkv)).bytes; }

cudaError_t launch_kv4_attn(const Kv4Args& k, cudaStream_t st) {
    AttnArgs a{};
    a.k = k;
    a.G = k.c.Hq / k.c.Hkv;
    a.R = k.T * a.G;
    plan(k.c, a.R, a);
    const Layout lay(k.c, a.R);
    char* w = static_cast<char*>(k.workspace);
    a.part_o = reinterpret_cast<float*>(w + lay.part_o);
    a.part_ml = reinterpret_cast<float4*>(w + lay.part_ml);
    if (k.mass) a.row_ref = reinterpret_cast<float4*>(w + lay.row_ref);
    if (chunk_takes(a.R)) {
        a.q_tile = reinterpret_cast<uint8_t*>(w + lay.q_tile);
        a.q_scale = reinterpret_cast<float*>(w + lay.q_scale);
    } else if (k.mass && keeps_logits(a.R)) {
        a.logits = reinterpret_cast<float*>(w + lay.logits);
    } else if (k.mass) {
        a.q_frag = reinterpret_cast<uint2*>(w + lay.q_frag);
    }
    if (k.c.D == 64)
        return k.c.dtype == PBSA_DTYPE_BF16 ? run_attn<64, __nv_bfloat16>(a, st) : run_attn<64, __half>(a, st);
    return k.c.dtype == PBSA_DTYPE_BF16 ? run_attn<128, __nv_bfloat16>(a, st) : run_attn<128, __half>(a, st);
}

}  // namespace pbsa
