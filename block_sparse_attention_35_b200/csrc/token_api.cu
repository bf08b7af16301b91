// token_api.cu - C ABI of the token operators: argument checks and launches.  Nothing here
// allocates device memory or synchronises the host.
#include <cuda_runtime.h>

#include <cmath>
#include <utility>

#include "pbsa.h"
#include "pbsa_internal.cuh"
#include "token_internal.cuh"

namespace {

using pbsa::api_cuda_fail;
using pbsa::api_failf;

int element_size(int dtype) { return dtype == PBSA_DTYPE_FP32 ? 4 : 2; }

int check_ptr(const void* p, const char* name) {
    if (!p) return api_failf(PBSA_ERR_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) & 15u) return api_failf(PBSA_ERR_ARG, "%s is not 16-byte aligned", name);
    return PBSA_OK;
}

#define CHECK(expr)                       \
    do {                                  \
        const int rc_ = (expr);           \
        if (rc_ != PBSA_OK) return rc_;   \
    } while (0)
#define NEED(p) CHECK(check_ptr(p, #p))
#define MAY(p)                            \
    do {                                  \
        if (p) CHECK(check_ptr(p, #p));   \
    } while (0)

// The i-th tensor's strides, or those of a contiguous [B, T, H, D] tensor.
int get_strides(pbsa::Strides* out, const int64_t* strides, int i, const char* name, int T, int H, int D, int es) {
    if (!strides) {
        out->h = D;
        out->t = (long long)H * D;
        out->b = (long long)T * H * D;
        return PBSA_OK;
    }
    const int64_t* s = strides + 3 * i;
    for (int k = 0; k < 3; ++k)
        if (s[k] < 0 || s[k] % (16 / es) != 0)
            return api_failf(PBSA_ERR_ARG, "%s: stride %lld is negative or not a multiple of 16 bytes", name, (long long)s[k]);
    out->b = s[0];
    out->t = s[1];
    out->h = s[2];
    return PBSA_OK;
}

// Whether the elements of a [B, T, H, D] output are its own: each stride, from the smallest on,
// steps over all that the smaller ones reach.
int check_own(const pbsa::Strides& s, const char* name, int B, int T, int H, int D) {
    struct { long long stride; int n; } d[3] = {{s.b, B}, {s.t, T}, {s.h, H}};
    if (d[0].stride > d[1].stride) std::swap(d[0], d[1]);
    if (d[1].stride > d[2].stride) std::swap(d[1], d[2]);
    if (d[0].stride > d[1].stride) std::swap(d[0], d[1]);
    __int128 reach = D;
    for (const auto& x : d) {
        if (x.n <= 1) continue;
        if (x.stride < reach) return api_failf(PBSA_ERR_ARG, "%s: stride %lld lets elements share memory", name, x.stride);
        reach += (__int128)x.stride * (x.n - 1);
    }
    return PBSA_OK;
}

int validate(const pbsa_qk_config* c) {
    if (!c) return api_failf(PBSA_ERR_ARG, "config is NULL");
    if (c->B < 1 || c->T < 0) return api_failf(PBSA_ERR_ARG, "B %d must be >= 1 and T %d >= 0", c->B, c->T);
    if (c->Hq < 1 || c->Hkv < 0 || c->Hq > 65535 || c->Hkv > 65535)
        return api_failf(PBSA_ERR_ARG, "Hq %d not in [1, 65535] or Hkv %d not in [0, 65535]", c->Hq, c->Hkv);
    const long long tokens = (long long)c->B * c->T;
    if (tokens > (1ll << 32) || tokens * (c->Hq + c->Hkv) > (1ll << 32))
        return api_failf(PBSA_ERR_UNSUPPORTED, "more than 2^32 heads of tokens");
    if (c->D != 64 && c->D != 128) return api_failf(PBSA_ERR_UNSUPPORTED, "head dim %d: only 64 and 128 are built", c->D);
    if (c->dtype < PBSA_DTYPE_BF16 || c->dtype > PBSA_DTYPE_FP32) return api_failf(PBSA_ERR_UNSUPPORTED, "dtype %d", c->dtype);
    if (c->grad_dtype != c->dtype && c->grad_dtype != PBSA_DTYPE_FP32)
        return api_failf(PBSA_ERR_UNSUPPORTED, "grad_dtype %d: only dtype (%d) and fp32 are built", c->grad_dtype, c->dtype);
    if (c->rot_dim < 0 || c->rot_dim > c->D) return api_failf(PBSA_ERR_ARG, "rot_dim %d not in [0, %d]", c->rot_dim, c->D);
    if (c->rot_dim % 16) return api_failf(PBSA_ERR_UNSUPPORTED, "rot_dim %d: only multiples of 16 are built", c->rot_dim);
    if (!(c->eps > 0.f) || std::isinf(c->eps)) return api_failf(PBSA_ERR_ARG, "eps %g must be positive", c->eps);
    if (c->rot_dim > 0) {
        if (c->n_axes < 1 || c->n_axes > 3) return api_failf(PBSA_ERR_ARG, "n_axes %d not in [1, 3]", c->n_axes);
        long long sum = 0;
        for (int i = 0; i < c->n_axes; ++i) {
            if (c->axis_pairs[i] < 0) return api_failf(PBSA_ERR_ARG, "axis_pairs[%d] %d < 0", i, c->axis_pairs[i]);
            sum += c->axis_pairs[i];
        }
        if (sum != c->rot_dim / 2)
            return api_failf(PBSA_ERR_ARG, "axis_pairs add to %lld, not rot_dim / 2 = %d", sum, c->rot_dim / 2);
        if (c->table_len < 1) return api_failf(PBSA_ERR_ARG, "table_len %d < 1", c->table_len);
    }
    return PBSA_OK;
}

int validate(const pbsa_kv4_config* c) {
    if (!c) return api_failf(PBSA_ERR_ARG, "config is NULL");
    if (c->B < 1 || c->Hq < 1 || c->Hkv < 1) return api_failf(PBSA_ERR_ARG, "B, Hq and Hkv must be >= 1 (%d, %d, %d)", c->B, c->Hq, c->Hkv);
    if (c->B > 65535 || c->Hq > 65535) return api_failf(PBSA_ERR_ARG, "B and Hq must be <= 65535");
    if (c->Hq % c->Hkv) return api_failf(PBSA_ERR_ARG, "Hq %d is not a multiple of Hkv %d", c->Hq, c->Hkv);
    if (c->D != 64 && c->D != 128) return api_failf(PBSA_ERR_UNSUPPORTED, "head dim %d: only 64 and 128 are built", c->D);
    if (c->capacity < 64 || c->capacity % 64)
        return api_failf(PBSA_ERR_ARG, "capacity %d is not a positive multiple of 64", c->capacity);
    if (c->capacity > (1 << 24)) return api_failf(PBSA_ERR_UNSUPPORTED, "capacity %d above 2^24", c->capacity);
    if ((long long)c->B * c->Hkv * (c->capacity / 64) > 0x7fffffffll)
        return api_failf(PBSA_ERR_UNSUPPORTED, "cache of more than 2^31 64-row groups");
    if (c->dtype != PBSA_DTYPE_BF16 && c->dtype != PBSA_DTYPE_FP16)
        return api_failf(PBSA_ERR_UNSUPPORTED, "dtype %d: only bf16 and fp16 are built", c->dtype);
    for (int i = 0; i < 2; ++i) {
        const float u = i ? c->v_unit : c->k_unit;
        int e = 0;
        if (!(u > 0.f) || std::isinf(u) || std::frexp(u, &e) != 0.5f || e < -39 || e > 41)
            return api_failf(PBSA_ERR_ARG, "%s %g is not a power of two in [2^-40, 2^40]", i ? "v_unit" : "k_unit", u);
    }
    return PBSA_OK;
}

int check_cache(const pbsa_kv4_cache* cache) {
    if (!cache) return api_failf(PBSA_ERR_ARG, "cache is NULL");
    NEED(cache->k_codes);
    NEED(cache->k_scales);
    NEED(cache->v_codes);
    NEED(cache->v_scales);
    NEED(cache->pos);
    return PBSA_OK;
}

// Tokens of a kv4 call: the grid and index types hold for these.
int check_tokens(const pbsa_kv4_config* c, int T) {
    if (T < 0) return api_failf(PBSA_ERR_ARG, "T %d < 0", T);
    if ((long long)T * (c->Hq / c->Hkv) > (1 << 20) || (long long)c->B * T * c->Hq > 0x7fffffffll ||
        (long long)T * c->Hkv * (c->D / 16) > 0x7fffff00ll)
        return api_failf(PBSA_ERR_UNSUPPORTED, "T %d: too many query rows in one call", T);
    return PBSA_OK;
}

int check_queries(const pbsa_kv4_config* c, int T) {
    CHECK(check_tokens(c, T));
    if (T > 0 && !pbsa::kv4_attn_fits(*c, T))
        return api_failf(PBSA_ERR_UNSUPPORTED, "T %d over this cache: too many query rows in one call", T);
    return PBSA_OK;
}

pbsa::Kv4Args kv4_args(const pbsa_kv4_config* c, const pbsa_kv4_cache* cache) {
    pbsa::Kv4Args a{};
    a.c = *c;
    a.cache = *cache;
    return a;
}

int qk_common(pbsa::QkArgs* a, const pbsa_qk_config* cfg, const void* q, const void* k, const int64_t* strides,
              const float* wq, const float* wk, const float* cos, const float* sin, const int32_t* pos,
              int32_t* status) {
    NEED(q);
    if (cfg->Hkv > 0) NEED(k);
    MAY(wq);
    MAY(wk);
    if (cfg->rot_dim > 0) {
        NEED(cos);
        NEED(sin);
        NEED(pos);
        NEED(status);
    }
    const int es = element_size(cfg->dtype);
    CHECK(get_strides(&a->sx[0], strides, 0, "q", cfg->T, cfg->Hq, cfg->D, es));
    CHECK(get_strides(&a->sx[1], strides, 1, "k", cfg->T, cfg->Hkv, cfg->D, es));
    a->c = *cfg;
    a->x[0] = q;
    a->x[1] = k;
    a->w[0] = wq;
    a->w[1] = wk;
    a->cos = cos;
    a->sin = sin;
    a->pos = pos;
    a->status = status;
    return PBSA_OK;
}

}  // namespace

extern "C" {

size_t pbsa_qk_workspace_size(const pbsa_qk_config* cfg) {
    if (validate(cfg) != PBSA_OK) return 0;
    const size_t blocks = pbsa::qk_bwd_blocks(*cfg);
    return (blocks < 1 ? 1 : blocks) * 2 * cfg->D * sizeof(float);
}

int pbsa_qk_norm_rope(const pbsa_qk_config* cfg, const void* q, const void* k, const int64_t* strides,
                      const float* wq, const float* wk, const float* cos, const float* sin, const int32_t* pos,
                      void* q_out, void* k_out, int32_t* status, void* stream) {
    CHECK(validate(cfg));
    if (cfg->T == 0) return PBSA_OK;
    pbsa::QkArgs a{};
    CHECK(qk_common(&a, cfg, q, k, strides, wq, wk, cos, sin, pos, status));
    NEED(q_out);
    if (cfg->Hkv > 0) NEED(k_out);
    const int es = element_size(cfg->dtype);
    CHECK(get_strides(&a.sy[0], strides, 2, "q_out", cfg->T, cfg->Hq, cfg->D, es));
    CHECK(get_strides(&a.sy[1], strides, 3, "k_out", cfg->T, cfg->Hkv, cfg->D, es));
    CHECK(check_own(a.sy[0], "q_out", cfg->B, cfg->T, cfg->Hq, cfg->D));
    if (cfg->Hkv > 0) CHECK(check_own(a.sy[1], "k_out", cfg->B, cfg->T, cfg->Hkv, cfg->D));
    a.y[0] = q_out;
    a.y[1] = k_out;
    const cudaError_t e = pbsa::launch_qk_fwd(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PBSA_OK : api_cuda_fail(e, "norm and rotation kernel launch");
}

int pbsa_qk_norm_rope_bwd(const pbsa_qk_config* cfg, const void* q, const void* k, const int64_t* strides,
                          const float* wq, const float* wk, const float* cos, const float* sin, const int32_t* pos,
                          const void* dq_out, const void* dk_out, void* dq, void* dk, float* dwq, float* dwk,
                          void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
    CHECK(validate(cfg));
    MAY(dwq);
    MAY(dwk);
    pbsa::QkArgs a{};
    a.c = *cfg;
    if (dwq || dwk) {
        NEED(workspace);
        const size_t need = pbsa_qk_workspace_size(cfg);
        if (workspace_bytes < need)
            return api_failf(PBSA_ERR_WORKSPACE, "workspace %zu < %zu bytes", workspace_bytes, need);
        a.partial = static_cast<float*>(workspace);
    }
    if (cfg->T > 0) {   // with no tokens only the weights' gradients are written (zeros)
        CHECK(qk_common(&a, cfg, q, k, strides, wq, wk, cos, sin, pos, status));
        NEED(dq_out);
        NEED(dq);
        if (cfg->Hkv > 0) {
            NEED(dk_out);
            NEED(dk);
        }
        const int es = element_size(cfg->dtype), gs = element_size(cfg->grad_dtype);
        CHECK(get_strides(&a.sg[0], strides, 2, "dq_out", cfg->T, cfg->Hq, cfg->D, gs));
        CHECK(get_strides(&a.sg[1], strides, 3, "dk_out", cfg->T, cfg->Hkv, cfg->D, gs));
        CHECK(get_strides(&a.sy[0], strides, 4, "dq", cfg->T, cfg->Hq, cfg->D, es));
        CHECK(get_strides(&a.sy[1], strides, 5, "dk", cfg->T, cfg->Hkv, cfg->D, es));
        CHECK(check_own(a.sy[0], "dq", cfg->B, cfg->T, cfg->Hq, cfg->D));
        if (cfg->Hkv > 0) CHECK(check_own(a.sy[1], "dk", cfg->B, cfg->T, cfg->Hkv, cfg->D));
        a.gy[0] = dq_out;
        a.gy[1] = dk_out;
        a.y[0] = dq;
        a.y[1] = dk;
    }
    a.dw[0] = dwq;
    a.dw[1] = dwk;
    const cudaError_t e = pbsa::launch_qk_bwd(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PBSA_OK : api_cuda_fail(e, "norm and rotation gradient kernel launch");
}

int pbsa_validate_kv4_config(const pbsa_kv4_config* cfg) { return validate(cfg); }

size_t pbsa_kv4_workspace_size(const pbsa_kv4_config* cfg, int T) {
    if (validate(cfg) != PBSA_OK || check_queries(cfg, T) != PBSA_OK) return 0;
    return T == 0 ? 0 : pbsa::kv4_attn_workspace(*cfg, T);
}

int pbsa_kv4_append(const pbsa_kv4_config* cfg, const pbsa_kv4_cache* cache, const void* k_new, const void* v_new,
                    const int64_t* strides, int T, const int32_t* pos_new, const int32_t* rows, float* mass,
                    int32_t* status, void* stream) {
    CHECK(validate(cfg));
    CHECK(check_tokens(cfg, T));
    if (T == 0) return PBSA_OK;
    CHECK(check_cache(cache));
    NEED(k_new);
    NEED(v_new);
    NEED(pos_new);
    MAY(rows);
    MAY(mass);
    NEED(status);
    pbsa::Kv4Args a = kv4_args(cfg, cache);
    CHECK(get_strides(&a.sk, strides, 0, "k_new", T, cfg->Hkv, cfg->D, 2));
    CHECK(get_strides(&a.sv, strides, 1, "v_new", T, cfg->Hkv, cfg->D, 2));
    a.T = T;
    a.k_new = k_new;
    a.v_new = v_new;
    a.pos_new = pos_new;
    a.rows = rows;
    a.mass = mass;
    a.status = status;
    const cudaError_t e = pbsa::launch_kv4_append(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PBSA_OK : api_cuda_fail(e, "token append kernel launch");
}

int pbsa_kv4_read(const pbsa_kv4_config* cfg, const pbsa_kv4_cache* cache, const int32_t* rows, int n, void* k_out,
                  void* v_out, int32_t* status, void* stream) {
    CHECK(validate(cfg));
    if (n < 0) return api_failf(PBSA_ERR_ARG, "n %d < 0", n);
    if (!rows && n > cfg->capacity) return api_failf(PBSA_ERR_ARG, "n %d > capacity %d", n, cfg->capacity);
    const long long row_blocks = (long long)n * (cfg->D / 16);
    if (row_blocks > 0x7fffff00ll || (long long)cfg->B * cfg->Hkv * ((row_blocks + 255) / 256) > 0x7fffffffll)
        return api_failf(PBSA_ERR_UNSUPPORTED, "n %d: too many rows in one call", n);
    if (n == 0) return PBSA_OK;
    CHECK(check_cache(cache));
    MAY(rows);
    NEED(k_out);
    NEED(v_out);
    NEED(status);
    pbsa::Kv4Args a = kv4_args(cfg, cache);
    a.rows = rows;
    a.n = n;
    a.k_out = k_out;
    a.v_out = v_out;
    a.status = status;
    const cudaError_t e = pbsa::launch_kv4_read(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PBSA_OK : api_cuda_fail(e, "token read kernel launch");
}

int pbsa_kv4_attn(const pbsa_kv4_config* cfg, const pbsa_kv4_cache* cache, const void* q, const int64_t* strides,
                  int T, const int32_t* q_pos, const int32_t* kv_len, void* out, float* lse, float* mass,
                  void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
    CHECK(validate(cfg));
    CHECK(check_queries(cfg, T));
    if (T == 0) return PBSA_OK;
    CHECK(check_cache(cache));
    NEED(q);
    MAY(q_pos);
    NEED(kv_len);
    NEED(out);
    NEED(lse);
    MAY(mass);
    NEED(workspace);
    NEED(status);
    const size_t need = pbsa::kv4_attn_workspace(*cfg, T);
    if (workspace_bytes < need)
        return api_failf(PBSA_ERR_WORKSPACE, "workspace %zu < %zu bytes", workspace_bytes, need);
    pbsa::Kv4Args a = kv4_args(cfg, cache);
    CHECK(get_strides(&a.sq, strides, 0, "q", T, cfg->Hq, cfg->D, 2));
    a.T = T;
    a.q = q;
    a.q_pos = q_pos;
    a.kv_len = kv_len;
    a.out = out;
    a.lse = lse;
    a.mass = mass;
    a.workspace = workspace;
    a.status = status;
    const cudaError_t e = pbsa::launch_kv4_attn(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PBSA_OK : api_cuda_fail(e, "token attention kernel launch");
}

int pbsa_kv4_evict(const pbsa_kv4_config* cfg, const int32_t* pos, const float* mass, int n, int n_sink,
                   const int32_t* keep_from, int32_t* rows, int32_t* status, void* stream) {
    CHECK(validate(cfg));
    if (n < 0 || n > cfg->capacity) return api_failf(PBSA_ERR_ARG, "n %d not in [0, %d]", n, cfg->capacity);
    if (n_sink < 0) return api_failf(PBSA_ERR_ARG, "n_sink %d < 0", n_sink);
    if (n == 0) return PBSA_OK;
    NEED(pos);
    NEED(mass);
    MAY(keep_from);
    NEED(rows);
    NEED(status);
    pbsa::EvictArgs a{cfg->B * cfg->Hkv, cfg->Hkv, cfg->capacity, n, n_sink, pos, mass, keep_from, rows, status};
    const cudaError_t e = pbsa::launch_kv4_evict(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PBSA_OK : api_cuda_fail(e, "token eviction kernel launch");
}

}  // extern "C"
