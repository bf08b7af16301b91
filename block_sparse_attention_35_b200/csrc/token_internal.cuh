// token_internal.cuh - arguments and launchers of the token operators: norm and rotation of
// heads (qk_norm_rope.cu) and the 4-bit token cache (kv4_*.cu).  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "pbsa.h"

namespace pbsa {

// Strides of a [B, T, H, D] tensor in elements; channels are contiguous.
struct Strides {
    long long b, t, h;
};

struct QkArgs {
    pbsa_qk_config c;
    const void* x[2];    // q, k
    const void* gy[2];   // dq_out, dk_out (backward)
    void* y[2];          // q_out, k_out, or dq, dk
    Strides sx[2], sg[2], sy[2];
    const float* w[2];   // nullable
    const float* cos;
    const float* sin;
    const int32_t* pos;
    float* dw[2];        // nullable (backward)
    float* partial;      // [blocks][2][D] (backward)
    int32_t* status;
};

cudaError_t launch_qk_fwd(const QkArgs& a, cudaStream_t st);
cudaError_t launch_qk_bwd(const QkArgs& a, cudaStream_t st);
// Blocks of the backward kernel: rows of `partial`.
int qk_bwd_blocks(const pbsa_qk_config& c);

struct Kv4Args {
    pbsa_kv4_config c;
    pbsa_kv4_cache cache;
    int T;
    // append
    const void* k_new;
    const void* v_new;
    Strides sk, sv;
    const int32_t* pos_new;
    const int32_t* rows;   // nullable; append and read
    // read
    int n;
    void* k_out;
    void* v_out;
    // attention
    const void* q;
    Strides sq;
    const int32_t* q_pos;  // nullable
    const int32_t* kv_len;
    void* out;
    float* lse;
    float* mass;           // nullable
    void* workspace;
    int32_t* status;
};

cudaError_t launch_kv4_append(const Kv4Args& a, cudaStream_t st);
cudaError_t launch_kv4_read(const Kv4Args& a, cudaStream_t st);
cudaError_t launch_kv4_attn(const Kv4Args& a, cudaStream_t st);
size_t kv4_attn_workspace(const pbsa_kv4_config& c, int T);
// Whether the pieces of work of a call can be counted (below 2^31).
bool kv4_attn_fits(const pbsa_kv4_config& c, int T);

struct EvictArgs {
    int BH, Hkv, N, n, n_sink;
    const int32_t* pos;
    const float* mass;
    const int32_t* keep_from;  // nullable
    int32_t* rows;
    int32_t* status;
};

cudaError_t launch_kv4_evict(const EvictArgs& a, cudaStream_t st);

// Streaming multiprocessors that launch shapes (and so workspaces) are sized for.  A constant,
// so that a workspace size asked for on another machine or device still fits.
constexpr int kSMs = 148;

}  // namespace pbsa
