// operators_internal.h -- launcher interfaces of the operators around the linear
// layers.  Apart from fgs_internal.h, which is a source of the GEMM kernel:
// the benchmark reports that kernel's counters only while its sources are
// those that they were taken on.
#pragma once

#include "fgs_internal.h"

namespace fgs {

// Causal attention over packed sequences (attention_fwd.hip, attention_bwd.hip).
struct AttentionArgs {
    fgs_heads q, k, v, out, dout, dq, dk, dv;   // the backward call uses all, the forward one the first four
    float* lse;                     // [H][T]
    float* delta;                   // backward workspace: two rows of T a head,
    float* shares;                  // ATTENTION_SLOTS sums of 128 keys x 2 x 128 values,
    int* arrived;                   // and as many counters (both from ATTENTION_SPLIT_TOKENS tokens on)
    const int32_t* cu_seqlens;      // device int32 [S + 1]
    int64_t T;
    int32_t S, H, Hk, D;
    float scale;
};
constexpr int ATTENTION_SLOTS = 512, ATTENTION_SPLIT_TOKENS = 1024;
constexpr size_t ATTENTION_SLOT_BYTES = 2 * 128 * 128 * sizeof(float);
hipError_t launch_attention_fwd(const AttentionArgs& a, hipStream_t stream);
hipError_t launch_attention_bwd(const AttentionArgs& a, hipStream_t stream);

// The block boundary: norm, gate, residual, norm (residual_norm.hip).
struct NormArgs {
    int64_t T, W;
    const void *y, *x, *gate;       // x: the residual (forward), r (backward)
    int64_t ldy, ldx, ldg;
    int fp32;                       // the residual is FP32, not BF16
    int gate_kind;                  // FGS_GATE_*
    const float *w_post, *w_pre;    // w_post may be nullptr
    float alpha, eps;
    void *r, *n;                    // forward outputs
    const void *dr, *dn;            // backward
    int64_t lddr, lddn;
    void *dx, *dy, *dgate;
    float *dw_post, *dw_pre;
    float* partial;                 // residual_norm_parts() x 3 x W
};
hipError_t launch_residual_norm_fwd(const NormArgs& a, hipStream_t stream);
hipError_t launch_residual_norm_bwd(const NormArgs& a, hipStream_t stream);
int residual_norm_parts(int64_t T, int64_t W);

// The global gradient norm and clipping (clip_grad.hip).
hipError_t launch_clip_grad_norm(const fgs_grad* grads, int32_t count, float max_norm, float* norm, double* partial,
                                 hipStream_t stream);
size_t clip_workspace_bytes(int32_t count);

} // namespace fgs
