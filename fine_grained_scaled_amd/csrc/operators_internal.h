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

// The output head with softmax cross entropy (cross_entropy.hip).
struct CrossEntropyArgs {
    const void *x, *w, *targets;    // BF16 [T][ldx], BF16 [V][ldw], int32 or (wide) int64 [T]
    int64_t ldx, ldw, T, V, K;
    int wide;
    float *loss, *lse;              // [T]; the backward call reads lse
    const float *dloss, *dlse;      // [T]; dlse may be nullptr
    void *dx, *dw;                  // BF16 [T][K], [V][K]
    void* workspace;
};
hipError_t launch_cross_entropy_fwd(const CrossEntropyArgs& a, hipStream_t stream);
hipError_t launch_cross_entropy_bwd(const CrossEntropyArgs& a, hipStream_t stream);
size_t cross_entropy_workspace_bytes(int64_t T, int64_t V, int64_t K, int backward);

// Token embedding and its gradient (embedding.hip).
struct EmbeddingArgs {
    const void* tokens;             // int32 or (wide) int64 [T]
    int wide;
    int64_t T, V, W;
    const void* weight;             // forward: [V][ldw]
    int64_t ldw;
    int weight_bf16, bf16;          // the weight's (gradient's) type, and that of out (dout): BF16, not FP32
    float scale;
    void* out;                      // [T][W]
    const void* dout;               // backward: [T][ldd]
    int64_t ldd;
    void* dweight;                  // [V][W]
    int add;                        // to what dweight holds
    void* workspace;
};
hipError_t launch_embedding_fwd(const EmbeddingArgs& a, hipStream_t stream);
hipError_t launch_embedding_bwd(const EmbeddingArgs& a, hipStream_t stream);
size_t embedding_workspace_bytes(int64_t T, int64_t W);

// SwiGLU with its input kept in 8 bits (swiglu.hip).
struct SwigluArgs {
    int64_t T, I;
    const void* gate_up;            // BF16 [T][ld]
    int64_t ld;
    void* h;                        // BF16 [T][I]
    uint8_t* q;                     // E4M3 [T][2 I], or nullptr: nothing kept (the backward call reads gate_up)
    float* scales;                  // [2 ceil(I / 128)][T]
    const void* dh;                 // BF16 [T][ldh]
    int64_t ldh;
    void* dgate_up;                 // BF16 [T][2 I]
};
int64_t swiglu_blocks(int64_t T, int64_t I);      // workgroups of a launch
hipError_t launch_swiglu_fwd(const SwigluArgs& a, hipStream_t stream);
hipError_t launch_swiglu_bwd(const SwigluArgs& a, hipStream_t stream);

} // namespace fgs
