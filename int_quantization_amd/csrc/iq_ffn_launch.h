// Internal interface between the feed-forward entry points (iq_ffn_api.cpp)
// and their kernel launchers (iq_norm.hip, iq_packed.hip, iq_gated.hip).
// Not part of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

namespace iqk {

// Activations use the public enum values of iq.h.
enum { A_SILU = 0, A_GELU = 1, A_GELU_TANH = 2 };

struct NormArgs {
    int in_dtype, param_dtype;
    int64_t rows, cols, ld;
    float eps;
    const void* x;
    const void* weight;      // may be null
    const void* bias;        // may be null
    void* y;
    float* mean;             // may be null
    float* rstd;             // may be null
};

struct NormGradArgs {
    int in_dtype, param_dtype;
    int64_t rows, cols, ld;
    const void* x;
    const void* dy;
    const void* weight;      // may be null
    const float* mean;
    const float* rstd;
    void* dx;                // may be null
    void* dweight;           // may be null
    void* dbias;             // may be null
    float* partial;          // [kNormParts][2][cols] where dweight or dbias is wanted
};

// Workgroups of the layer norm's backward pass, one partial row of the
// weight's and the bias's gradient each.
constexpr int kNormParts = 256;

// A weight matrix of the few-token products: packed codes with their block
// scales, or BF16 elements (fmt F_BF16W: codes are the elements).
enum { F_BF16W = 16 };
struct PackedWeight {
    const void* codes;
    const void* scales;
    const float* global_scale;
};

struct PackedArgs {
    int fmt;                 // F_INT4, F_NVFP4, F_MXFP4 or F_BF16W
    bool gated;              // w[0] gate and w[1] up, or w[0] alone
    int act;
    PackedWeight w[2];
    const void* x;           // BF16 [n1, K], row stride ldx
    int64_t ldx;
    void* out;               // [n1, n0]
    int out_dtype;
    float* saved;            // g and u [2][n1][n0], may be null
    int64_t n0, n1, K;
};
constexpr int64_t kPackedTokens = 64;   // most tokens of one call

struct GatedArgs {
    int act;
    int64_t tokens, cols, features, ldx;
    const void* x;
    const void* wg;
    const void* wu;
    void* h;
    float* saved;            // may be null
};

struct GatedGradArgs {
    int act;
    int64_t tokens, cols, features, ldx;
    const void* dh;
    const void* x;
    const void* wg;
    const void* wu;
    const float* saved;
    void* dx;                // may be null
    void* dwg;               // both weight gradients, or both null
    void* dwu;
    void* workspace;
};

// Each returns hipSuccess or the launch error.
hipError_t launch_layer_norm(const NormArgs& a, hipStream_t stream);
hipError_t launch_layer_norm_grad(const NormGradArgs& a, hipStream_t stream);
hipError_t launch_packed(const PackedArgs& a, hipStream_t stream);
hipError_t launch_gated(const GatedArgs& a, hipStream_t stream);
hipError_t launch_gated_grad(const GatedGradArgs& a, hipStream_t stream);
// Workspace of launch_gated_grad: dg and du in BF16, then the partial sums
// of a dx whose long sum is split.
size_t gated_workspace_bytes(int64_t tokens, int64_t cols, int64_t features);

}  // namespace iqk
