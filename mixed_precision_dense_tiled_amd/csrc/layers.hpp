// layers.hpp -- internal (C++) interface between the C ABI and the kernels of a
// decoder layer's operators: norm, rotation on the way into the cache, products
// grouped by expert.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "serving.hpp"

namespace mpdt {

// What a norm writes (the values of the C ABI's mpdt_norm_out).
enum : int { NORM_PLAIN = 0, NORM_I8_ROWS = 1, NORM_E4M3_ROWS = 2, NORM_E4M3_BLOCKS = 3 };

constexpr int CUS = 256;   // compute units

constexpr int64_t NORM_MAX_DIM = 32768;
// Rows of a norm's launch, a workgroup of up to 1024 threads to each.  (Its gradient's workgroups
// walk rows: any number.)
constexpr int64_t NORM_MAX_ROWS = LAUNCH_THREADS / 1024;
static_assert(NORM_MAX_ROWS == 4194303, "as the C ABI says");

struct NormArgs {
    const char* x;          // strides in bytes
    int64_t x_b;
    const char* residual;   // or null
    int64_t res_b;
    char* h;                // x + residual, or null
    int64_t h_b;
    const char* weight;
    double eps;
    char* out;
    int64_t out_b;
    float* scales;
    int64_t ld_scales;
    float* rstd;            // or null
    int rows, dim;
    int type, w_f32;        // w_f32: the weight is FP32 (else x's type)
    int quant;              // NORM_*
};
hipError_t launch_rms_norm(const NormArgs& a, hipStream_t stream);

struct NormGradArgs {
    const char* grad;       // strides in bytes
    int64_t grad_b;
    const char* h;
    int64_t h_b;
    const char* weight;
    const float* rstd;
    const char* grad_res;   // or null
    int64_t gres_b;
    char* grad_h;
    int64_t gh_b;
    float* grad_weight;     // [dim]
    float* ws;              // partial sums of the weight's gradient
    int rows, dim;
    int type, w_f32;
};
int64_t rms_norm_backward_ws(int64_t rows, int64_t dim);
hipError_t launch_rms_norm_backward(const NormGradArgs& a, hipStream_t stream);

struct RopeArgs {
    AppendArgs ap;
    const float* inv_freq;  // [pairs]
    int pairs, interleaved, heads;
    const char* q;          // strides in bytes
    int64_t q_tok_b, q_head_b;
    char* q_out;
    int64_t qo_tok_b, qo_head_b;
};
hipError_t launch_paged_append_rope(const RopeArgs& a, hipStream_t stream);

// Products grouped by expert: M = rows of a group, or for the weights' gradient
// M x N = K x N of the call, summed over a group's rows.
enum : int { GROUPED_NN = 0, GROUPED_NT = 1, GROUPED_TN = 2 };   // A . B, A . B^T, A^T . B

struct GroupedArgs {
    const char* A;
    const char* B;
    char* D;
    int64_t lda_b, ldb_b;   // bytes
    int64_t group_b;        // bytes between groups of B (NN, NT)
    int64_t ldd, group_d;   // elements (group_d: between groups of D, TN)
    const int32_t* offsets; // [groups + 1]
    int groups;
    int rows;               // of A (and of G)
    int M, N, K;            // TN: M x N of D; NN, NT: N x K of the weights (M is a group's)
    int out16;
    // W8A8
    const float* x_scale;
    const float* w_scale;
    const float* bias;      // or null
    int64_t ld_ws, ld_bias;
};
enum class GroupedType { BF16, F16, I8 };
bool grouped_fits(int mode, const GroupedArgs& a);   // its launch
hipError_t launch_grouped(GroupedType type, int mode, const GroupedArgs& a, hipStream_t stream);

}  // namespace mpdt
