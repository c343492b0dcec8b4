// Norm, 8-bit quantisation and 8-bit matrix product: kernel parameters and launchers.
// Not part of the public ABI (include/moe.h describes operands and layouts).
#pragma once

#include "kv_internal.h"

namespace moe {

constexpr int kF8Block = 128;  // elements (of a row; each way of a weight) that share a scale
constexpr int kNormMaxDim = 32768;

struct NormArgs {
    const void* x;
    const void* res;     // or null
    const void* weight;  // or null
    void* sum;           // or null
    void* out;           // or null
    uint8_t* codes;      // or null
    float* scales;       // with codes
    int64_t xt, xh, rt, rh, st, sh, ot, oh;  // element strides by token and head
    int64_t ct, scale_stride;
    unsigned rows;  // tokens * heads
    int dim;
    float eps, inv_dim;
    FastDiv by_head{1};
    moe_dtype x_type, res_type, weight_type, out_type;  // sum has res_type
};
cudaError_t launch_rms_norm(const NormArgs& a, int sms, cudaStream_t s);

struct QuantArgs {
    const void* x;
    int64_t x_stride, code_stride, scale_stride;  // elements
    uint8_t* codes;
    float* scales;
    int n, dim;
    moe_dtype type;
    FastDiv by_row{1};  // / blocks of a row; set by the launcher
};
cudaError_t launch_f8_quant_rows(const QuantArgs& a, int sms, cudaStream_t s);
cudaError_t launch_f8_quant_weight(const QuantArgs& a, cudaStream_t s);

struct MatmulArgs {
    const uint8_t* a;  // rows
    const uint8_t* w;  // weights
    const float* sa;   // [block][row]
    const float* sw;   // [n block][k block]
    void* out;
    int64_t a_stride, w_stride, sa_stride, sw_stride, out_stride;
    int m, n, k;
    moe_dtype type;  // of out
    unsigned* err;   // mapped word: a bounded wait expired
};
cudaError_t launch_f8_matmul(const MatmulArgs& a, int sms, cudaStream_t s);

}  // namespace moe
