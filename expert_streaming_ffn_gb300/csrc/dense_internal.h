// Norm, 8-bit quantisation and 8-bit matrix product: kernel parameters and launchers.
// Not part of the public ABI (include/moe.h describes operands and layouts).
#pragma once

#include "kv_internal.h"

namespace moe {

constexpr int kF8Block = 128;  // elements (of a row; each way of a weight) that share a scale
constexpr int kNormMaxDim = 32768;

// Whether a kernel that writes outputs of these types may let the next one start before it is done. moe_forward's expert
// kernel reads its bf16 rows x before it waits for what is in front of it (the router, which lets it start at once), so x
// has to be there when the router starts: a kernel that may be writing x does not let it start early.
inline bool may_release_early(bool writes, moe_dtype t) { return !writes || t != MOE_BF16; }

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
    bool early;  // may_release_early()
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
    bool early;      // may_release_early()
};
cudaError_t launch_f8_matmul(const MatmulArgs& a, int sms, cudaStream_t s);

}  // namespace moe
