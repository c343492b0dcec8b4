// libmoe C ABI: norm of rows, quantisation to 8 bits, and matrix products of 8-bit rows and weights.
#include <cuda_runtime.h>
#include <math.h>

#include "dense_internal.h"

using namespace moe;

#define CUDA_TRY(call)                                                                                 \
    do {                                                                                               \
        cudaError_t e_ = (call);                                                                       \
        if (e_ != cudaSuccess)                                                                         \
            return set_error(MOE_ECUDA, "%s failed: %s (%s:%d)", #call, cudaGetErrorString(e_), __FILE__, \
                             __LINE__);                                                                \
    } while (0)

namespace {

int type_size(moe_dtype t) { return t == MOE_F32 ? 4 : 2; }
bool type_ok(moe_dtype t) { return t == MOE_F32 || t == MOE_F16 || t == MOE_BF16; }
bool at16(const void* p) { return !(reinterpret_cast<uintptr_t>(p) & 15); }
bool at4(const void* p) { return !(reinterpret_cast<uintptr_t>(p) & 3); }

// Rows of `t` that start on 16-byte boundaries.
bool rows_ok(const void* p, int64_t ts, int64_t hs, moe_dtype t) {
    const int64_t per = 16 / type_size(t);
    return at16(p) && ts % per == 0 && hs % per == 0;
}

int blocks(int n) { return (n - 1) / kF8Block + 1; }

// Most rows, and most elements of a row: the launchers and kernels round these up to whole tiles and step past
// the end by part of one in 32 bits.
constexpr int32_t kMaxRows = 0x7FFFFFFF - 1023, kMaxK = 1 << 30;

// Counts a launch; with profiling on, times it.
struct Launch {
    void* rec = nullptr;
    Launch(moe_ctx* C, int kind, double bytes, double flops, cudaStream_t s) {
        if (ctx_profiling(C))
            rec = ctx_launch_begin(C, kind, bytes, flops, s);
        else
            ctx_count_launch(C);
    }
    ~Launch() {
        if (rec) ctx_launch_end(rec);
    }
};

moe_status quant(const char* who, moe_ctx* C, const void* x, int64_t x_stride, moe_dtype dtype, int32_t n, int32_t k,
                 void* codes, int64_t code_stride, float* scales, int64_t scale_stride, bool weight, void* stream) {
    if (!C) return set_error(MOE_EINVAL, "%s: ctx is NULL", who);
    if (!type_ok(dtype)) return set_error(MOE_EINVAL, "%s: dtype %d (MOE_F32, MOE_F16 or MOE_BF16)", who, (int)dtype);
    if (n < 0 || n > kMaxRows || k < 16 || k % 16 || k > kMaxK)
        return set_error(MOE_EINVAL, "%s: n = %d, k = %d (n at most 2^31 - 1024; k a multiple of 16, 16 to 2^30)", who, n, k);
    if (n == 0) return MOE_OK;
    if ((int64_t)(weight ? blocks(n) : n) * blocks(k) >= ((int64_t)1 << 31) - 1024)
        return set_error(MOE_EINVAL, "%s: more than 2^31 - 1024 blocks", who);
    if (!x || !codes || !scales) return set_error(MOE_EINVAL, "%s: NULL argument", who);
    if (!rows_ok(x, x_stride, 0, dtype) || !at16(codes) || code_stride % 16 || !at4(scales))
        return set_error(MOE_EINVAL, "%s: rows of x and of codes must start on 16-byte boundaries", who);
    if (code_stride < k && n > 1) return set_error(MOE_EINVAL, "%s: rows of codes overlap", who);
    if (weight ? scale_stride < blocks(k) && blocks(n) > 1 : scale_stride < n && blocks(k) > 1)
        return set_error(MOE_EINVAL, "%s: rows of scales overlap", who);
    CUDA_TRY(cudaSetDevice(ctx_device(C)));
    QuantArgs a{};
    a.x = x;
    a.x_stride = x_stride, a.code_stride = code_stride, a.scale_stride = scale_stride;
    a.codes = static_cast<uint8_t*>(codes);
    a.scales = scales;
    a.n = n, a.dim = k;
    a.type = dtype;
    cudaStream_t s = (cudaStream_t)stream;
    Launch l(C, K_F8_QUANT, (double)n * k * (type_size(dtype) + 1) + 4.0 * (weight ? blocks(n) : n) * blocks(k), 0, s);
    CUDA_TRY(weight ? launch_f8_quant_weight(a, s) : launch_f8_quant_rows(a, ctx_sms(C), s));
    return MOE_OK;
}

}  // namespace

extern "C" moe_status moe_rms_norm(moe_ctx* C, const moe_norm_args* p, void* stream) {
    const char* who = "moe_rms_norm";
    if (!C || !p) return set_error(MOE_EINVAL, "%s: NULL argument", who);
    if (!type_ok(p->x_dtype) || (p->residual && !type_ok(p->residual_dtype)) || (p->weight && !type_ok(p->weight_dtype)) ||
        (p->out && !type_ok(p->out_dtype)))
        return set_error(MOE_EINVAL, "%s: a dtype is not MOE_F32, MOE_F16 or MOE_BF16", who);
    if (p->n_tokens < 0 || p->n_heads < 1 || p->dim < 16 || p->dim % 16 || p->dim > kNormMaxDim)
        return set_error(MOE_EINVAL, "%s: n_tokens = %d, n_heads = %d, dim = %d (dim a multiple of 16, 16 to %d)", who,
                         p->n_tokens, p->n_heads, p->dim, kNormMaxDim);
    if ((int64_t)p->n_tokens * p->n_heads >= (int64_t)1 << 31)
        return set_error(MOE_EINVAL, "%s: n_tokens * n_heads must be below 2^31", who);
    if (!(p->eps >= 0.0f) || !isfinite(p->eps)) return set_error(MOE_EINVAL, "%s: eps must be finite, not negative", who);
    if (p->n_tokens == 0) return MOE_OK;
    if (!p->out && !p->codes && !p->sum) return set_error(MOE_EINVAL, "%s: no output", who);
    if (p->sum && !p->residual) return set_error(MOE_EINVAL, "%s: sum without a residual", who);
    if (p->codes && (p->n_heads != 1 || !p->scales))
        return set_error(MOE_EINVAL, "%s: codes need scales, and n_heads = 1", who);
    if (!p->x) return set_error(MOE_EINVAL, "%s: NULL argument", who);
    if (!rows_ok(p->x, p->x_token_stride, p->x_head_stride, p->x_dtype) ||
        (p->residual && !rows_ok(p->residual, p->residual_token_stride, p->residual_head_stride, p->residual_dtype)) ||
        (p->sum && !rows_ok(p->sum, p->sum_token_stride, p->sum_head_stride, p->residual_dtype)) ||
        (p->out && !rows_ok(p->out, p->out_token_stride, p->out_head_stride, p->out_dtype)) || (p->weight && !at16(p->weight)) ||
        (p->codes && (!at16(p->codes) || p->code_stride % 16 || !at4(p->scales))))
        return set_error(MOE_EINVAL, "%s: rows, weight and codes must start on 16-byte boundaries", who);
    if (p->codes && ((p->code_stride < p->dim && p->n_tokens > 1) || (p->scale_stride < p->n_tokens && p->dim > kF8Block)))
        return set_error(MOE_EINVAL, "%s: rows of codes or of scales overlap", who);
    CUDA_TRY(cudaSetDevice(ctx_device(C)));
    NormArgs a{};
    a.x = p->x, a.res = p->residual, a.weight = p->weight, a.sum = p->sum, a.out = p->out;
    a.codes = static_cast<uint8_t*>(p->codes);
    a.scales = p->scales;
    a.xt = p->x_token_stride, a.xh = p->x_head_stride, a.rt = p->residual_token_stride, a.rh = p->residual_head_stride;
    a.st = p->sum_token_stride, a.sh = p->sum_head_stride, a.ot = p->out_token_stride, a.oh = p->out_head_stride;
    a.ct = p->code_stride, a.scale_stride = p->scale_stride;
    a.rows = (unsigned)p->n_tokens * (unsigned)p->n_heads;
    a.dim = p->dim;
    a.eps = p->eps;
    a.inv_dim = 1.0f / (float)p->dim;
    a.by_head = FastDiv((uint32_t)p->n_heads);
    a.x_type = p->x_dtype, a.res_type = p->residual_dtype, a.weight_type = p->weight_dtype, a.out_type = p->out_dtype;
    double per = type_size(p->x_dtype);
    if (p->residual) per += type_size(p->residual_dtype);
    if (p->sum) per += type_size(p->residual_dtype);
    if (p->out) per += type_size(p->out_dtype);
    if (p->codes) per += 1.0 + 4.0 / kF8Block;
    cudaStream_t s = (cudaStream_t)stream;
    Launch l(C, K_RMS_NORM, per * a.rows * a.dim, 0, s);
    CUDA_TRY(launch_rms_norm(a, ctx_sms(C), s));
    return MOE_OK;
}

extern "C" moe_status moe_f8_quant_rows(moe_ctx* C, const void* x, int64_t x_stride, moe_dtype dtype, int32_t n,
                                        int32_t k, void* codes, int64_t code_stride, float* scales,
                                        int64_t scale_stride, void* stream) {
    return quant("moe_f8_quant_rows", C, x, x_stride, dtype, n, k, codes, code_stride, scales, scale_stride, false, stream);
}

extern "C" moe_status moe_f8_quant_weight(moe_ctx* C, const void* w, int64_t w_stride, moe_dtype dtype, int32_t n,
                                          int32_t k, void* codes, int64_t code_stride, float* scales,
                                          int64_t scale_stride, void* stream) {
    return quant("moe_f8_quant_weight", C, w, w_stride, dtype, n, k, codes, code_stride, scales, scale_stride, true, stream);
}

extern "C" moe_status moe_f8_matmul(moe_ctx* C, const moe_f8_matmul_args* p, void* stream) {
    const char* who = "moe_f8_matmul";
    if (!C || !p) return set_error(MOE_EINVAL, "%s: NULL argument", who);
    if (!type_ok(p->out_dtype))
        return set_error(MOE_EINVAL, "%s: out_dtype %d (MOE_F32, MOE_F16 or MOE_BF16)", who, (int)p->out_dtype);
    if (p->m < 0 || p->m > kMaxRows || p->n < 1 || p->n > kMaxRows || p->k < 16 || p->k % 16 || p->k > kMaxK)
        return set_error(MOE_EINVAL, "%s: m = %d, n = %d, k = %d (m and n at most 2^31 - 1024; k a multiple of 16, 16 to 2^30)", who,
                         p->m, p->n, p->k);
    if (p->m == 0) return MOE_OK;
    if ((int64_t)blocks(p->m) * blocks(p->n) >= (int64_t)1 << 29)
        return set_error(MOE_EINVAL, "%s: m = %d by n = %d is too large", who, p->m, p->n);
    if (!p->a || !p->a_scales || !p->w || !p->w_scales || !p->out) return set_error(MOE_EINVAL, "%s: NULL argument", who);
    if (!at16(p->a) || p->a_stride % 16 || !at16(p->w) || p->w_stride % 16)
        return set_error(MOE_EINVAL, "%s: rows of a and w must start on 16-byte boundaries", who);
    if (p->a_stride < p->k || p->w_stride < p->k || p->a_stride >= (int64_t)1 << 40 || p->w_stride >= (int64_t)1 << 40)
        return set_error(MOE_EINVAL, "%s: strides of a and w must be at least k = %d, below 2^40", who, p->k);
    if (!at4(p->a_scales) || !at4(p->w_scales) || (reinterpret_cast<uintptr_t>(p->out) & (type_size(p->out_dtype) - 1)))
        return set_error(MOE_EINVAL, "%s: scales and out must be aligned to their elements", who);
    if ((p->a_scale_stride < p->m && blocks(p->k) > 1) || (p->w_scale_stride < blocks(p->k) && blocks(p->n) > 1))
        return set_error(MOE_EINVAL, "%s: rows of scales overlap", who);
    if (p->out_stride < p->n && p->m > 1) return set_error(MOE_EINVAL, "%s: rows of out overlap", who);
    CUDA_TRY(cudaSetDevice(ctx_device(C)));
    if (const unsigned code = *ctx_f8_word(C))  // for moe_f8_check to take back: the call that failed may be another thread's
        return set_error(MOE_ETIMEOUT, "%s: a bounded device wait expired in an earlier product (code %u; moe_f8_check)", who, code);
    MatmulArgs a{};
    a.a = static_cast<const uint8_t*>(p->a), a.w = static_cast<const uint8_t*>(p->w);
    a.sa = p->a_scales, a.sw = p->w_scales;
    a.out = p->out;
    a.a_stride = p->a_stride, a.w_stride = p->w_stride, a.sa_stride = p->a_scale_stride, a.sw_stride = p->w_scale_stride;
    a.out_stride = p->out_stride;
    a.m = p->m, a.n = p->n, a.k = p->k;
    a.type = p->out_dtype;
    a.err = ctx_f8_err(C);
    cudaStream_t s = (cudaStream_t)stream;
    const double m = p->m, n = p->n, k = p->k;
    Launch l(C, K_F8_MATMUL, m * k + n * k + m * n * type_size(p->out_dtype) + 4.0 * blocks(p->k) * (m + blocks(p->n)),
             2 * m * n * k, s);
    CUDA_TRY(launch_f8_matmul(a, ctx_sms(C), s));
    return MOE_OK;
}

extern "C" moe_status moe_f8_check(moe_ctx* C) {
    if (!C) return set_error(MOE_EINVAL, "moe_f8_check: ctx is NULL");
    if (const unsigned code = __atomic_exchange_n(const_cast<unsigned*>(ctx_f8_word(C)), 0u, __ATOMIC_RELAXED))
        return set_error(MOE_ETIMEOUT, "a bounded device wait expired in an earlier product (code %u)", code);
    return MOE_OK;
}

extern "C" moe_status moe_ctx_inject_f8_timeout(moe_ctx* C) {
    if (!C) return set_error(MOE_EINVAL, "moe_ctx_inject_f8_timeout: ctx is NULL");
    *ctx_f8_word(C) = 1u;
    return MOE_OK;
}
