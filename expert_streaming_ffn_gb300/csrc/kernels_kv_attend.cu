// Attention over the 4-bit cache: one warp per new token and query head.
#include <cuda_bf16.h>

#include "kv_internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

template <class T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<__half>(__half x) {
    return __half2float(x);
}
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) {
    return __bfloat162float(x);
}
template <class T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ __half from_f<__half>(float x) {
    return __float2half_rn(x);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

template <int D, class T>
__global__ void __launch_bounds__(128) kv_attend_kernel(const __grid_constant__ KvAttend a) {
    constexpr int NG = D / 64;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (w >= (int64_t)a.n_q * a.Hq) return;
    const int row = (int)(w / a.Hq), hq = (int)(w % a.Hq), h = hq / a.G;
    int b = 0, n = a.T, first = 0;
    if (a.q_start) {
        int hi = a.B - 1;
        while (b < hi) {  // the last sequence that starts at or before the row
            const int mid = (b + hi + 1) >> 1;
            if (a.q_start[mid] <= row)
                b = mid;
            else
                hi = mid - 1;
        }
        first = a.q_start[b];
        n = a.q_start[b + 1] - first;
    } else {
        b = row / a.T;
        first = b * a.T;
    }
    const int len = min(a.kv_len[b], a.max_pages << a.c.page_shift);
    const int pos = len - n + (row - first);
    const int hi = a.causal ? min(len, pos + 1) : len;
    const int lo = a.window && pos >= a.window ? pos - a.window + 1 : 0;
    // lane: words lane, lane + 32, ... of the row (8 elements each)
    constexpr int W = D / 8;
    const bool act = lane < W;
    float q[8], acc[8] = {};
    const int i = lane / NG, g = lane % NG;
    const T* qp = static_cast<const T*>(a.q) + (int64_t)row * a.qt + (int64_t)hq * a.qh + g * 64 + i * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = act ? to_f<T>(qp[e]) * a.scale_log2 : 0.0f;
    float m = -INFINITY, l = 0.0f;
    for (int j = lo; j < hi; ++j) {
        const int page = a.table[(int64_t)b * a.table_stride + (j >> a.c.page_shift)];
        if ((unsigned)page >= (unsigned)a.c.n_pages) {
            *(volatile unsigned*)a.bad = 1u;
            continue;
        }
        const int place = j & (a.c.P - 1), r = place & 15;
        const uint8_t* rec = a.c.pages + (((size_t)page * a.c.H + h) * (a.c.P >> 4) + (place >> 4)) * kv_record_bytes(D);
        float z = 0.0f, v[8];
        if (act) {
            const uint32_t kw = reinterpret_cast<const uint32_t*>(rec)[r * W + lane];
            const uint32_t vw = reinterpret_cast<const uint32_t*>(rec + kv_v_codes(D))[r * W + lane];
            const __half2 ka = *reinterpret_cast<const __half2*>(rec + kv_k_affine(D) + (r * NG + g) * 4);
            const __half2 va = *reinterpret_cast<const __half2*>(rec + kv_v_affine(D) + (r * NG + g) * 4);
            const float2 kf = __half22float2(ka), vf = __half22float2(va);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int nb = 4 * ((e & 1) * 4 + (e >> 1));
                z = fmaf(q[e], fmaf(kf.x, (float)((kw >> nb) & 15u), kf.y), z);
                v[e] = fmaf(vf.x, (float)((vw >> nb) & 15u), vf.y);
            }
        }
#pragma unroll
        for (int s = 16; s; s >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, s);
        const float mn = fmaxf(m, z);
        const float c = m == -INFINITY ? 0.0f : exp2f(m - mn), p = exp2f(z - mn);
        l = fmaf(l, c, p);
        m = mn;
        if (act) {
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = fmaf(acc[e], c, p * v[e]);
        }
    }
    if (act) {
        T* op = static_cast<T*>(a.out) + (int64_t)row * a.ot + (int64_t)hq * a.oh + g * 64 + i * 8;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int e = 0; e < 8; ++e) op[e] = from_f<T>(acc[e] * inv);
    }
    if (a.lse && lane == 0) a.lse[(int64_t)row * a.Hq + hq] = l == 0.0f ? -INFINITY : 0.6931471805599453f * (m + log2f(l));
}

}  // namespace

cudaError_t launch_kv_attend(const KvAttend& a, int d, moe_dtype t, cudaStream_t s) {
    const unsigned grid = (unsigned)(((int64_t)a.n_q * a.Hq + 3) / 4);
    const bool bf = t == MOE_BF16;
    if (d == 64)
        bf ? kv_attend_kernel<64, __nv_bfloat16><<<grid, 128, 0, s>>>(a) : kv_attend_kernel<64, __half><<<grid, 128, 0, s>>>(a);
    else if (d == 128)
        bf ? kv_attend_kernel<128, __nv_bfloat16><<<grid, 128, 0, s>>>(a) : kv_attend_kernel<128, __half><<<grid, 128, 0, s>>>(a);
    else
        bf ? kv_attend_kernel<256, __nv_bfloat16><<<grid, 128, 0, s>>>(a) : kv_attend_kernel<256, __half><<<grid, 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
