// Rows of keys and values into the 4-bit cache and back.
#include <cuda_bf16.h>

#include "kv_internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr float kF16Max = 65504.0f;

template <class T>
struct Row8;  // eight consecutive elements of a row

template <>
struct Row8<__nv_bfloat16> {
    static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&x)[8]) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <>
struct Row8<__half> {
    static __device__ __forceinline__ void load(const __half* p, float (&x)[8]) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ void store(__half* p, const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <>
struct Row8<float> {
    static __device__ __forceinline__ void load(const float* p, float (&x)[8]) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    static __device__ __forceinline__ void store(float* p, const float (&x)[8]) {
        reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
};

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Eight elements of a group, one thread of the eight that hold it: the word of
// their codes, and the group's affine word. Called by whole groups.
__device__ __forceinline__ uint32_t quantise8(float (&x)[8], uint32_t& affine) {
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = min_nan(lo, x[i]);
        hi = max_nan(hi, x[i]);
    }
#pragma unroll
    for (int m = 4; m; m >>= 1) {
        lo = min_nan(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, m));
        hi = max_nan(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, m));
    }
    // the clamp commutes with min and max; NaN passes through both
    lo = max_nan(min_nan(lo, kF16Max), -kF16Max);
    hi = max_nan(min_nan(hi, kF16Max), -kF16Max);
    const __half b16 = __float2half_rd(lo);
    const float b = __half2float(b16);
    const __half s16 = __float2half_ru(__fdiv_rn(__fsub_rn(hi, b), 15.0f));
    const float s = __half2float(s16);
    affine = (uint32_t)__half_as_ushort(s16) | ((uint32_t)__half_as_ushort(b16) << 16);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float c = fmaxf(fminf(x[i], kF16Max), -kF16Max);
        const float q = s > 0.0f ? rintf(__fdiv_rn(__fsub_rn(c, b), s)) : 0.0f;
        // element e = {0,2,4,6,1,3,5,7}[n] in nibble n
        const int n = (i & 1) * 4 + (i >> 1);
        word |= (uint32_t)(int)q << (4 * n);
    }
    return word;
}

// Thread e of the D/8 threads of a row takes elements 8e .. 8e+7 of K and V.
template <int D, class T>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ KvRows a) {
    constexpr int kPer = D / 8, NG = D / 64;
    const uint64_t idx = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
    const unsigned row = (unsigned)(idx / kPer);
    const int e = (int)(idx % kPer);
    const bool in = row < a.n;
    const unsigned t = a.by_head.div(in ? row : 0), h = (in ? row : 0) - t * a.by_head.d;
    float k[8], v[8];
    Row8<T>::load(static_cast<const T*>(a.k_in) + (int64_t)t * a.kt + (int64_t)h * a.kh + e * 8, k);
    Row8<T>::load(static_cast<const T*>(a.v_in) + (int64_t)t * a.vt + (int64_t)h * a.vh + e * 8, v);
    const int slot = __ldg(a.slots + t);
    uint32_t ka, va;
    const uint32_t kw = quantise8(k, ka), vw = quantise8(v, va);
    if (!in || slot < 0) return;
    if ((unsigned)slot >= a.c.n_slots) {
        *(volatile unsigned*)a.bad = 1u;
        return;
    }
    const int page = slot >> a.c.page_shift, place = slot & (a.c.P - 1), r = place & 15;
    uint8_t* rec = a.c.pages + (((size_t)page * a.c.H + h) * (a.c.P >> 4) + (place >> 4)) * kv_record_bytes(D);
    const int g = e >> 3, i = e & 7;
    const int word = r * (D / 8) + i * NG + g;
    reinterpret_cast<uint32_t*>(rec)[word] = kw;
    reinterpret_cast<uint32_t*>(rec + kv_v_codes(D))[word] = vw;
    if (i == 0) {
        reinterpret_cast<uint32_t*>(rec + kv_k_affine(D))[r * NG + g] = ka;
        reinterpret_cast<uint32_t*>(rec + kv_v_affine(D))[r * NG + g] = va;
    }
}

__device__ __forceinline__ void dequantise8(uint32_t w, uint32_t affine, float (&x)[8]) {
    const float s = __half2float(__ushort_as_half((unsigned short)(affine & 0xFFFFu)));
    const float b = __half2float(__ushort_as_half((unsigned short)(affine >> 16)));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int n = (i & 1) * 4 + (i >> 1);
        x[i] = fmaf(s, (float)((w >> (4 * n)) & 15u), b);
    }
}

template <int D, class T>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const __grid_constant__ KvRows a) {
    constexpr int kPer = D / 8, NG = D / 64;
    const uint64_t idx = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
    const unsigned row = (unsigned)(idx / kPer);
    const int e = (int)(idx % kPer);
    if (row >= a.n) return;
    const unsigned t = a.by_head.div(row), h = row - t * a.by_head.d;
    const int slot = __ldg(a.slots + t);
    float k[8] = {}, v[8] = {};
    if (slot >= 0 && (unsigned)slot < a.c.n_slots) {
        const int page = slot >> a.c.page_shift, place = slot & (a.c.P - 1), r = place & 15;
        const uint8_t* rec =
            a.c.pages + (((size_t)page * a.c.H + h) * (a.c.P >> 4) + (place >> 4)) * kv_record_bytes(D);
        const int g = e >> 3, i = e & 7;
        const int word = r * (D / 8) + i * NG + g;
        const uint32_t kw = reinterpret_cast<const uint32_t*>(rec)[word];
        const uint32_t vw = reinterpret_cast<const uint32_t*>(rec + kv_v_codes(D))[word];
        dequantise8(kw, reinterpret_cast<const uint32_t*>(rec + kv_k_affine(D))[r * NG + g], k);
        dequantise8(vw, reinterpret_cast<const uint32_t*>(rec + kv_v_affine(D))[r * NG + g], v);
    } else if (slot >= 0) {
        *(volatile unsigned*)a.bad = 1u;
    }
    Row8<T>::store(static_cast<T*>(a.k_out) + (int64_t)t * a.kt + (int64_t)h * a.kh + e * 8, k);
    Row8<T>::store(static_cast<T*>(a.v_out) + (int64_t)t * a.vt + (int64_t)h * a.vh + e * 8, v);
}

template <int D, class T>
cudaError_t launch_rows(const KvRows& a, bool append, cudaStream_t s) {
    const uint64_t threads = (uint64_t)a.n * (D / 8);
    const unsigned grid = (unsigned)((threads + kThreads - 1) / kThreads);
    if (append)
        kv_append_kernel<D, T><<<grid, kThreads, 0, s>>>(a);
    else
        kv_read_kernel<D, T><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_rows_of(const KvRows& a, moe_dtype t, bool append, cudaStream_t s) {
    if (t == MOE_BF16) return launch_rows<D, __nv_bfloat16>(a, append, s);
    if (t == MOE_F16) return launch_rows<D, __half>(a, append, s);
    return launch_rows<D, float>(a, append, s);
}

cudaError_t launch_any(const KvRows& a, int d, moe_dtype t, bool append, cudaStream_t s) {
    return d == 64 ? launch_rows_of<64>(a, t, append, s) : d == 128 ? launch_rows_of<128>(a, t, append, s)
                                                                    : launch_rows_of<256>(a, t, append, s);
}

}  // namespace

cudaError_t launch_kv_append(const KvRows& a, int d, moe_dtype t, cudaStream_t s) {
    return launch_any(a, d, t, true, s);
}
cudaError_t launch_kv_read(const KvRows& a, int d, moe_dtype t, cudaStream_t s) {
    return launch_any(a, d, t, false, s);
}

}  // namespace moe
