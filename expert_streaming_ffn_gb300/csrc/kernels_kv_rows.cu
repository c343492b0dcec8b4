// Rows of keys and values into the 4-bit cache and back.
#include <cuda_bf16.h>

#include "kv_internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr float kF16Max = 65504.0f;

// Eight consecutive elements of a row, as loaded.
template <class T>
struct Row8;

template <class T>
struct Row8Pairs {  // 16-bit types
    uint32_t w[4];
    __device__ __forceinline__ void load(const T* p) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
};

template <>
struct Row8<__nv_bfloat16> : Row8Pairs<__nv_bfloat16> {
    using Pair = __nv_bfloat162;
    __device__ __forceinline__ uint64_t two(int i) const {
        return ptx::f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
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
struct Row8<__half> : Row8Pairs<__half> {
    using Pair = __half2;
    __device__ __forceinline__ uint64_t two(int i) const {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        return ptx::f2(f.x, f.y);
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
    float x[8];
    __device__ __forceinline__ void load(const float* p) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *(reinterpret_cast<const float4*>(p) + 1);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    __device__ __forceinline__ uint64_t two(int i) const { return ptx::f2(x[2 * i], x[2 * i + 1]); }
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

// The least and the largest of a group's 64 elements, of which each of eight
// lanes holds eight; NaN if there is one. 16-bit types work in pairs, the largest
// negated, so that one exchange a step serves both.
__device__ __forceinline__ float2 group_range(const Row8<float>& r) {
    float lo = r.x[0], hi = r.x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = min_nan(lo, r.x[i]);
        hi = max_nan(hi, r.x[i]);
    }
#pragma unroll
    for (int m = 4; m; m >>= 1) {
        lo = min_nan(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, m));
        hi = max_nan(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, m));
    }
    return make_float2(lo, hi);
}

template <class R>
__device__ __forceinline__ float2 group_range(const R& r) {
    using P = typename R::Pair;
    auto pair = [](uint32_t w) { return *reinterpret_cast<const P*>(&w); };
    auto word = [](P p) { return *reinterpret_cast<const uint32_t*>(&p); };
    const P lo = __hmin2_nan(__hmin2_nan(pair(r.w[0]), pair(r.w[1])), __hmin2_nan(pair(r.w[2]), pair(r.w[3])));
    const P hi = __hmax2_nan(__hmax2_nan(pair(r.w[0]), pair(r.w[1])), __hmax2_nan(pair(r.w[2]), pair(r.w[3])));
    // (least, largest negated) of the even elements, and of the odd ones
    const uint32_t neg = word(hi) ^ 0x80008000u;
    P p = __hmin2_nan(pair(__byte_perm(word(lo), neg, 0x5410)), pair(__byte_perm(word(lo), neg, 0x7632)));
#pragma unroll
    for (int m = 4; m; m >>= 1) p = __hmin2_nan(p, pair(__shfl_xor_sync(0xFFFFFFFFu, word(p), m)));
    return make_float2((float)p.x, -(float)p.y);
}

// Eight elements of a group, one lane of the eight that hold it: the word of
// their codes, and the group's affine word. Called by whole warps.
// The quotient (x - b) / s is IEEE's: t = d y with y = 1 / s rounded to nearest
// is within an ulp of it, and t + y (d - s t), the remainder exact in a fused
// multiply-add, rounds to it (Markstein's theorem; s has 11 bits, so its one exception,
// a divisor of all ones, cannot come up). Adding 1.5 * 2^23 rounds it to an
// integer, ties to even, in the low bits. Two elements go through each instruction.
template <class R>
__device__ __forceinline__ uint32_t quantise8(const R& row, uint32_t& affine) {
    const float2 r = group_range(row);
    float lo = r.x, hi = r.y;
    uint64_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = row.two(i);
    if (lo < -kF16Max || hi > kF16Max) {  // held as +-65504; NaN is left as it is
        lo = max_nan(min_nan(lo, kF16Max), -kF16Max);
        hi = max_nan(min_nan(hi, kF16Max), -kF16Max);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = ptx::f2(x[i]);
            x[i] = ptx::f2(fmaxf(fminf(v.x, kF16Max), -kF16Max), fmaxf(fminf(v.y, kF16Max), -kF16Max));
        }
    }
    const __half b16 = __float2half_rd(lo);
    const float b = __half2float(b16);
    const __half s16 = __float2half_ru(__fdiv_rn(__fsub_rn(hi, b), 15.0f));
    const float s = __half2float(s16), y = s > 0.0f ? __frcp_rn(s) : 0.0f;
    affine = (uint32_t)__half_as_ushort(s16) | ((uint32_t)__half_as_ushort(b16) << 16);
    const uint64_t nb = ptx::f2(-b, -b), ns = ptx::f2(-s, -s), yy = ptx::f2(y, y), magic = ptx::f2(12582912.0f, 12582912.0f);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t d = ptx::add2(x[i], nb), t = ptx::mul2(d, yy);
        const float2 q = ptx::f2(ptx::add2(ptx::fma2(ptx::fma2(t, ns, d), yy, t), magic));
        // elements 2i, 2i + 1 in nibbles i, i + 4; what the sums carry besides is taken off at the end
        word += (__float_as_uint(q.x) << (4 * i)) + (__float_as_uint(q.y) << (4 * i + 16));
    }
    uint32_t carried = 0;
#pragma unroll
    for (int n = 0; n < 8; ++n) carried += 0x4B400000u << (4 * n);
    return s > 0.0f ? word - carried : 0;
}

// N consecutive words, one store
template <int N>
__device__ __forceinline__ void store_words(uint32_t* p, const uint32_t (&w)[N]) {
    if constexpr (N == 4)
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (N == 2)
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else
        *p = w[0];
}
template <int N>
__device__ __forceinline__ void load_words(const uint32_t* p, uint32_t (&w)[N]) {
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = *p;
    }
}

// Rows into records, in one pass: a group's range by exchanges between its eight
// lanes, then codes by quantise8. Eight threads a row: thread i takes elements
// 8i .. 8i+7 of every group of K and V. Their words are neighbours in the record,
// a group's eight threads read 128 bytes side by side, and the whole row is in
// flight before the first exchange. (D / 8 threads a row, eight elements of K and V each,
// every quotient a division of its own, took 94 us below.)
//
// 32,768 tokens of 8 heads of 128 in bf16, 134 MB in and 38 MB out: 35.8 us, 4.8 TB/s,
// 0.72 of the copy bandwidth measured on this GPU. Bound by issue slots: 74.6 % of
// the cycles issue. From fp32 46.4 us, 6.6 TB/s (0.99), bound by HBM. 1 token: 2.4 us, the launch.
template <int D, class T>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ KvRows a) {
    constexpr int NG = D / 64;
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const uint64_t idx = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
    const unsigned row = (unsigned)(idx >> 3);
    const int i = (int)(idx & 7);
    const bool in = row < a.n;
    const unsigned t = a.by_head.div(in ? row : 0), h = (in ? row : 0) - t * a.by_head.d;
    const T* kp = static_cast<const T*>(a.k_in) + (int64_t)t * a.kt + (int64_t)h * a.kh + i * 8;
    const T* vp = static_cast<const T*>(a.v_in) + (int64_t)t * a.vt + (int64_t)h * a.vh + i * 8;
    Row8<T> k[NG], v[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) k[g].load(kp + g * 64);
#pragma unroll
    for (int g = 0; g < NG; ++g) v[g].load(vp + g * 64);
    const int slot = a.slots[t];
    uint32_t ka[NG], va[NG], kw[NG], vw[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        kw[g] = quantise8(k[g], ka[g]);
        vw[g] = quantise8(v[g], va[g]);
    }
    if (!in || slot < 0) return;
    if ((unsigned)slot >= a.c.n_slots) {
        *(volatile unsigned*)a.bad = 1u;
        return;
    }
    const int page = slot >> a.c.page_shift, place = slot & (a.c.P - 1), r = place & 15;
    uint8_t* rec = a.c.pages + (((size_t)page * a.c.H + h) * (a.c.P >> 4) + (place >> 4)) * kv_record_bytes(D);
    store_words<NG>(reinterpret_cast<uint32_t*>(rec) + r * (D / 8) + i * NG, kw);
    store_words<NG>(reinterpret_cast<uint32_t*>(rec + kv_v_codes(D)) + r * (D / 8) + i * NG, vw);
    if (i == 0) store_words<NG>(reinterpret_cast<uint32_t*>(rec + kv_k_affine(D)) + r * NG, ka);
    if (i == 1) store_words<NG>(reinterpret_cast<uint32_t*>(rec + kv_v_affine(D)) + r * NG, va);
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

// Records into rows, s q + b in one fused multiply-add, by the same eight threads a row: each row's
// words come in whole before any is used, and its stores are 16 bytes a thread, 128 a group.
// Bound by HBM: 65,536 tokens of 8 heads of 128 to bf16, 75 MB in and 268 MB out, 53.6 us, 6.4 TB/s,
// 0.96 of the measured copy bandwidth; 32,768 of them 28.4 us (0.91), to fp32 63 us (0.72).
template <int D, class T>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const __grid_constant__ KvRows a) {
    constexpr int NG = D / 64;
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const uint64_t idx = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
    const unsigned row = (unsigned)(idx >> 3);
    const int i = (int)(idx & 7);
    if (row >= a.n) return;
    const unsigned t = a.by_head.div(row), h = row - t * a.by_head.d;
    const int slot = a.slots[t];
    uint32_t kw[NG] = {}, vw[NG] = {}, ka[NG] = {}, va[NG] = {};  // zeros where there is nothing
    if ((unsigned)slot < a.c.n_slots) {
        const int page = slot >> a.c.page_shift, place = slot & (a.c.P - 1), r = place & 15;
        const uint8_t* rec =
            a.c.pages + (((size_t)page * a.c.H + h) * (a.c.P >> 4) + (place >> 4)) * kv_record_bytes(D);
        load_words<NG>(reinterpret_cast<const uint32_t*>(rec) + r * (D / 8) + i * NG, kw);
        load_words<NG>(reinterpret_cast<const uint32_t*>(rec + kv_v_codes(D)) + r * (D / 8) + i * NG, vw);
        load_words<NG>(reinterpret_cast<const uint32_t*>(rec + kv_k_affine(D)) + r * NG, ka);
        load_words<NG>(reinterpret_cast<const uint32_t*>(rec + kv_v_affine(D)) + r * NG, va);
    } else if (slot >= 0) {
        *(volatile unsigned*)a.bad = 1u;
    }
    T* kp = static_cast<T*>(a.k_out) + (int64_t)t * a.kt + (int64_t)h * a.kh + i * 8;
    T* vp = static_cast<T*>(a.v_out) + (int64_t)t * a.vt + (int64_t)h * a.vh + i * 8;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        float x[8];
        dequantise8(kw[g], ka[g], x);
        Row8<T>::store(kp + g * 64, x);
        dequantise8(vw[g], va[g], x);
        Row8<T>::store(vp + g * 64, x);
    }
}

template <int D, class T>
cudaError_t launch_rows(const KvRows& a, bool append, cudaStream_t s) {
    const unsigned grid = (unsigned)(((uint64_t)a.n * 8 + kThreads - 1) / kThreads);
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = launch_config(dim3(grid), dim3(kThreads), 0, s, true, &attr);
    return append ? cudaLaunchKernelEx(&cfg, kv_append_kernel<D, T>, a) : cudaLaunchKernelEx(&cfg, kv_read_kernel<D, T>, a);
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
