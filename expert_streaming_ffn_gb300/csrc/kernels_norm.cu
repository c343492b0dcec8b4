// Root-mean-square norm of rows, with the residual's addition and an 8-bit output, and quantisation to 8 bits.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "dense_internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr float kE4m3Max = 448.0f;
constexpr float kLeast = 448.0f * 1.17549435e-38f;  // a block's largest magnitude counts as at least this: no scale is subnormal
constexpr float kSmallScale = 0x1p-90f, kUp = 0x1p64f;  // blocks of smaller scales are divided with both sides taken kUp times

// Eight consecutive elements of B bytes each, as loaded.
template <int B>
struct Raw {
    uint32_t w[2 * B];
    __device__ __forceinline__ void load(const void* base, int64_t at) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + at * B);
#pragma unroll
        for (int i = 0; i < B / 2; ++i) {
            const uint4 v = p[i];
            w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 2 * B; ++i) w[i] = 0;
    }
    // the values, by pairs; `bf` tells the 16-bit types apart
    __device__ __forceinline__ void get(uint64_t (&f)[4], bool bf) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (B == 4) {
                f[i] = ptx::f2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
            } else if (bf) {
                f[i] = ptx::f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
            } else {
                const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                f[i] = ptx::f2(v.x, v.y);
            }
        }
    }
};
template <>
struct Raw<0> {
    __device__ __forceinline__ void load(const void*, int64_t) {}
    __device__ __forceinline__ void zero() {}
};

// Eight values to memory, rounded once to the type.
__device__ __forceinline__ void store8(void* base, int64_t at, const uint64_t (&f)[4], moe_dtype t) {
    if (t == MOE_F32) {
        ulonglong2* p = reinterpret_cast<ulonglong2*>(static_cast<float*>(base) + at);
        p[0] = make_ulonglong2(f[0], f[1]);
        p[1] = make_ulonglong2(f[2], f[3]);
        return;
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = ptx::f2(f[i]);
        if (t == MOE_BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __half2 h = __floats2half2_rn(v.x, v.y);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float largest8(const uint64_t (&f)[4]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = ptx::f2(f[i]);
        m = max_nan(m, max_nan(fabsf(v.x), fabsf(v.y)));
    }
    return m;
}
// Of raw elements; 16-bit types by pairs.
__device__ __forceinline__ float largest8(const Raw<4>& v, bool) {
    uint64_t f[4];
    v.get(f, false);
    return largest8(f);
}
__device__ __forceinline__ float largest8(const Raw<2>& v, bool bf) {
    uint32_t m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = v.w[i] & 0x7FFF7FFFu;
    // (as magnitudes, halves compare like unsigned integers, and NaN above all)
    const uint32_t p = __vmaxu2(__vmaxu2(m[0], m[1]), __vmaxu2(m[2], m[3]));
    const uint32_t top = max(p & 0xFFFFu, p >> 16);
    return bf ? __uint_as_float(top << 16) : __half2float(__ushort_as_half((unsigned short)top));
}

// The scale of a block by its largest magnitude, and 1 / scale. An infinity or a NaN makes the whole block NaN.
// The division by 448 is IEEE's: the product with 1 / 448 rounded to nearest is within an ulp of the quotient, and one
// step with the remainder, exact in a fused multiply-add, rounds to it (Markstein's theorem). 1 / scale is the
// approximation's after a Newton step, within an ulp.
__device__ __forceinline__ float block_scale(float largest, float& inv) {
    constexpr float r = 1.0f / kE4m3Max;
    const float top = fmaxf(largest, kLeast), t = top * r;
    float s = fmaf(fmaf(t, -kE4m3Max, top), r, t);
    if (!(largest < __int_as_float(0x7F800000))) s = __int_as_float(0x7FC00000);
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
    inv = fmaf(fmaf(-s, y, 1.0f), y, y);
    return s;
}

// Eight values to codes, the fp32 quotients f / s rounded. t = f y with y = 1 / s is within two ulps of the quotient, and in
// t + y (f - s t) the remainder is exact in a fused multiply-add, so that the sum before its rounding is within 2^-21 ulp of
// the quotient: ties between codes, which are short numbers, come out as such. A plain product f y would move them, and
// 16-bit inputs have many. (Exact as long as the remainder's last place is in fp32's range: for t of 2^-10, half the least
// code, it is 2^-56 of s, which 2^-149 allows for s from 2^-93 on; for smaller ones the quantisers take small_codes8. The norm does
// not: its values are products rounded before, so that a tie is chance, and two multiplies a pair took 2 % of 32,768 x 2,816 from bf16.)
__device__ __forceinline__ uint2 codes8(const uint64_t (&f)[4], float s, float inv) {
    uint32_t h[4];
    const uint64_t yy = ptx::f2(inv, inv), ns = ptx::f2(-s, -s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t t = ptx::mul2(f[i], yy);
        const float2 q = ptx::f2(ptx::fma2(ptx::fma2(t, ns, f[i]), yy, t));
        uint16_t c;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(q.y), "f"(q.x));
        h[i] = c;
    }
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// Rows by groups of G threads, U rows a group, all loaded before the first is used: a thread holds V vectors of eight
// elements of each, vector i + v * G for thread i. kCta: the group is the CTA; else G = 8, 16 or 32 lanes of a warp.
// One pass: a row stays in registers between its sum of squares (exchanges in a warp, then through shared memory) and its
// outputs, and a block of 128 elements is 16 neighbouring vectors, so its largest magnitude is an exchange of 16 lanes.
//
// Bound by HBM: 32,768 rows of 2,816, fp32 plus a bf16 residual into bf16 sums and 8 bits, 833 MB: 117.5 us, 7.1 TB/s, 1.06
// of the copy bandwidth measured on this GPU; from bf16 100.6 us (0.96). 4,099 tokens of 32 heads of 128, 67 MB: 13.0 us
// (0.77), of which about 3 are the launch and the ends. One row of 2,816 with four outputs: 2.2 us, the launch. Bound by
// instructions: bf16 into bf16 and codes, 32,768 of 640 25.6 us (15.7 of bytes), where 48 of a warp's 128 places hold no vector
// and are computed all the same, and 20,000 of 1,008 18.5 us (15.1).
template <int XB, int RB, int V, int U, bool kCta>
__global__ void __launch_bounds__(!kCta ? 256 : V == 4 ? 1024 : 512) norm_kernel(const __grid_constant__ NormArgs a, const int group) {
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int G = kCta ? (int)blockDim.x : group;
    const unsigned per = kCta ? 1 : blockDim.x / (unsigned)group;
    const int i = kCta ? (int)threadIdx.x : (int)threadIdx.x & (G - 1);
    const unsigned first = kCta ? blockIdx.x * U : blockIdx.x * (per * U) + threadIdx.x / (unsigned)G;
    const int nv = a.dim >> 3;
    unsigned t[U], h[U];
    bool live[U];
    Raw<XB> x[U][V];
    Raw<RB> r[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const unsigned row = first + u * per;
        live[u] = row < a.rows;
        t[u] = a.by_head.div(live[u] ? row : 0);
        h[u] = (live[u] ? row : 0) - t[u] * a.by_head.d;
        const int64_t xo = (int64_t)t[u] * a.xt + (int64_t)h[u] * a.xh, ro = (int64_t)t[u] * a.rt + (int64_t)h[u] * a.rh;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int j = i + v * G;
            if (live[u] && j < nv) {
                x[u][v].load(a.x, xo + 8 * j);
                r[u][v].load(a.res, ro + 8 * j);
            } else {
                x[u][v].zero();
                r[u][v].zero();
            }
        }
    }
    uint64_t f[U][V][4];
    float ss[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        uint64_t sum = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            x[u][v].get(f[u][v], a.x_type == MOE_BF16);
            if constexpr (RB != 0) {
                uint64_t g[4];
                r[u][v].get(g, a.res_type == MOE_BF16);
#pragma unroll
                for (int e = 0; e < 4; ++e) f[u][v][e] = ptx::add2(f[u][v][e], g[e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) sum = ptx::fma2(f[u][v][e], f[u][v][e], sum);
        }
        const float2 two = ptx::f2(sum);
        ss[u] = two.x + two.y;
    }
    for (int m = (kCta ? 32 : G) >> 1; m; m >>= 1)
#pragma unroll
        for (int u = 0; u < U; ++u) ss[u] += __shfl_xor_sync(kFull, ss[u], m);
    if constexpr (kCta) {
        __shared__ float part[U][32];
        const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0)
#pragma unroll
            for (int u = 0; u < U; ++u) part[u][threadIdx.x >> 5] = ss[u];
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            ss[u] = lane < warps ? part[u][lane] : 0.0f;
#pragma unroll
            for (int m = 16; m; m >>= 1) ss[u] += __shfl_xor_sync(kFull, ss[u], m);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int j = i + v * G;
        uint64_t w[4] = {};
        if (a.weight && j < nv) {
            if (a.weight_type == MOE_F32) {
                Raw<4> q;
                q.load(a.weight, 8 * j);
                q.get(w, false);
            } else {
                Raw<2> q;
                q.load(a.weight, 8 * j);
                q.get(w, a.weight_type == MOE_BF16);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = live[u] && j < nv;
            uint64_t(&y)[4] = f[u][v];
            if constexpr (RB != 0)
                if (a.sum && in) store8(a.sum, (int64_t)t[u] * a.st + (int64_t)h[u] * a.sh + 8 * j, y, a.res_type);
            const float k = rsqrtf(fmaf(ss[u], a.inv_dim, a.eps));
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = ptx::mul2(y[e], ptx::f2(k, k));
            if (a.weight)
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = ptx::mul2(y[e], w[e]);
            if (a.out && in) store8(a.out, (int64_t)t[u] * a.ot + (int64_t)h[u] * a.oh + 8 * j, y, a.out_type);
            if (a.codes) {  // a block is 16 neighbouring vectors, so 16 lanes of a warp (8 where a row has no more)
                float top = largest8(y);
                for (int m = min(16, G) >> 1; m; m >>= 1) top = max_nan(top, __shfl_xor_sync(kFull, top, m));
                float inv;
                const float s = block_scale(top, inv);
                if (in) {
                    *reinterpret_cast<uint2*>(a.codes + (int64_t)t[u] * a.ct + 8 * j) = codes8(y, s, inv);
                    if ((j & 15) == 0) a.scales[(int64_t)(j >> 4) * a.scale_stride + t[u]] = s;
                }
            }
        }
    }
}

template <int XB, int RB, int V, int U, bool kCta>
cudaError_t launch_norm(const NormArgs& a, unsigned threads, int group, cudaStream_t s) {
    const unsigned per = (kCta ? 1 : threads / group) * U;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = launch_config(dim3((a.rows + per - 1) / per), dim3(threads), 0, s, true, &attr);
    return cudaLaunchKernelEx(&cfg, norm_kernel<XB, RB, V, U, kCta>, a, group);
}

// Up to 512 elements a row goes to a warp or a part of one, more to a CTA; up to 1,024 to a warp too where rows are many.
// Many rows: several vectors a thread, so that more loads are under way for as many exchanges between threads; few: one, as
// a row's time counts. us, one and two (at 6,144 two and four) vectors a thread of a CTA: 32,768 rows of 2,816, fp32 into 8
// bits with a bf16 residual 125 117, from bf16 114 96 (no weights); 16,384 of 4,096, bf16: 53.7 42.0; of 2,048: 25.0 21.2; of 6,144:
// 63.9 60.5; 64 rows of 4,096: 1.9 1.7. Rows of 128 by two a half warp: 12.1 (one 14.0, four 12.3).
template <int XB, int RB>
cudaError_t launch_norm_of(const NormArgs& a, int sms, cudaStream_t s) {
    const int nv = a.dim >> 3;
    const bool many = (uint64_t)a.rows * nv >= (uint64_t)sms * 2048 * 2;  // twice what the SMs' threads take at once
    if (nv <= 32) {
        const int G = nv <= 8 ? 8 : nv <= 16 ? 16 : 32;
        return many ? launch_norm<XB, RB, 1, 2, false>(a, 256, G, s) : launch_norm<XB, RB, 1, 1, false>(a, 256, G, s);
    }
    if (nv <= 64) return many ? launch_norm<XB, RB, 2, 2, false>(a, 256, 32, s) : launch_norm<XB, RB, 2, 1, false>(a, 256, 32, s);
    if (nv <= 128 && many) return launch_norm<XB, RB, 4, 1, false>(a, 256, 32, s);
    const unsigned v = nv <= (many ? 0 : 384) ? 1 : nv <= (many ? 512 : 1024) ? 2 : 4;
    const unsigned threads = (unsigned)((nv + v - 1) / v + 31) / 32 * 32;
    return v == 1 ? launch_norm<XB, RB, 1, 1, true>(a, threads, 0, s)
                  : v == 2 ? launch_norm<XB, RB, 2, 1, true>(a, threads, 0, s) : launch_norm<XB, RB, 4, 1, true>(a, threads, 0, s);
}

template <int XB>
cudaError_t launch_norm_of(const NormArgs& a, int sms, cudaStream_t s) {
    return !a.res ? launch_norm_of<XB, 0>(a, sms, s)
                  : a.res_type == MOE_F32 ? launch_norm_of<XB, 4>(a, sms, s) : launch_norm_of<XB, 2>(a, sms, s);
}

// The codes of a block whose scale is below kSmallScale. The kernels below write these a second time, behind everything else and
// from memory again, so that others pay one comparison a vector: with a branch for each vector 16,385 x 4,096 from fp16 took 40.7 us
// in place of 34.8, from registers kept for it 38.4.
__device__ __forceinline__ uint2 small_codes8(uint64_t (&f)[4], float s, float inv) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = ptx::mul2(f[i], ptx::f2(kUp, kUp));
    return codes8(f, s * kUp, inv * (1.0f / kUp));
}

// A block's largest magnitude, from its 16 lanes; `mask` has all lanes that are here.
template <int B>
__device__ __forceinline__ float block_top(const Raw<B>& x, bool bf, unsigned mask) {
    float top = largest8(x, bf);
#pragma unroll
    for (int m = 8; m; m >>= 1) top = max_nan(top, __shfl_xor_sync(mask, top, m));
    return top;
}

// Rows to codes: 16 lanes a block, eight elements each. V vectors a thread, a CTA's threads apart, so that 64 bytes a
// thread are under way.
// 16,385 rows of 4,096, fp16: 35.6 us, 5.66 TB/s, 0.85 of the copy bandwidth; issue slots 73 % busy. From fp32 47.8 us (1.05),
// bound by HBM. 64 rows: 1.4 us, the launch.
template <int B, int V>
__global__ void __launch_bounds__(256) quant_rows_kernel(const __grid_constant__ QuantArgs a) {
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const uint64_t first = (uint64_t)blockIdx.x * (256 * V) + threadIdx.x;
    const unsigned per = a.by_row.d;
    Raw<B> x[V];
    int row[V], vec[V];
    bool in[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const uint64_t at = first + 256 * v;
        row[v] = (int)a.by_row.div((uint32_t)(at >> 4));
        vec[v] = (int)((at >> 4) - (uint64_t)row[v] * per) * 16 + (int)(at & 15);
        in[v] = row[v] < a.n && 8 * vec[v] < a.dim;
        if (in[v])
            x[v].load(a.x, (int64_t)row[v] * a.x_stride + 8 * vec[v]);
        else
            x[v].zero();
    }
    float least = kSmallScale;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float top = block_top(x[v], a.type == MOE_BF16, kFull);
        float inv;
        const float s = block_scale(top, inv);
        least = fminf(least, s);
        if (!in[v]) continue;
        uint64_t f[4];
        x[v].get(f, a.type == MOE_BF16);
        *reinterpret_cast<uint2*>(a.codes + (int64_t)row[v] * a.code_stride + 8 * vec[v]) = codes8(f, s, inv);
        if ((vec[v] & 15) == 0) a.scales[(int64_t)(vec[v] >> 4) * a.scale_stride + row[v]] = s;
    }
    if (least < kSmallScale) {  // of all 16 lanes of a block: its codes a second time
        const unsigned lanes = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll 1
        for (int v = 0; v < V; ++v) {
            const uint64_t at = first + 256 * v;
            const int r = (int)a.by_row.div((uint32_t)(at >> 4)), j = (int)((at >> 4) - (uint64_t)r * per) * 16 + (int)(at & 15);
            const bool live = r < a.n && 8 * j < a.dim;
            Raw<B> again;
            if (live)
                again.load(a.x, (int64_t)r * a.x_stride + 8 * j);
            else
                again.zero();
            float inv;
            const float s = block_scale(block_top(again, a.type == MOE_BF16, lanes), inv);
            uint64_t f[4];
            again.get(f, a.type == MOE_BF16);
            if (live && s < kSmallScale) *reinterpret_cast<uint2*>(a.codes + (int64_t)r * a.code_stride + 8 * j) = small_codes8(f, s, inv);
        }
    }
}

// A block of 128 x 128 weights a CTA, in registers between the pass for its largest magnitude and the pass for its codes.
// 10,000 x 2,864, fp32: 24.7 us, 5.8 TB/s, 0.87 of the copy bandwidth; from bf16 14.4 us (0.89). What is left is a CTA's two
// passes one after the other, three (bf16: four) of them on an SM.
template <int B>
__global__ void __launch_bounds__(256) quant_weight_kernel(const __grid_constant__ QuantArgs a) {
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int nb = (int)a.by_row.div(blockIdx.x), kb = (int)(blockIdx.x - (unsigned)nb * a.by_row.d);
    const int i = threadIdx.x & 15, r0 = nb * kF8Block + (threadIdx.x >> 4), col = kb * kF8Block + 8 * i;
    Raw<B> x[8];
#pragma unroll
    for (int v = 0; v < 8; ++v) {
        if (r0 + 16 * v < a.n && col < a.dim)
            x[v].load(a.x, (int64_t)(r0 + 16 * v) * a.x_stride + col);
        else
            x[v].zero();
    }
    float top = 0.0f;
#pragma unroll
    for (int v = 0; v < 8; ++v) top = max_nan(top, largest8(x[v], a.type == MOE_BF16));
#pragma unroll
    for (int m = 16; m; m >>= 1) top = max_nan(top, __shfl_xor_sync(kFull, top, m));
    __shared__ float part[8];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) top = max_nan(top, part[w]);
    float inv;
    const float s = block_scale(top, inv);
    if (threadIdx.x == 0) a.scales[(int64_t)nb * a.scale_stride + kb] = s;
#pragma unroll
    for (int v = 0; v < 8; ++v) {
        if (r0 + 16 * v >= a.n || col >= a.dim) continue;
        uint64_t f[4];
        x[v].get(f, a.type == MOE_BF16);
        *reinterpret_cast<uint2*>(a.codes + (int64_t)(r0 + 16 * v) * a.code_stride + col) = codes8(f, s, inv);
    }
    if (s < kSmallScale) {
#pragma unroll 1
        for (int v = 0; v < 8; ++v) {
            if (r0 + 16 * v >= a.n || col >= a.dim) continue;
            Raw<B> again;
            again.load(a.x, (int64_t)(r0 + 16 * v) * a.x_stride + col);
            uint64_t f[4];
            again.get(f, a.type == MOE_BF16);
            *reinterpret_cast<uint2*>(a.codes + (int64_t)(r0 + 16 * v) * a.code_stride + col) = small_codes8(f, s, inv);
        }
    }
}

template <int B, int V>
cudaError_t launch_quant_rows(const QuantArgs& a, uint64_t vecs, cudaStream_t s) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg =
        launch_config(dim3((unsigned)((vecs + 256 * V - 1) / (256 * V))), dim3(256), 0, s, true, &attr);
    return cudaLaunchKernelEx(&cfg, quant_rows_kernel<B, V>, a);
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& a, int sms, cudaStream_t s) {
    return a.x_type == MOE_F32 ? launch_norm_of<4>(a, sms, s) : launch_norm_of<2>(a, sms, s);
}

cudaError_t launch_f8_quant_rows(const QuantArgs& a0, int sms, cudaStream_t s) {
    QuantArgs a = a0;
    a.by_row = FastDiv((uint32_t)((a.dim + kF8Block - 1) / kF8Block));
    const uint64_t vecs = (uint64_t)a.n * a.by_row.d * 16;
    const bool many = vecs >= (uint64_t)sms * 2048 * 4;
    if (a.type == MOE_F32) return many ? launch_quant_rows<4, 2>(a, vecs, s) : launch_quant_rows<4, 1>(a, vecs, s);
    return many ? launch_quant_rows<2, 4>(a, vecs, s) : launch_quant_rows<2, 1>(a, vecs, s);
}

cudaError_t launch_f8_quant_weight(const QuantArgs& a0, cudaStream_t s) {
    QuantArgs a = a0;
    a.by_row = FastDiv((uint32_t)((a.dim + kF8Block - 1) / kF8Block));
    cudaLaunchAttribute attr;
    const dim3 grid(a.by_row.d * (unsigned)((a.n + kF8Block - 1) / kF8Block));
    const cudaLaunchConfig_t cfg = launch_config(grid, dim3(256), 0, s, true, &attr);
    return a.type == MOE_F32 ? cudaLaunchKernelEx(&cfg, quant_weight_kernel<4>, a)
                             : cudaLaunchKernelEx(&cfg, quant_weight_kernel<2>, a);
}

}  // namespace moe
