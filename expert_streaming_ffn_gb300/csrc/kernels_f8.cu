// Matrix product of 8-bit rows and 8-bit weights on the 5th-generation tensor cores (sm_103a).
//
//   out[m][n] = sum over K-blocks of 128 of  sa[kb][m] sw[n / 128][kb] sum_{k in kb} a[m][k] w[n][k]
//
// tcgen05.mma multiplies e4m3 codes and sums them in fp32; as every K-block has scales of its own, a K-block's sums go
// to an accumulator buffer in tensor memory of their own, and epilogue warps add scale * sum into fp32 registers. The
// tensor cores work on the next K-blocks meanwhile.
//
// A CTA's tile has 128 lanes (the MMA's M) and C columns (its N). Two forms:
//   rows form (many rows): lanes are rows, columns 256 weights. A lane's scale is its row's times the weights' block's.
//   weights form (few rows): lanes are 128 weights, which share a scale, columns up to C rows (16, 32, 64 or 128), so
//     that no tensor work or memory goes to rows that are not there. K is split over the CTAs of a cluster where tiles
//     are few, and each of them adds a share of the columns through distributed shared memory, in a fixed order.
//
// Warps: E epilogue warps (warp q mod 4 reads TMEM lanes 32 (q mod 4) on), one warp that loads both operands by TMA
// into a ring of K-blocks (128 bytes a row, 128-byte swizzle), one that issues the MMAs.
// Every wait is bounded; when one expires the kernel sets an error word, every other wait gives up, its own copies and
// MMAs in flight are waited for and its tensor memory is freed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>

#include "dense_internal.h"
#include "ptx.cuh"
#include "tc_operand.cuh"

namespace moe {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kLanes = 128;
constexpr int kLaneBytes = kLanes * 128;  // of a K-block: 128 rows of 128 codes

template <int C_, bool kRows_>
struct Form {
    static constexpr int C = C_;
    static constexpr bool kRows = kRows_;  // lanes are rows
    static constexpr int kEpi = kRows ? 8 : 4;
    static constexpr int kThreads = 32 * (kEpi + 2);
    static constexpr int kPer = kRows ? C / 2 : C;  // columns of an epilogue thread
    static constexpr int kStageBytes = kLaneBytes + C * 128;
    static constexpr int kStages = kRows ? 4 : C == 16 ? 6 : C == 32 ? 5 : C == 64 ? 4 : 6;
    static constexpr int kBufs = kRows ? 2 : 4;
    static constexpr int kTmem = kBufs * C;
    static constexpr int kChunk = C == 128 ? 8 : 16;  // weights form: K-blocks of row scales held at a time, twice
    static constexpr int kScaleBytes = kRows ? 0 : 2 * kChunk * C * 4;
    static constexpr int kSmem = 1024 + kStages * kStageBytes + kScaleBytes + 256;
    static constexpr int kCtas = !kRows && C <= 64 ? 2 : 1;  // resident on an SM
    static_assert(kTmem >= 32 && kTmem * kCtas <= 512 && (kTmem & (kTmem - 1)) == 0, "tensor memory");
    static_assert(kSmem * kCtas <= 232448 - 1024 * (kCtas - 1), "shared memory");
    static_assert(kRows || kStages * kStageBytes >= C * kLanes * 4, "partial sums of a split lie in the ring");
};

struct Tiles {
    int lanes, cols;  // tiles that way
    int total;
    int kblocks;
    int splits;
};

__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor: e4m3 A and B (type 0), both K-major, fp32 D, M x N.
__device__ __forceinline__ uint32_t f8_idesc(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// 32 lanes x 16 columns, as eight register pairs
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* v) {
    ptx::tmem_ld16(taddr, *reinterpret_cast<uint32_t(*)[16]>(v));
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_peer(uint32_t addr, uint32_t rank) {
    float v;
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ void store1(void* out, int64_t at, float v, moe_dtype t) {
    if (t == MOE_F32)
        static_cast<float*>(out)[at] = v;
    else if (t == MOE_BF16)
        static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
    else
        static_cast<__half*>(out)[at] = __float2half_rn(v);
}

__device__ __forceinline__ uint32_t pack2(float x, float y, moe_dtype t) {
    if (t == MOE_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// N consecutive elements of a row from fp32 pairs, the first `n` of them; `wide`: on 16-byte boundaries.
template <int N>
__device__ __forceinline__ void store_row(void* out, int64_t at, const uint64_t (&v)[N / 2], int n, bool wide, moe_dtype t) {
    if (n >= N && wide) {
        if (t == MOE_F32) {
            float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
#pragma unroll
            for (int i = 0; i < N / 4; ++i) {
                const float2 x = ptx::f2(v[2 * i]), y = ptx::f2(v[2 * i + 1]);
                p[i] = make_float4(x.x, x.y, y.x, y.y);
            }
        } else {
            uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at);
#pragma unroll
            for (int i = 0; i < N / 8; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 x = ptx::f2(v[4 * i + j]);
                    w[j] = pack2(x.x, x.y, t);
                }
                p[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float2 x = ptx::f2(v[i]);
        if (2 * i < n) store1(out, at + 2 * i, x.x, t);
        if (2 * i + 1 < n) store1(out, at + 2 * i + 1, x.y, t);
    }
}

template <class F>
__global__ void __launch_bounds__(F::kThreads, F::kCtas)
    f8_matmul_kernel(const __grid_constant__ MatmulArgs a, const __grid_constant__ Tiles T,
                     const __grid_constant__ CUtensorMap map_lanes, const __grid_constant__ CUtensorMap map_cols) {
    constexpr int C = F::C, kStages = F::kStages, kBufs = F::kBufs, kPer = F::kPer, kChunk = F::kChunk;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* ring =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    float* scales = reinterpret_cast<float*>(ring + kStages * F::kStageBytes);  // [2][kChunk][C]
    uint64_t* full = reinterpret_cast<uint64_t*>(ring + kStages * F::kStageBytes + F::kScaleBytes);
    uint64_t* empty = full + kStages;
    uint64_t* acc_full = empty + kStages;
    uint64_t* acc_empty = acc_full + kBufs;
    uint64_t* drain = acc_empty + kBufs;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    __shared__ int abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(full + i, 1);
            ptx::mbar_init(empty + i, 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            ptx::mbar_init(acc_full + i, 1);
            ptx::mbar_init(acc_empty + i, F::kEpi);
        }
        ptx::mbar_init(drain, 1);
        abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&map_lanes);
        ptx::prefetch_tensormap(&map_cols);
    }
    if (warp == F::kEpi) {
        ptx::tmem_alloc(tmem_slot, F::kTmem);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    volatile int* abortp = &abort_flag;
    auto fail = [&](unsigned bit) {
        if (!*abortp) *(volatile unsigned*)a.err = bit;
        abort_flag = 1;
    };
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();

    const int rank = T.splits > 1 ? (int)cluster_rank() : 0;
    const int kb0 = (int)((int64_t)T.kblocks * rank / T.splits), kb1 = (int)((int64_t)T.kblocks * (rank + 1) / T.splits);
    const int first = (int)blockIdx.x / T.splits, step = (int)gridDim.x / T.splits;
    // neighbouring tiles go along the lanes' operand 16 deep, so that tiles of one time share both operands in L2
    auto place = [&](int t, int& lt, int& ct) {
        const int group = 16 * T.cols, g = t / group, deep = min(16, T.lanes - 16 * g), r = t - g * group;
        ct = r / deep;
        lt = 16 * g + (r - ct * deep);
    };

    if (warp == F::kEpi) {
        if (lane == 0) {
            // ---------------- loads ----------------
            int st = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = first; t < T.total && ok; t += step) {
                int lt, ct;
                place(t, lt, ct);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!ptx::mbar_wait_sleep(empty + st, ph ^ 1, abortp)) {
                        fail(1u);
                        ok = false;
                        break;
                    }
                    unsigned char* p = ring + st * F::kStageBytes;
                    ptx::mbar_arrive_expect_tx(full + st, F::kStageBytes);
                    ptx::tma_load_2d(p, &map_lanes, kb * 128, lt * kLanes, full + st);
                    ptx::tma_load_2d(p + kLaneBytes, &map_cols, kb * 128, ct * C, full + st);
                    ++issued;
                    if (++st == kStages) {
                        st = 0;
                        ph ^= 1;
                    }
                }
            }
            // no copy may land after the CTA has gone
            for (int i = 0; i < kStages && i < issued; ++i) {
                const int sl = st - 1 - i < 0 ? st - 1 - i + kStages : st - 1 - i;
                ptx::mbar_wait_bounded(full + sl, st - 1 - i < 0 ? ph ^ 1 : ph, nullptr);
            }
        }
    } else if (warp == F::kEpi + 1) {
        if (lane == 0) {
            // ---------------- MMA issue ----------------
            const uint32_t idesc = f8_idesc(kLanes, C);
            const uint64_t d0 = sw128_desc(ptx::smem_addr(ring));
            int st = 0, buf = 0;
            uint32_t ph = 0, bph = 0;
            bool ok = true;
            for (int t = first; t < T.total && ok; t += step) {
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!ptx::mbar_wait_bounded(full + st, ph, abortp) ||
                        !ptx::mbar_wait_bounded(acc_empty + buf, bph ^ 1, abortp)) {
                        fail(2u);
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint64_t ad = d0 + (uint64_t)((st * F::kStageBytes) >> 4), bd = ad + (kLaneBytes >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)  // K = 32 an MMA: 32 bytes on in the swizzled rows
                        mma_f8_ss(tmem + buf * C, ad + 2 * k, bd + 2 * k, idesc, k > 0);
                    ptx::mma_commit(empty + st);
                    ptx::mma_commit(acc_full + buf);
                    if (++st == kStages) {
                        st = 0;
                        ph ^= 1;
                    }
                    if (++buf == kBufs) {
                        buf = 0;
                        bph ^= 1;
                    }
                }
            }
            ptx::mma_commit(drain);
            ptx::mbar_wait_bounded(drain, 0, nullptr);
        }
    } else {
        // ---------------- epilogue ----------------
        const int q = warp & 3, half = warp >> 2;  // rows form: warps 4-7 take the second half of the columns
        const uint32_t taddr = tmem + ((uint32_t)(32 * q) << 16) + half * kPer;
        int buf = 0;
        uint32_t bph = 0;
        bool ok = true;
        const bool wide = !(reinterpret_cast<uintptr_t>(a.out) & 15) && a.out_stride % (a.type == MOE_F32 ? 4 : 8) == 0;
        for (int t = first; t < T.total; t += step) {
            int lt, ct;
            place(t, lt, ct);
            uint64_t acc[kPer / 2];
#pragma unroll
            for (int i = 0; i < kPer / 2; ++i) acc[i] = 0;
            const int lrow = lt * kLanes + 32 * q + lane;  // this thread's lane: a row, or a weight
            if constexpr (F::kRows) {
                const bool in = lrow < a.m;
                const int nb = ct * (C / kF8Block) + half;
                const bool nin = nb * kF8Block < a.n;
                const float* sa = a.sa + (in ? lrow : 0);
                const float* sw = a.sw + (nin ? (int64_t)nb * a.sw_stride : 0);
                float s_next[4], w_lane = 0.0f;
                auto fetch = [&](int kb) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s_next[i] = in && kb + i < kb1 ? sa[(int64_t)(kb + i) * a.sa_stride] : 0.0f;
                };
                fetch(kb0);
                for (int kb = kb0; kb < kb1 && ok; kb += 4) {
                    if (((kb - kb0) & 31) == 0) w_lane = nin && kb + lane < kb1 ? sw[kb + lane] : 0.0f;
                    float s_now[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) s_now[i] = s_next[i];
                    fetch(kb + 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (kb + i >= kb1) break;
                        const float sc = s_now[i] * __shfl_sync(kFull, w_lane, (kb + i - kb0) & 31);
                        if (!__all_sync(kFull, ptx::mbar_wait_sleep(acc_full + buf, bph, abortp))) {
                            if (lane == 0) fail(4u);
                            ok = false;
                            break;
                        }
                        ptx::tc_fence_after();
                        const uint64_t s2 = ptx::f2(sc, sc);
                        const uint32_t at = taddr + buf * C;
                        uint32_t d[2][16];
                        tmem_ld16(at, d[0]);
#pragma unroll
                        for (int c = 0; c < kPer / 16; ++c) {
                            ptx::tmem_ld_wait();
                            if (c + 1 < kPer / 16) tmem_ld16(at + 16 * (c + 1), d[(c + 1) & 1]);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                acc[8 * c + e] = ptx::fma2(
                                    ptx::f2(__uint_as_float(d[c & 1][2 * e]), __uint_as_float(d[c & 1][2 * e + 1])), s2,
                                    acc[8 * c + e]);
                        }
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(acc_empty + buf);
                        if (++buf == kBufs) {
                            buf = 0;
                            bph ^= 1;
                        }
                    }
                }
                if (ok && in) {
                    const int n0 = ct * C + half * kPer;
                    if (n0 < a.n) store_row<kPer>(a.out, (int64_t)lrow * a.out_stride + n0, acc, a.n - n0, wide, a.type);
                }
            } else {
                const bool nin = lt * kLanes < a.n;
                const float* sw = a.sw + (nin ? (int64_t)lt * a.sw_stride : 0);
                const int m0 = ct * C;
                // row scales, kChunk K-blocks at a time, a chunk ahead
                auto fetch = [&](int kb, int half_of) {
                    for (int i = threadIdx.x; i < kChunk * C; i += 32 * F::kEpi) {
                        const int b = kb + i / C, r = m0 + i % C;
                        const bool in = b < kb1 && r < a.m;
                        cp_async4(ptx::smem_addr(scales + half_of * kChunk * C + i),
                                  a.sa + (in ? (int64_t)b * a.sa_stride + r : 0), in);
                    }
                    cp_async_commit();
                };
                fetch(kb0, 0);
                float w_lane = 0.0f;
                int turn = 0;
                for (int kb = kb0; kb < kb1; ++kb) {  // to the end even after a failed wait: the warps meet at barriers
                    const int i = (kb - kb0) % kChunk;
                    if (i == 0) {
                        // the last chunk's readers are done before its place is written again
                        if (kb > kb0) turn ^= 1;
                        ptx::named_sync(1, 32 * F::kEpi);
                        fetch(kb + kChunk, turn ^ 1);
                        cp_async_wait<1>();
                        ptx::named_sync(1, 32 * F::kEpi);
                    }
                    if (((kb - kb0) & 31) == 0) w_lane = kb + lane < kb1 ? sw[kb + lane] : 0.0f;
                    const float ws = __shfl_sync(kFull, w_lane, (kb - kb0) & 31);
                    const uint64_t w2 = ptx::f2(ws, ws);
                    if (ok && !__all_sync(kFull, ptx::mbar_wait_sleep(acc_full + buf, bph, abortp))) {
                        if (lane == 0) fail(4u);
                        ok = false;
                    }
                    if (ok) {
                        ptx::tc_fence_after();
                        const uint32_t at = taddr + buf * C;
                        const uint32_t sp = ptx::smem_addr(scales + (turn * kChunk + i) * C);
                        uint32_t d[2][16];
                        tmem_ld16(at, d[0]);
#pragma unroll
                        for (int c = 0; c < kPer / 16; ++c) {
                            ptx::tmem_ld_wait();
                            if (c + 1 < kPer / 16) tmem_ld16(at + 16 * (c + 1), d[(c + 1) & 1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float4 s4 = ptx::lds_f4(sp + 64 * c + 16 * e);
                                acc[8 * c + 2 * e] = ptx::fma2(
                                    ptx::f2(__uint_as_float(d[c & 1][4 * e]), __uint_as_float(d[c & 1][4 * e + 1])),
                                    ptx::mul2(ptx::f2(s4.x, s4.y), w2), acc[8 * c + 2 * e]);
                                acc[8 * c + 2 * e + 1] = ptx::fma2(
                                    ptx::f2(__uint_as_float(d[c & 1][4 * e + 2]), __uint_as_float(d[c & 1][4 * e + 3])),
                                    ptx::mul2(ptx::f2(s4.z, s4.w), w2), acc[8 * c + 2 * e + 1]);
                            }
                        }
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(acc_empty + buf);
                        if (++buf == kBufs) {
                            buf = 0;
                            bph ^= 1;
                        }
                    }
                }
                cp_async_wait<0>();
                if (T.splits == 1) {
                    if (ok && lrow < a.n) {
#pragma unroll
                        for (int c = 0; c < C / 2; ++c) {
                            const float2 v = ptx::f2(acc[c]);
                            if (m0 + 2 * c < a.m) store1(a.out, (int64_t)(m0 + 2 * c) * a.out_stride + lrow, v.x, a.type);
                            if (m0 + 2 * c + 1 < a.m)
                                store1(a.out, (int64_t)(m0 + 2 * c + 1) * a.out_stride + lrow, v.y, a.type);
                        }
                    }
                    ptx::named_sync(1, 32 * F::kEpi);  // this tile's scales are read before the next tile's come
                } else if (ok) {
                    // the ring is done with: the last accumulator's MMAs have read it
                    float* part = reinterpret_cast<float*>(ring) + 32 * q + lane;
#pragma unroll
                    for (int c = 0; c < C / 2; ++c) {
                        const float2 v = ptx::f2(acc[c]);
                        part[(2 * c) * kLanes] = v.x;
                        part[(2 * c + 1) * kLanes] = v.y;
                    }
                }
            }
        }
    }
    if constexpr (!F::kRows) {
        if (T.splits > 1) {  // one tile a cluster
            __syncwarp();
            cluster_sync();
            int lt, ct;
            place(first, lt, ct);
            if (warp < F::kEpi && !*abortp) {
                const int n = lt * kLanes + 32 * warp + lane, cols = min(C, a.m - ct * C);
                const uint32_t at = ptx::smem_addr(ring) + 4 * (32 * warp + lane);
                for (int c = rank; c < cols; c += T.splits) {
                    float v[8];
#pragma unroll
                    for (int r = 0; r < 8; ++r) v[r] = r < T.splits ? ld_peer(at + c * (kLanes * 4), r) : 0.0f;
#pragma unroll
                    for (int r = 1; r < 8; ++r) v[0] += v[r];
                    if (n < a.n) store1(a.out, (int64_t)(ct * C + c) * a.out_stride + n, v[0], a.type);
                }
            }
            __syncwarp();
            cluster_sync();  // a CTA's part stays until its peers have read it
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == F::kEpi) ptx::tmem_dealloc(tmem, F::kTmem);
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() {
    static EncodeTiled fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiled>(p);
        else
            cudaGetLastError();
    });
    return fn;
}

// Codes [rows][k], rows `stride` bytes apart: boxes of 128 codes by `box` rows, 128-byte swizzle; zeros outside.
cudaError_t encode_codes(CUtensorMap* m, const uint8_t* base, int rows, int k, int64_t stride, int box) {
    EncodeTiled fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride};
    const cuuint32_t b[2] = {128, (cuuint32_t)box};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, b, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <class F>
cudaError_t launch_form(const MatmulArgs& a, int sms, cudaStream_t s) {
    Tiles T;
    const int ln = F::kRows ? a.m : a.n, cn = F::kRows ? a.n : a.m;
    T.lanes = (ln + kLanes - 1) / kLanes;
    T.cols = (cn + F::C - 1) / F::C;
    T.total = T.lanes * T.cols;
    T.kblocks = (a.k + kF8Block - 1) / kF8Block;
    T.splits = 1;
    const int room = sms * F::kCtas;
    if (!F::kRows && T.total < room) T.splits = std::max(1, std::min({8, room / T.total, T.kblocks / 2}));
    CUtensorMap ml, mc;
    cudaError_t e = F::kRows ? encode_codes(&ml, a.a, a.m, a.k, a.a_stride, kLanes)
                             : encode_codes(&ml, a.w, a.n, a.k, a.w_stride, kLanes);
    if (e != cudaSuccess) return e;
    e = F::kRows ? encode_codes(&mc, a.w, a.n, a.k, a.w_stride, F::C) : encode_codes(&mc, a.a, a.m, a.k, a.a_stride, F::C);
    if (e != cudaSuccess) return e;
    e = ensure_smem_attr(reinterpret_cast<const void*>(f8_matmul_kernel<F>), F::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    const unsigned grid = T.splits > 1 ? (unsigned)(T.total * T.splits) : (unsigned)std::min(T.total, room);
    cudaLaunchConfig_t cfg = launch_config(dim3(grid), dim3(F::kThreads), F::kSmem, s, true, attr);
    if (T.splits > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)T.splits;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, f8_matmul_kernel<F>, a, T, ml, mc);
}

}  // namespace

cudaError_t launch_f8_matmul(const MatmulArgs& a, int sms, cudaStream_t s) {
    if (a.m <= 16) return launch_form<Form<16, false>>(a, sms, s);
    if (a.m <= 32) return launch_form<Form<32, false>>(a, sms, s);
    if (a.m <= 64) return launch_form<Form<64, false>>(a, sms, s);
    if (a.m <= 256) return launch_form<Form<128, false>>(a, sms, s);
    return launch_form<Form<256, true>>(a, sms, s);
}

}  // namespace moe
