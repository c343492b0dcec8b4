// Matrix product of 8-bit rows and 8-bit weights on the 5th-generation tensor cores (sm_103a).
//
//   out[m][n] = sum over K-blocks of 128 of  sa[kb][m] sw[n / 128][kb] sum_{k in kb} a[m][k] w[n][k]
//
// The tensor cores multiply e4m3 codes and sum a K-block in fp32; as every K-block has scales of its own, scale * sum is
// added in fp32 registers, K-block by K-block, in order. Three forms (launch_f8_matmul chooses):
//   up to 16 rows and one round of CTAs, K up to 4,096: mma.sync straight from each lane's own copies (f8_few_kernel);
//   weights form (f8_matmul_kernel): tcgen05.mma, 128 weights as its lanes, which share a scale, and 16, 32 or 64 rows as
//     its columns, so that no tensor work or memory goes to rows that are not there;
//   rows form (f8_rows_kernel): tcgen05.mma of CTA pairs, 256 rows as its lanes by 256 weights.
// In the last two a K-block's sums go to a buffer in tensor memory of their own and the tensor cores go on with the next
// ones, while epilogue warps add scale * sum. Where tiles are few the CTAs of a cluster share K and join their sums through
// distributed shared memory, in a fixed order; so the same call gives the same bits.
//
// Weights form, warps: four or eight epilogue warps (warp w reads TMEM lanes 32 (w mod 4) on), one that loads both operands
// by TMA into a ring of K-blocks (128 bytes a row, 128-byte swizzle), one that issues the MMAs.
//   100,003 weights of 2,048 by 5 rows: 33.3 us, 6.2 TB/s, 0.92 of the copy bandwidth measured on this GPU, bound by HBM.
//   2,816 of 4,096 by 77 rows 8.4 us (floor 1.8), 6,144 of 2,816 by 143 9.2 us (2.9): 3 to 4 us of start, first loads
//   and last stores (5 with a join), then 0.27 us a K-block for one CTA on an SM (0.41 for two): an epilogue warp's chain of barrier (120
//   cycles when it is there), load from tensor memory (100), scales and sums. Deeper rings (one CTA on an SM) and sixteen
//   epilogue warps of 16 columns were no faster.
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

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Weights form, up to C rows a tile.
template <int C_>
struct Form {
    static constexpr int C = C_;
    static constexpr int kEpi = C == 16 ? 4 : 8;
    static constexpr int kPer = 4 * C / kEpi;  // columns of an epilogue warp
    static constexpr int kThreads = 32 * (kEpi + 2);
    static constexpr int kStageBytes = kLaneBytes + C * 128;
    static constexpr int kStages = C == 16 ? 6 : C == 32 ? 5 : 4;
    static constexpr int kBufs = 4;
    static constexpr int kTmem = kBufs * C;
    static constexpr int kChunk = 16;  // K-blocks of row scales held at a time, twice
    static constexpr int kScaleBytes = 2 * kChunk * C * 4;
    static constexpr int kSmem = 1024 + kStages * kStageBytes + kScaleBytes + 256;
    static constexpr int kCtas = 2;  // resident on an SM
    static_assert(kTmem >= 32 && kTmem * kCtas <= 512 && (kTmem & (kTmem - 1)) == 0, "tensor memory");
    static_assert(kSmem * kCtas <= 232448 - 1024 * (kCtas - 1), "shared memory");
    static_assert(kStages * kStageBytes >= C * kLanes * 4, "partial sums of a split lie in the ring");
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

// 32 lanes x 32 columns
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr)
        : "memory");
}

// One lane's arrival at a barrier of this CTA.
__device__ __forceinline__ void arrive_one(bool one, uint32_t addr) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t@p mbarrier.arrive.shared::cta.b64 _, [%1];\n\t}" ::"r"((uint32_t)one),
        "r"(addr)
        : "memory");
}

template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A box of a tensor map into L2.
__device__ __forceinline__ void prefetch_box(const void* map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y)
                 : "memory");
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The same for a count that unrolling makes a constant.
__device__ __forceinline__ void cp_async_wait_at_most(int n) {
    if (n == 3)
        cp_async_wait<3>();
    else if (n == 2)
        cp_async_wait<2>();
    else if (n == 1)
        cp_async_wait<1>();
    else
        cp_async_wait<0>();
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same from branches that the cluster's warps come to apart.
__device__ __forceinline__ void cluster_sync_apart() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float4 ld_peer4(uint32_t addr, uint32_t rank) {
    float4 v;
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at)
                 : "memory");
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

// Four consecutive elements of a row, the first `n` of them.
__device__ __forceinline__ void store4(const MatmulArgs& a, int64_t at, const float4& x, int n) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.out) + at * (a.type == MOE_F32 ? 4 : 2);
    if (n >= 4 && !(p & (a.type == MOE_F32 ? 15 : 7))) {
        if (a.type == MOE_F32)
            *reinterpret_cast<float4*>(p) = x;
        else
            *reinterpret_cast<uint2*>(p) = make_uint2(pack2(x.x, x.y, a.type), pack2(x.z, x.w, a.type));
        return;
    }
    if (n > 0) store1(a.out, at, x.x, a.type);
    if (n > 1) store1(a.out, at + 1, x.y, a.type);
    if (n > 2) store1(a.out, at + 2, x.z, a.type);
    if (n > 3) store1(a.out, at + 3, x.w, a.type);
}

// A warp's 32 rows from m0 on by 64 columns from n0 on, a lane a row, to memory by way of `stage` (32 rows x 16 columns in
// shared memory, groups of four swizzled so that neither way has bank conflicts), so that lanes that store side by side
// write a row's neighbouring elements.
__device__ __forceinline__ void store_tile(const MatmulArgs& a, float* stage, int m0, int n0, const uint64_t (&v)[32]) {
    const int lane = threadIdx.x & 31;
    const bool wide = !(reinterpret_cast<uintptr_t>(a.out) & 15) && a.out_stride % (a.type == MOE_F32 ? 4 : 8) == 0 && n0 + 64 <= a.n;
    const int rows = min(32, a.m - m0);
    float4* const mine = reinterpret_cast<float4*>(stage) + 4 * lane;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if (n0 + 16 * c >= a.n) break;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const float2 x = ptx::f2(v[8 * c + 2 * g]), y = ptx::f2(v[8 * c + 2 * g + 1]);
            mine[g ^ ((lane >> 1) & 3)] = make_float4(x.x, x.y, y.x, y.y);
        }
        __syncwarp();
        if (wide) {
#pragma unroll 1
            for (int r = lane >> 2; r < rows; r += 8) {
                const int g = lane & 3;
                store4(a, (int64_t)(m0 + r) * a.out_stride + n0 + 16 * c + 4 * g,
                       reinterpret_cast<const float4*>(stage)[4 * r + (g ^ ((r >> 1) & 3))], 4);
            }
        } else {
            const int e = lane & 15, n = n0 + 16 * c + e;
#pragma unroll 8
            for (int i = 0; i < 16; ++i) {
                const int r = 2 * i + (lane >> 4);
                if (r < rows && n < a.n)
                    store1(a.out, (int64_t)(m0 + r) * a.out_stride + n, stage[16 * r + 4 * ((e >> 2) ^ ((r >> 1) & 3)) + (e & 3)], a.type);
            }
        }
        __syncwarp();
    }
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }

// Element n of `cols` rows from m0 on, from pairs. (Short code per element: a call of one tile runs it once, from memory.)
template <class T, int N>
__device__ __forceinline__ void store_columns(const MatmulArgs& a, int m0, int n, int cols, const uint64_t (&v)[N]) {
    T* p = static_cast<T*>(a.out) + (int64_t)m0 * a.out_stride + n;
#pragma unroll
    for (int c = 0; c < N; ++c) {
        if (2 * c >= cols) break;
        const float2 x = ptx::f2(v[c]);
        put(p, x.x);
        p += a.out_stride;
        if (2 * c + 1 < cols) put(p, x.y);
        p += a.out_stride;
    }
}

template <class F>
__global__ void __launch_bounds__(F::kThreads, F::kCtas)
    f8_matmul_kernel(const __grid_constant__ MatmulArgs a, const __grid_constant__ Tiles T,
                     const __grid_constant__ CUtensorMap map_lanes, const __grid_constant__ CUtensorMap map_cols) {
    constexpr int C = F::C, kPer = F::kPer, kStages = F::kStages, kBufs = F::kBufs, kChunk = F::kChunk;
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

    const int warp = __shfl_sync(kFull, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
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
    const int rank = T.splits > 1 ? (int)cluster_rank() : 0;
    const int kb0 = (int)((int64_t)T.kblocks * rank / T.splits), kb1 = (int)((int64_t)T.kblocks * (rank + 1) / T.splits);
    const int first = (int)blockIdx.x / T.splits, step = (int)gridDim.x / T.splits;
    // neighbouring tiles go along the lanes' operand 16 deep, so that tiles of one time share both operands in L2
    auto place = [&](int t, int& lt, int& ct) {
        const int group = 16 * T.cols, g = t / group, deep = min(16, T.lanes - 16 * g), r = t - g * group;
        ct = r / deep;
        lt = 16 * g + (r - ct * deep);
    };

    // the weights may be what the kernel before writes, so before the wait they are only brought into L2
    if (warp == F::kEpi && lane == 0 && first < T.total) {
        int lt, ct;
        place(first, lt, ct);
        for (int kb = kb0; kb < min(kb1, kb0 + 2 * kStages); ++kb) prefetch_box(&map_lanes, kb * 128, lt * kLanes);
    }
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();

    if (warp >= F::kEpi) {
        if (warp == F::kEpi) {
            // ---------------- loads ----------------
            const bool leader = elect_one();
            int st = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = first; t < T.total && ok; t += step) {
                int lt, ct;
                place(t, lt, ct);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!__all_sync(kFull, ptx::mbar_wait_sleep(empty + st, ph ^ 1, abortp))) {
                        if (leader) fail(1u);
                        ok = false;
                        break;
                    }
                    if (leader) {
                        unsigned char* p = ring + st * F::kStageBytes;
                        ptx::mbar_arrive_expect_tx(full + st, F::kStageBytes);
                        ptx::tma_load_2d(p, &map_lanes, kb * 128, lt * kLanes, full + st);
                        ptx::tma_load_2d(p + kLaneBytes, &map_cols, kb * 128, ct * C, full + st);
                    }
                    __syncwarp();
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
        if (warp == F::kEpi + 1) {
            // ---------------- MMA issue ----------------
            // the whole warp goes round, so that descriptors stay in uniform registers, and one lane issues
            const bool leader = elect_one();
            const uint32_t idesc = f8_idesc(kLanes, C);
            const uint64_t d0 = sw128_desc(ptx::smem_addr(ring));
            int st = 0, buf = 0;
            uint32_t ph = 0, bph = 0;
            bool ok = true;
            for (int t = first; t < T.total && ok; t += step) {
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!__all_sync(kFull, ptx::mbar_wait_sleep(full + st, ph, abortp) &&
                                               ptx::mbar_wait_sleep(acc_empty + buf, bph ^ 1, abortp))) {
                        if (leader) fail(2u);
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint64_t ad = d0 + (uint64_t)((st * F::kStageBytes) >> 4), bd = ad + (kLaneBytes >> 4);
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)  // K = 32 an MMA: 32 bytes on in the swizzled rows
                            mma_f8_ss(tmem + buf * C, ad + 2 * k, bd + 2 * k, idesc, k > 0);
                        ptx::mma_commit(empty + st);
                        ptx::mma_commit(acc_full + buf);
                    }
                    __syncwarp();
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
            if (leader) ptx::mma_commit(drain);
            __syncwarp();
            ptx::mbar_wait_bounded(drain, 0, nullptr);
        }
    } else {
        // ---------------- epilogue ----------------
        const int q = warp & 3, col0 = (warp >> 2) * kPer;  // TMEM lanes 32 q on, columns col0 on
        const uint32_t taddr = tmem + ((uint32_t)(32 * q) << 16) + col0;
        int buf = 0;
        uint32_t bph = 0;
        bool ok = true;
        for (int t = first; t < T.total; t += step) {
            int lt, ct;
            place(t, lt, ct);
            uint64_t acc[kPer / 2];
#pragma unroll
            for (int i = 0; i < kPer / 2; ++i) acc[i] = 0;
            const int lrow = lt * kLanes + 32 * q + lane;  // this thread's lane: a weight
            const float* sw = a.sw + (int64_t)lt * a.sw_stride;
            const int m0 = ct * C;
            // Scales, rows' times weights', kChunk K-blocks at a time and a chunk ahead: a thread copies rows' scales to
            // shared memory, and multiplies them by the weights' once they are there.
            constexpr int kMine = kChunk * C / (32 * F::kEpi);
            float w_next[kMine], w_now[kMine];
            auto fetch = [&](int kb, int half_of) {
#pragma unroll
                for (int j = 0; j < kMine; ++j) {
                    const int i = threadIdx.x + j * 32 * F::kEpi, b = kb + i / C, r = m0 + i % C;
                    const bool in = b < kb1 && r < a.m;
                    cp_async4(ptx::smem_addr(scales + half_of * kChunk * C + i),
                              a.sa + (in ? (int64_t)b * a.sa_stride + r : 0), in);
                    w_next[j] = b < kb1 ? sw[b] : 0.0f;
                }
                cp_async_commit();
            };
            fetch(kb0, 0);
            int turn = 0;
            for (int kc = kb0; kc < kb1; kc += kChunk, turn ^= 1) {  // to the end even after a failed wait: the warps meet at barriers
                ptx::named_sync(1, 32 * F::kEpi);  // the other half's readers are done with it
#pragma unroll
                for (int j = 0; j < kMine; ++j) w_now[j] = w_next[j];
                fetch(kc + kChunk, turn ^ 1);
                cp_async_wait<1>();
#pragma unroll
                for (int j = 0; j < kMine; ++j) scales[turn * kChunk * C + threadIdx.x + j * 32 * F::kEpi] *= w_now[j];
                ptx::named_sync(1, 32 * F::kEpi);
                uint32_t sp = ptx::smem_addr(scales + turn * kChunk * C + col0);
                const int n = min(kChunk, kb1 - kc);
                for (int i = 0; i < n; ++i, sp += 4 * C) {
                    if (ok && !__all_sync(kFull, ptx::mbar_wait_sleep(acc_full + buf, bph, abortp))) {
                        if (lane == 0) fail(4u);
                        ok = false;
                    }
                    if (!ok) continue;
                    ptx::tc_fence_after();
                    uint32_t d[kPer];
                    if constexpr (kPer == 32)
                        tmem_ld32(taddr + buf * C, d);
                    else
                        ptx::tmem_ld16(taddr + buf * C, d);
                    float4 s4[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) s4[e] = ptx::lds_f4(sp + 16 * e);
                    ptx::tmem_ld_wait();
                    ptx::tc_fence_before();
                    arrive_one(lane == 0, ptx::smem_addr(acc_empty + buf));
#pragma unroll
                    for (int e = 0; e < kPer / 4; ++e) {
                        const float4 x = e < 4 ? s4[e & 3] : ptx::lds_f4(sp + 16 * e);
                        acc[2 * e] = ptx::fma2(ptx::f2(__uint_as_float(d[4 * e]), __uint_as_float(d[4 * e + 1])),
                                               ptx::f2(x.x, x.y), acc[2 * e]);
                        acc[2 * e + 1] = ptx::fma2(ptx::f2(__uint_as_float(d[4 * e + 2]), __uint_as_float(d[4 * e + 3])),
                                                   ptx::f2(x.z, x.w), acc[2 * e + 1]);
                    }
                    if (++buf == kBufs) {
                        buf = 0;
                        bph ^= 1;
                    }
                }
            }
            cp_async_wait<0>();
            const int cols = min(kPer, a.m - m0 - col0);
            if (T.splits == 1) {
                if (ok && lrow < a.n) {
                    if (a.type == MOE_F32)
                        store_columns<float>(a, m0 + col0, lrow, cols, acc);
                    else if (a.type == MOE_BF16)
                        store_columns<__nv_bfloat16>(a, m0 + col0, lrow, cols, acc);
                    else
                        store_columns<__half>(a, m0 + col0, lrow, cols, acc);
                }
                ptx::named_sync(1, 32 * F::kEpi);  // this tile's scales are read before the next tile's come
            } else if (ok) {
                // the ring is done with: the last accumulator's MMAs have read it
                float* part = reinterpret_cast<float*>(ring) + col0 * kLanes + 32 * q + lane;
#pragma unroll
                for (int c = 0; c < kPer / 2; ++c) {
                    if (2 * c >= cols) break;
                    const float2 v = ptx::f2(acc[c]);
                    part[(2 * c) * kLanes] = v.x;
                    part[(2 * c + 1) * kLanes] = v.y;
                }
            }
        }
    }
    if (T.splits > 1) {  // one tile a cluster
        __syncwarp();
        cluster_sync();
        int lt, ct;
        place(first, lt, ct);
        if (warp < F::kEpi && !*abortp) {
            // a warp a column, a lane four weights; the loads of two columns before the first sum, as a peer's memory is far
            const int n = lt * kLanes + 4 * lane, cols = min(C, a.m - ct * C);
            const uint32_t at = ptx::smem_addr(ring) + 16 * lane;
            for (int j = warp; rank + T.splits * j < cols; j += 2 * F::kEpi) {
                float4 v[2][8];
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    const int c = rank + T.splits * (j + F::kEpi * d);
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        v[d][r] = r < T.splits && c < cols ? ld_peer4(at + c * (kLanes * 4), r) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    const int c = rank + T.splits * (j + F::kEpi * d);
                    if (c >= cols) break;
                    float4 x = v[d][0];
#pragma unroll
                    for (int r = 1; r < 8; ++r) x.x += v[d][r].x, x.y += v[d][r].y, x.z += v[d][r].z, x.w += v[d][r].w;
                    store4(a, (int64_t)(ct * C + c) * a.out_stride + n, x, a.n - n);
                }
            }
        }
        __syncwarp();
        cluster_sync();  // a CTA's part stays until its peers have read it
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == F::kEpi) ptx::tmem_dealloc(tmem, F::kTmem);
}

// ---- rows form ------------------------------------------------------------------
//
// Two CTAs of a cluster share a tile of 256 rows by 256 weights (cta_group::2): each brings its 128 rows and half of
// the weights, 32 KB a K-block, and holds the sums of its rows. An SM then moves two thirds of the bytes into shared
// memory that a tile of 128 x 256 of its own would take, and one thread issues for two SMs. Tensor memory holds two
// K-blocks' sums. Their buffers go back and forth by halves of 128 weights, which the MMAs take one after the other: from
// the end of a half until its buffer is needed again there are three halves, 768 cycles of tensor work, for the way to the
// epilogue, its loads (eight warps a half, 64 columns each) and the way back.
//
// 8,192 rows of 8,192 by 8,192 weights: 367 us, 3.0 PFLOP/s, 1.57 times the bf16 rate that this GPU's library reaches (380 to
// 400 us when warm, 428 to 434 in a row of calls of a second or more, where the power cap brings the clock to about 1.7 GHz; all-zero
// codes, which draw less, take 350 us at any length). 4,096 rows of 2,816 by 6,144: 69 us, 2.1 PFLOP/s, a last wave of tiles a twentieth full.
// A K-block of 256 x 256 takes 800 cycles, where its products take 512: the epilogue's 64 columns a warp cost two loads, 32
// two-wide multiply-adds (128 a scheduler, two cycles each) and about 60 other instructions, and a buffer's way round is
// longer than three halves. Eight epilogue warps of 128 columns, sixteen of 32 a half, single buffers of 256 and scalar
// multiply-adds took 818 to 1,160 cycles; without the multiply-adds a K-block takes 660. Powers of two as scales could be
// left to the tensor cores' own block scaling; fp32 scales cannot.

struct Pair {
    static constexpr int C = 256, kCtaRows = 128, kEpi = 16, kScaleWarps = 2;
    static constexpr int kWarpLoad = kEpi, kWarpMma = kEpi + 1, kWarpScale = kEpi + 2;
    static constexpr int kThreads = 32 * (kEpi + 4);
    static constexpr int kStageBytes = 2 * kLaneBytes;
    static constexpr int kStages = 5, kSlots = 4;  // a slot: the sums of a K-block and half of the weights
    static constexpr int kScaleBytes = kSlots * kCtaRows * 4;
    static constexpr int kOutBytes = kEpi * 2048;  // a warp's 32 rows x 16 sums, on their way to memory
    static constexpr int kSmem = 1024 + kStages * kStageBytes + kScaleBytes + kOutBytes + 256;
    // 640 threads x 96 registers at launch = 512 x 112 + 128 x 32
    static constexpr int kRegsEpi = 112, kRegsOther = 32;
    static constexpr int kPartStride = C + 4;  // floats of a row of partial sums: rows begin on different banks
    static_assert(kSmem <= 232448, "shared memory");
    static_assert(kCtaRows * kPartStride * 4 <= kStages * kStageBytes, "partial sums of a split lie in the ring");
};

__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_addr(p)), "r"(rank));
    return at;
}
// One lane's arrival at a barrier of the cluster and at one of this CTA.
// (No release at cluster scope: it would wait for all memory operations of the thread, and what is handed over here is
// tensor memory, which tcgen05's fences order.)
__device__ __forceinline__ void arrive_both(bool one, uint32_t cluster_addr, uint32_t own_addr) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t"
        "@p mbarrier.arrive.shared::cluster.b64 _, [%1];\n\t"
        "@p mbarrier.arrive.shared::cta.b64 _, [%2];\n\t}" ::"r"((uint32_t)one),
        "r"(cluster_addr), "r"(own_addr)
        : "memory");
}
// A box into this CTA's shared memory, its bytes counted at a barrier of the pair's first CTA.
__device__ __forceinline__ void tma_load_pair(void* dst, const void* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(ptx::smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void mma_f8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives at the barrier of this offset in both CTAs of the pair (a mask of ranks) when every MMA issued before is done.
__device__ __forceinline__ void commit_pair(uint64_t* bar, uint16_t pair) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            ptx::smem_addr(bar)),
        "h"(pair)
        : "memory");
}

// This CTA's share of the columns of its rows, summed over the S pairs of its cluster in their order.
template <int S>
__device__ __forceinline__ void join_pairs(const MatmulArgs& a, uint32_t sums, uint32_t rank, int share, int m0, int n0) {
    constexpr int kVecs = Pair::C / S / 4, kRowsAtOnce = 32 * Pair::kEpi / kVecs, kDeep = 8 / S;
    const int c = share * (Pair::C / S) + 4 * ((int)threadIdx.x % kVecs), n = n0 + c;
    const int rows = min(Pair::kCtaRows, a.m - m0);
    for (int r0 = (int)threadIdx.x / kVecs; r0 < rows; r0 += kRowsAtOnce * kDeep) {
        float4 v[kDeep][S];  // the loads of several rows before the first sum, as a peer's memory is far
#pragma unroll
        for (int d = 0; d < kDeep; ++d)
#pragma unroll
            for (int p = 0; p < S; ++p)
                v[d][p] = ld_peer4(sums + 4 * (min(r0 + d * kRowsAtOnce, Pair::kCtaRows - 1) * Pair::kPartStride + c), 2 * p + rank);
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
            const int r = r0 + d * kRowsAtOnce;
            if (r >= rows) break;
            float4 x = v[d][0];
#pragma unroll
            for (int p = 1; p < S; ++p) x.x += v[d][p].x, x.y += v[d][p].y, x.z += v[d][p].z, x.w += v[d][p].w;
            store4(a, (int64_t)(m0 + r) * a.out_stride + n, x, a.n - n);
        }
    }
}

// kSplit: clusters of 2 * T.splits CTAs share a tile's K-blocks, and have one tile each.
template <bool kSplit>
__global__ void __launch_bounds__(Pair::kThreads, 1)
    f8_rows_kernel(const __grid_constant__ MatmulArgs a, const __grid_constant__ Tiles T,
                   const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w) {
    using F = Pair;
    constexpr int kStages = F::kStages, kSlots = F::kSlots, C = F::C;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* ring =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    float* scales = reinterpret_cast<float*>(ring + kStages * F::kStageBytes);  // [kSlots][128]
    float* outs = reinterpret_cast<float*>(ring + kStages * F::kStageBytes + F::kScaleBytes);  // [kEpi][32][16]
    uint64_t* full =
        reinterpret_cast<uint64_t*>(ring + kStages * F::kStageBytes + F::kScaleBytes + F::kOutBytes);  // first CTA's: both loaded
    uint64_t* empty = full + kStages;
    uint64_t* acc_full = empty + kStages;        // sums and scales are there
    uint64_t* acc_empty = acc_full + kSlots;     // first CTA's: both have read their sums
    uint64_t* scale_empty = acc_empty + kSlots;  // this CTA has
    uint64_t* drain = scale_empty + kSlots;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    __shared__ int abort_flag;

    const int warp = __shfl_sync(kFull, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    // the cluster's pairs take a part of the K-blocks each
    const uint32_t crank = cluster_rank(), rank = crank & 1, lead = kSplit ? crank & ~1u : 0;
    const uint16_t both = (uint16_t)(3u << lead);
    const int splits = kSplit ? T.splits : 1, share = kSplit ? (int)(crank >> 1) : 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(full + i, 1);
            ptx::mbar_init(empty + i, 1);
        }
        for (int i = 0; i < kSlots; ++i) {
            ptx::mbar_init(acc_full + i, 2);
            ptx::mbar_init(acc_empty + i, F::kEpi);  // half of either CTA's warps
            ptx::mbar_init(scale_empty + i, F::kEpi / 2);
        }
        ptx::mbar_init(drain, 1);
        abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&map_a);
        ptx::prefetch_tensormap(&map_w);
    }
    if (warp == F::kWarpMma) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(ptx::smem_addr(tmem_slot)),
                     "r"(kSlots * C / 2)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    ptx::tc_fence_before();
    __syncthreads();
    cluster_sync();  // barriers are there before the other CTA uses them
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    volatile int* abortp = &abort_flag;
    auto fail = [&](unsigned bit) {
        if (!*abortp) *(volatile unsigned*)a.err = bit;
        abort_flag = 1;
    };
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();

    const int first = (int)blockIdx.x / (2 * splits), step = (int)gridDim.x / (2 * splits);
    const int kb0 = (int)((int64_t)T.kblocks * share / splits);
    const int kblocks = (int)((int64_t)T.kblocks * (share + 1) / splits) - kb0;
    // neighbouring tiles go along the rows, 8 deep, so that tiles of one time share both operands in L2
    auto place = [&](int t, int& lt, int& ct) {
        const int group = 8 * T.cols, g = t / group, deep = min(8, T.lanes - 8 * g), r = t - g * group;
        ct = r / deep;
        lt = 8 * g + (r - ct * deep);
    };

    if (warp >= F::kEpi) {
        fewer_registers<F::kRegsOther>();
        if (warp == F::kWarpLoad) {
            // ---------------- loads ----------------
            const bool leader = elect_one();
            int st = 0;
            uint32_t ph = 0;
            bool ok = true;
            const uint32_t full0 = peer_addr(full, lead);
            for (int t = first; t < T.total && ok; t += step) {
                int lt, ct;
                place(t, lt, ct);
                const int ya = lt * 256 + (int)rank * 128, yw = ct * C + (int)rank * 64;
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!__all_sync(kFull, ptx::mbar_wait_sleep(empty + st, ph ^ 1, abortp))) {
                        if (leader) fail(1u);
                        ok = false;
                        break;
                    }
                    if (leader) {
                        unsigned char* p = ring + st * F::kStageBytes;
                        if (rank == 0) ptx::mbar_arrive_expect_tx(full + st, 2 * F::kStageBytes);
                        tma_load_pair(p, &map_a, (kb0 + kb) * 128, ya, full0 + 8 * st);
                        tma_load_pair(p + kLaneBytes, &map_w, (kb0 + kb) * 128, yw, full0 + 8 * st);
                        tma_load_pair(p + kLaneBytes + kLaneBytes / 2, &map_w, (kb0 + kb) * 128, yw + 128, full0 + 8 * st);
                    }
                    __syncwarp();
                    if (++st == kStages) {
                        st = 0;
                        ph ^= 1;
                    }
                }
            }
        } else if (warp == F::kWarpMma && rank == 0) {
            // ---------------- MMA issue ----------------
            // the whole warp goes round, so that descriptors stay in uniform registers, and one lane issues
            const bool leader = elect_one();
            const uint32_t idesc = f8_idesc(256, C / 2);
            const uint64_t d0 = sw128_desc(ptx::smem_addr(ring));
            int st = 0, slot = 0;
            uint32_t ph = 0, bph = 0;
            bool ok = true;
            for (int t = first; t < T.total && ok; t += step) {
                for (int kb = 0; kb < kblocks; ++kb) {
                    const uint64_t ad = d0 + (uint64_t)((st * F::kStageBytes) >> 4), bd = ad + (kLaneBytes >> 4);
                    ok = __all_sync(kFull, ptx::mbar_wait_sleep(full + st, ph, abortp));
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        ok = ok && __all_sync(kFull, ptx::mbar_wait_sleep(acc_empty + slot, bph ^ 1, abortp));
                        if (!ok) break;
                        ptx::tc_fence_after();
                        if (leader) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)  // K = 32 an MMA: 32 bytes on in the swizzled rows
                                mma_f8_pair(tmem + slot * (C / 2), ad + 2 * k, bd + 512 * h + 2 * k, idesc, k > 0);
                            commit_pair(acc_full + slot, both);
                            if (h == 1) commit_pair(empty + st, both);
                        }
                        __syncwarp();
                        if (++slot == kSlots) {
                            slot = 0;
                            bph ^= 1;
                        }
                    }
                    if (!ok) {
                        if (leader) fail(2u);
                        break;
                    }
                    if (++st == kStages) {
                        st = 0;
                        ph ^= 1;
                    }
                }
            }
            if (leader) commit_pair(drain, both);
            __syncwarp();
            ptx::mbar_wait_sleep(drain, 0, nullptr);
        } else if (warp >= F::kWarpScale) {
            // ---------------- scales: rows' times weights' ----------------
            // a warp a half of the weights, a lane four rows, two K-blocks ahead; the weight block's scales 32 K-blocks
            // a register
            const int h = warp - F::kWarpScale;
            int slot = h;
            uint32_t bph = 0;
            bool ok = true;
            for (int t = first; t < T.total && ok; t += step) {
                int lt, ct;
                place(t, lt, ct);
                const int m = lt * 256 + (int)rank * 128 + lane, left = a.m - m, nb = ct * 2 + h;
                const float* sa = a.sa + (int64_t)kb0 * a.sa_stride + (left > 0 ? m : 0);
                const bool nin = nb * kF8Block < a.n;
                const float* sw = a.sw + (nin ? (int64_t)nb * a.sw_stride : 0) + kb0;
                float q[2][4], w = 0.0f;
                auto fetch = [&](float (&v)[4], int kb) {
                    const float* p = sa + (int64_t)kb * a.sa_stride;
#pragma unroll
                    for (int r = 0; r < 4; ++r) v[r] = kb < kblocks && 32 * r < left ? p[32 * r] : 0.0f;
                };
#pragma unroll
                for (int i = 0; i < 2; ++i) fetch(q[i], i);
                for (int k2 = 0; k2 < kblocks && ok; k2 += 2) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int kb = k2 + i;
                        if (kb >= kblocks) break;
                        if ((kb & 31) == 0) w = nin && kb + lane < kblocks ? sw[kb + lane] : 0.0f;
                        if (!__all_sync(kFull, ptx::mbar_wait_sleep(scale_empty + slot, bph ^ 1, abortp))) {
                            if (lane == 0) fail(8u);
                            ok = false;
                            break;
                        }
                        const float x = __shfl_sync(kFull, w, kb & 31);
                        float* to = scales + slot * 128 + lane;
#pragma unroll
                        for (int r = 0; r < 4; ++r) to[32 * r] = q[i][r] * x;
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(acc_full + slot);
                        fetch(q[i], kb + 2);
                        slot += 2;
                        if (slot >= kSlots) {
                            slot = h;
                            bph ^= 1;
                        }
                    }
                }
            }
        }
        if constexpr (kSplit) {  // where the epilogue's warps wait for the other pairs' sums
            __syncwarp();
            cluster_sync_apart();
        }
    } else {
        more_registers<F::kRegsEpi>();
        // ---------------- epilogue ----------------
        // TMEM lanes 32 q on; of the slots of half h, columns 64 part on of 128
        const int q = warp & 3, part = (warp >> 2) & 1, h = warp >> 3;
        const uint32_t taddr = tmem + ((uint32_t)(32 * q) << 16) + part * 64;
        const uint32_t free0 = peer_addr(acc_empty, lead), mine0 = ptx::smem_addr(scale_empty), sp = ptx::smem_addr(scales) + 4 * (32 * q + lane);
        int slot = h;
        uint32_t bph = 0;
        bool ok = true;
        for (int t = first; t < T.total && ok; t += step) {
            uint64_t acc[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[i] = 0;
            for (int kb = 0; kb < kblocks; ++kb) {
                if (!__all_sync(kFull, ptx::mbar_wait_sleep(acc_full + slot, bph, abortp))) {
                    if (lane == 0) fail(4u);
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                uint32_t d[32];
                tmem_ld32(taddr + slot * (C / 2), d);
                const float sc = ptx::lds_f32(sp + slot * 512);
                const uint64_t s2 = ptx::f2(sc, sc);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    acc[e] = ptx::fma2(ptx::f2(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1])), s2, acc[e]);
                tmem_ld32(taddr + slot * (C / 2) + 32, d);
                ptx::tmem_ld_wait();
                ptx::tc_fence_before();
                arrive_both(lane == 0, free0 + 8 * slot, mine0 + 8 * slot);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    acc[16 + e] = ptx::fma2(ptx::f2(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1])), s2, acc[16 + e]);
                slot += 2;
                if (slot >= kSlots) {
                    slot = h;
                    bph ^= 1;
                }
            }
            int lt, ct;
            place(t, lt, ct);
            const int m0 = lt * 256 + (int)rank * 128;
            if constexpr (!kSplit) {
                if (ok) store_tile(a, outs + warp * 512, m0 + 32 * q, ct * C + h * 128 + part * 64, acc);
            } else {
                // One tile a cluster: its pairs' sums go through the ring, which is done with once the second half's warps
                // have seen the last K-block's sums.
                ptx::named_sync(1, 32 * F::kEpi);
                if (ok) {
                    float4* to = reinterpret_cast<float4*>(reinterpret_cast<float*>(ring) + (32 * q + lane) * F::kPartStride + h * 128 + part * 64);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 x = ptx::f2(acc[2 * i]), y = ptx::f2(acc[2 * i + 1]);
                        to[i] = make_float4(x.x, x.y, y.x, y.y);
                    }
                }
                cluster_sync_apart();
                if (!*abortp) {
                    if (splits == 2)
                        join_pairs<2>(a, ptx::smem_addr(ring), rank, share, m0, ct * C);
                    else
                        join_pairs<4>(a, ptx::smem_addr(ring), rank, share, m0, ct * C);
                }
            }
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (*abortp) {
        // Where a wait expired, a copy may be on its way that no barrier of this CTA counts: they take microseconds, so
        // a millisecond is given to them.
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    }
    // the commits' arrivals are the other CTA's last writes here
    if (warp == F::kWarpMma && rank == 1) ptx::mbar_wait_sleep(drain, 0, nullptr);
    __syncwarp();
    cluster_sync();  // nothing of the pair's is under way in either CTA
    ptx::tc_fence_after();
    if (warp == F::kWarpMma)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kSlots * C / 2) : "memory");
}

// ---- a few rows ------------------------------------------------------------------
//
// Up to 16 rows are bound by the weights' way from memory, and short calls by latency. So there are no roles and no
// tensor memory: a CTA takes 16 weights, its warps take their K-blocks in turn, and the product is
// mma.sync's (m16n8k32, e4m3, the weights as the 16). The order of K within a block is free as long as both operands
// share it, so a lane takes 16 consecutive bytes of a row, four words of which pairs feed two MMAs. A lane copies
// exactly the weights that it will use itself (cp.async), so its shared memory is its own: nothing to
// synchronise, no bank conflict, and all of a warp's K-blocks, kFewDeep at most, in flight at no cost in registers. (Loads into
// registers, as many in flight, left one CTA on an SM: 8.3 us below.)
// 6,144 weights of 2,816 by one row, 17.3 MB: 4.6 us (floor 2.6); 1,024 of 1,024: 1.5 us, the launch.

constexpr int kFewWarps = 8, kFewDeep = 4, kFewLanes = 16;
constexpr int kFewMaxK = kFewWarps * kFewDeep * kF8Block;
constexpr int kFewSmem = kFewWarps * kFewDeep * 4 * 512;
constexpr int few_ctas(int NT) { return NT == 1 ? 3 : 2; }  // resident on an SM

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(  // in order with the copies that overwrite its operands' places
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

// What a K-block needs besides its weights: NT tiles of eight rows, a lane's 16 bytes of each half, and scales.
template <int NT>
struct FewRows {
    uint4 x[NT][2];
    float s[NT][2], w;
};

template <int NT>
__global__ void __launch_bounds__(32 * kFewWarps, few_ctas(NT)) f8_few_kernel(const __grid_constant__ MatmulArgs a, const int kblocks) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ float part[kFewWarps][8 * NT][kFewLanes + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t n0 = (int64_t)blockIdx.x * kFewLanes;  // the CTA's weights
    const uint32_t own = ptx::smem_addr(smem_raw) + warp * (kFewDeep * 4 * 512) + lane * 16;
    // the weights may be what the kernel before writes, so they are only brought into L2 before the wait
    if (threadIdx.x < kFewLanes && n0 + threadIdx.x < a.n)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a.w + (n0 + threadIdx.x) * a.w_stride), "r"(a.k) : "memory");
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const uint8_t* ap[NT];
    bool ain[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        ain[i] = 8 * i + g < a.m;
        ap[i] = a.a + (ain[i] ? (8 * i + g) * a.a_stride : 0) + 16 * t;
    }
#pragma unroll
    for (int d = 0; d < kFewDeep; ++d) {
        const int kb = warp + kFewWarps * d, k = kb * kF8Block + 16 * t;
        if (kb < kblocks) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t n = n0 + g + 8 * h;
                const uint8_t* p = a.w + (n < a.n ? n * a.w_stride : 0);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const bool in = n < a.n && k + 64 * c < a.k;
                    cp_async16(own + d * 2048 + (2 * h + c) * 512, p + (in ? k + 64 * c : 0), in);
                }
            }
        }
        cp_async_commit();
    }
    auto rows = [&](FewRows<NT>& r, int kb) {
        const bool in = kb < kblocks;
        const int k = kb * kF8Block;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                r.x[i][c] = in && ain[i] && k + 64 * c + 16 * t < a.k ? *reinterpret_cast<const uint4*>(ap[i] + k + 64 * c)
                                                                      : make_uint4(0, 0, 0, 0);
                const int m = 8 * i + 2 * t + c;
                r.s[i][c] = in && m < a.m ? a.sa[(int64_t)kb * a.sa_stride + m] : 0.0f;
            }
        r.w = in ? a.sw[n0 / kF8Block * a.sw_stride + kb] : 0.0f;
    };
    FewRows<NT> next;
    rows(next, warp);
    float acc[NT][4] = {};
#pragma unroll
    for (int d = 0; d < kFewDeep; ++d) {
        const int kb = warp + kFewWarps * d;
        if (kb >= kblocks) break;
        const FewRows<NT> r = next;
        rows(next, kb + kFewWarps);
        cp_async_wait_at_most(kFewDeep - 1 - d);
        uint4 w[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < 2; ++c) w[h][c] = ptx::lds_u4(own + d * 2048 + (2 * h + c) * 512);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            float s[4] = {};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint4 u = w[0][c], v = w[1][c], b = r.x[i][c];
                mma_e4m3(s, u.x, v.x, u.y, v.y, b.x, b.y);
                mma_e4m3(s, u.z, v.z, u.w, v.w, b.z, b.w);
            }
            // lanes hold rows 2t, 2t + 1 of weights g and g + 8
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float sc = r.s[i][c] * r.w;
                acc[i][c] = fmaf(s[c], sc, acc[i][c]);
                acc[i][2 + c] = fmaf(s[2 + c], sc, acc[i][2 + c]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) part[warp][8 * i + 2 * t + (e & 1)][g + 8 * (e >> 1)] = acc[i][e];
    __syncthreads();
    if (threadIdx.x < 8 * NT * kFewLanes) {
        const int r = threadIdx.x / kFewLanes, c = threadIdx.x % kFewLanes;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) v += part[w][r][c];
        if (r < a.m && n0 + c < a.n) store1(a.out, r * a.out_stride + n0 + c, v, a.type);
    }
    cp_async_wait<0>();
}

template <int NT>
cudaError_t launch_few(const MatmulArgs& a, cudaStream_t s) {
    static_assert(8 * NT * kFewLanes <= 32 * kFewWarps, "a thread an output");
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(f8_few_kernel<NT>), kFewSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg =
        launch_config(dim3((unsigned)((a.n + kFewLanes - 1) / kFewLanes)), dim3(32 * kFewWarps), kFewSmem, s, true, &attr);
    return cudaLaunchKernelEx(&cfg, f8_few_kernel<NT>, a, (a.k + kF8Block - 1) / kF8Block);
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

Tiles tiles_of(int lanes, int cols, int lane_tile, int col_tile, int k) {
    Tiles T;
    T.lanes = (lanes + lane_tile - 1) / lane_tile;
    T.cols = (cols + col_tile - 1) / col_tile;
    T.total = T.lanes * T.cols;
    T.kblocks = (k + kF8Block - 1) / kF8Block;
    T.splits = 1;
    return T;
}

// Programmatic dependent launch of clusters of `cluster` CTAs (attr must outlive the launch).
cudaLaunchConfig_t cluster_config(unsigned grid, unsigned threads, size_t smem, cudaStream_t s, unsigned cluster,
                                  cudaLaunchAttribute (&attr)[2]) {
    cudaLaunchConfig_t cfg = launch_config(dim3(grid), dim3(threads), smem, s, true, attr);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cfg;
}

// How many clusters of n (2 .. 8) CTAs of the kernel the runtime counts as resident at once. A cluster lies within a GPC, so large
// ones leave SMs idle: of 2 CTAs 76, of 3 46, of 4 36, of 5 28, of 6 23, of 7 and 8 15. For every form it counts one CTA an SM; the
// weights form's run two where there are more.
template <class F, class K>
int resident_clusters(K* kernel, int n) {
    constexpr int kDevices = 64;
    static std::mutex mu;
    static int held[kDevices][9];  // [device][n]; [device][0]: known
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) return 0;
    std::lock_guard<std::mutex> lock(mu);
    int(&of)[9] = held[dev];
    for (int i = 1; !of[0] && i <= 8; ++i) {
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t cfg = cluster_config(8u * i, F::kThreads, F::kSmem, nullptr, (unsigned)i, attr);
        if (cudaOccupancyMaxActiveClusters(&of[i], kernel, &cfg) != cudaSuccess) {
            cudaGetLastError();
            of[i] = 0;
        }
    }
    of[0] = 1;
    return of[n];
}

// CTAs that share a tile's K-blocks: as many as find an SM each at once, at least two K-blocks each. Only where tiles leave
// more than half of the SMs without one and there are some K-blocks to share, as joining the parts takes about 1 us. us for
// 1, 2, 4, 6 and 8 CTAs, 32 rows: 22 tiles of 32 K-blocks 9.5 7.4 5.5 5.4 6.5; 48 tiles of 22 (where the rule says 2) 8.2 7.7 7.3
// 11.1 (a second wave); 64 tiles of 64 (2) 18.4 15.7 13.9; 128 tiles of 16 9.0 9.2; 22 tiles of 6 3.7 4.2. 77 rows, 44 tiles of 32 (3),
// for 2 to 6: 8.8 8.4 8.7 9.0 8.6.
template <class F>
int splits_of(const Tiles& T, int sms) {
    if (2 * T.total > sms || T.kblocks < 8) return 1;
    int s = std::min(8, T.kblocks / 2);
    while (s > 1 && resident_clusters<F>(f8_matmul_kernel<F>, s) < T.total) --s;
    return s;
}

template <class F>
cudaError_t launch_form(const MatmulArgs& a, int sms, cudaStream_t s) {
    const cudaError_t e0 = ensure_smem_attr(reinterpret_cast<const void*>(f8_matmul_kernel<F>), F::kSmem);
    if (e0 != cudaSuccess) return e0;
    Tiles T = tiles_of(a.n, a.m, kLanes, F::C, a.k);
    T.splits = splits_of<F>(T, sms);
    CUtensorMap mw, ma;
    cudaError_t e = encode_codes(&mw, a.w, a.n, a.k, a.w_stride, kLanes);
    if (e == cudaSuccess) e = encode_codes(&ma, a.a, a.m, a.k, a.a_stride, F::C);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    const unsigned grid = T.splits > 1 ? (unsigned)(T.total * T.splits) : (unsigned)std::min(T.total, sms * F::kCtas);
    const cudaLaunchConfig_t cfg = cluster_config(grid, F::kThreads, F::kSmem, s, (unsigned)T.splits, attr);
    return cudaLaunchKernelEx(&cfg, f8_matmul_kernel<F>, a, T, mw, ma);
}

cudaError_t launch_rows(const MatmulArgs& a, int splits, int sms, cudaStream_t s) {
    Tiles T = tiles_of(a.m, a.n, 2 * Pair::kCtaRows, Pair::C, a.k);
    T.splits = splits;
    CUtensorMap ma, mw;
    cudaError_t e = encode_codes(&ma, a.a, a.m, a.k, a.a_stride, Pair::kCtaRows);
    if (e == cudaSuccess) e = encode_codes(&mw, a.w, a.n, a.k, a.w_stride, Pair::C / 4);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    const unsigned grid = 2u * (unsigned)(splits > 1 ? T.total * splits : std::min(T.total, sms / 2));
    const cudaLaunchConfig_t cfg = cluster_config(grid, Pair::kThreads, Pair::kSmem, s, 2u * (unsigned)splits, attr);
    return splits > 1 ? cudaLaunchKernelEx(&cfg, f8_rows_kernel<true>, a, T, ma, mw)
                      : cudaLaunchKernelEx(&cfg, f8_rows_kernel<false>, a, T, ma, mw);
}

}  // namespace

// us of a call in the weights form of 64 rows and in the rows form, by what they measured: a fixed part (more where K is
// shared and parts are joined), and a time per K-block of a tile (for two tiles on an SM at a time, which share its
// bandwidth, or one), for as many tiles as an SM gets.
namespace {
double weights_form_us(const MatmulArgs& a, int sms) {
    using F = Form<64>;
    const Tiles T = tiles_of(a.n, a.m, kLanes, F::C, a.k);
    const int s = splits_of<F>(T, sms), each = (T.total + sms - 1) / sms;
    if (s > 1) return 5.5 + 0.28 * ((T.kblocks + s - 1) / s);
    return each == 1 ? 3.9 + 0.28 * T.kblocks : 3.5 + 0.41 * T.kblocks * ((each + 1) / 2);
}

// *splits: pairs of CTAs a tile. us for 1, 2 and 4: 1,052 rows of 7,536 by 1,154 weights (25 tiles) 29.0 19.5 29.4; 300 of
// 16,384 by 300 (4 tiles) 50.3 27.4 18.6; 700 of 2,048 by 2,048 (24 tiles) 11.6 10.7 20.9.
double rows_form_us(const MatmulArgs& a, int sms, int* splits) {
    const Tiles T = tiles_of(a.m, a.n, 2 * Pair::kCtaRows, Pair::C, a.k);
    *splits = 1;
    // (a tile's stores: rows of an odd stride, or not on 16-byte boundaries, go out an element at a time)
    const bool wide = !(reinterpret_cast<uintptr_t>(a.out) & 15) && a.out_stride % (a.type == MOE_F32 ? 4 : 8) == 0 && a.n % 64 == 0;
    double best = 3.5 + (0.40 * T.kblocks + (wide ? 1.7 : 4.5)) * ((T.total + sms / 2 - 1) / (sms / 2));
    for (int s = 2; s <= 4 && T.kblocks >= 4 * s; s *= 2) {
        const double us = (s == 2 ? 8.0 : 9.5) + 0.40 * ((T.kblocks + s - 1) / s);
        if (us < best && T.total <= resident_clusters<Pair>(f8_rows_kernel<true>, 2 * s)) best = us, *splits = s;
    }
    return best;
}
}  // namespace

// Measured, us (columns: mma.sync, weights form of 16 rows):
//   1 row, one round of CTAs: 1,024 x 1,024 1.5 3.1; 6,144 x 2,816 4.7 7.0; 7,168 x 4,096 7.1 9.2
//   8 rows, one round: 7,296 x 512 2.3 3.1; 2,816 x 4,096 4.6 5.0; 7,296 x 4,096 7.8 9.3; more: 8,192 x 1,024 4.3 4.7; 8,192 x 4,096
//     10.8 9.6; 14,592 x 1,024 5.2 4.6; 20,000 x 512 5.8 3.7
//   16 rows, one round: 1,024 x 1,024 2.0 3.4; 4,864 x 2,048 4.1 5.5; 2,048 x 4,096 4.1 5.0; 4,864 x 4,096 6.4 8.0, but 2,816 x 4,096
//     5.6 5.2; more: 9,728 x 1,024 5.1 4.9; 8,192 x 2,048 7.0 5.9; 20,000 x 512 8.9 3.7
// and (weights form of 32 / 64 rows, rows form):
//   64 rows: 2,816 x 4,096: 7.4 6.3 16.6; 8,192 x 8,192: 18.8 17.3 27.7; 6,144 x 2,816: 8.4 8.8 13.6
//   128 rows (of 64, rows): 6,144 x 2,816: 9.2 13.9; 512 of them: 21.3 14.9; 192 of 16,384 x 2,048: 16.4 13.7
// mma.sync pays where the CTAs, of 16 weights each, are one round and a warp holds all of its K-blocks.
cudaError_t launch_f8_matmul(const MatmulArgs& a, int sms, cudaStream_t s) {
    const int groups = (a.n + kFewLanes - 1) / kFewLanes;
    if (a.m <= 8 && a.k <= kFewMaxK && groups <= few_ctas(1) * sms) return launch_few<1>(a, s);
    if (a.m <= 16 && a.k <= kFewMaxK && groups <= few_ctas(2) * sms) return launch_few<2>(a, s);
    if (a.m <= 16) return launch_form<Form<16>>(a, sms, s);
    if (a.m <= 32) return launch_form<Form<32>>(a, sms, s);
    if (a.m <= 64) return launch_form<Form<64>>(a, sms, s);
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(f8_matmul_kernel<Form<64>>), Form<64>::kSmem);
    if (e == cudaSuccess) e = ensure_smem_attr(reinterpret_cast<const void*>(f8_rows_kernel<false>), Pair::kSmem);
    if (e == cudaSuccess) e = ensure_smem_attr(reinterpret_cast<const void*>(f8_rows_kernel<true>), Pair::kSmem);
    if (e != cudaSuccess) return e;
    int splits;
    const double rows = rows_form_us(a, sms, &splits);
    return weights_form_us(a, sms) <= rows ? launch_form<Form<64>>(a, sms, s) : launch_rows(a, splits, sms, s);
}

}  // namespace moe
