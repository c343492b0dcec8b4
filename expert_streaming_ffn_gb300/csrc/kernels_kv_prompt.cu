// Attention of many query rows over the 4-bit cache (prompts), on the
// 5th-generation tensor cores.
//
// A CTA holds 256 query rows (two tiles of 128; one tile for head_dim 256),
// rows being (new token, query head) pairs of one kv head, so a key tile is
// dequantised once for all of them. Per key tile of 128 (64 for head_dim 256):
//   eight warps dequantise K, then V, from global memory (the next tile's words
//     already in registers) to fp16 in shared memory, 128-byte swizzled; V is used
//     as it lies, [key][dim], as an operand whose rows run along dim;
//   two warps issue S = Q K^T into tensor memory and, later, O += P V with P
//     from tensor memory, where it takes the place of S;
//   four warps per tile, a row a thread, turn S into P = 2^(c s - m + 7), fp16, in two
//     halves, so that O += P V starts on the first. The bound m moves only when a
//     score passes it by 8 (P <= 2^15), and then O is rescaled in tensor memory.
// With two tiles, one's softmax runs under the other's products; with one tile
// (head_dim 256, whose O takes half of tensor memory) S has two buffers instead.
// Row tiles that would leave SMs idle, all of a short call's or the last wave of a
// long one's, have their keys split over CTAs, and a second kernel joins the fp32
// partial results.
//
// Rounding beyond fp32: K and V values, P and Q (scaled by a power of two per row)
// to fp16 (2^-11 each; fp16 outputs 4.3e-4 to 6e-4 off in all, 2.1e-4 of it their own rounding; keys and values
// past fp16's range are its largest number). A weight 2^21 below the row's largest is below fp16's normal
// range and off by 2^-32 of the largest instead: the 2^7 in P is the range that the bound leaves.
//
// What it measured, 32 query heads on 8 kv heads of 128 but where said:
//   4,096 new tokens behind 12,288 keys: 710 us, 1,355 TFLOP/s, 0.71 of the bf16 rate measured on this
//     GPU for a library product (the first calls after a pause 820 to 850, under the power cap). Its cycle is 1.65 us for 256 rows by 128 keys, the time in which one
//     warp gets 2 x 2 products through, those with P from tensor memory and those from shared memory in
//     turn: the products alone, without softmax or dequantisation, took 733 us at the cut that was then
//     in use, the whole kernel 809.
//   4,096 alone: 130 us, 1,060 TFLOP/s: row tiles see 1 to 32 key tiles, and 512 of them make 3.4 waves
//     on 152 SMs (tensor pipe busy 46 % of the time, 51 % of the cycles issuing).
//   128 behind 16,383: 43 us, 802 TFLOP/s, 16 row tiles, each one's keys split over 9 CTAs.
//   As the first, head_dim 256, 16 heads: 1,070 TFLOP/s; head_dim 64: 877. Of neither is a single unit busy (4,096
//     alone: tensor pipe 36 % and 31 %, half of the cycles issuing). Four prompts to 1,024 tokens, 16 heads of
//     64: 17.7 us, of which the start and the end of a CTA are most.
#include <cuda_bf16.h>

#include <algorithm>

#include "kv_internal.h"
#include "ptx.cuh"
#include "tc_operand.cuh"

namespace moe {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr float kLazy = 8.0f;
constexpr float kNone = -3e38f;
constexpr float kHead = 7.0f;  // log2 of what P is scaled by: P <= 2^(kLazy + kHead)

template <int D>
struct PShape {
    static constexpr int NG = D / 64;
    static constexpr int MT = D <= 128 ? 2 : 1;    // row tiles
    static constexpr int NS = MT == 2 ? 1 : 2;     // S buffers of a row tile
    static constexpr int KT = D <= 128 ? 128 : 64; // keys of a tile
    static constexpr int kRows = 128 * MT;
    static constexpr int kRec = kv_record_bytes(D);
    // Warps 0 and 1 issue (their warpgroup's other two idle), the next eight dequantise, the rest are the
    // softmax's. The issuing warps come first as the scheduler prefers older warps: as the CTA's last,
    // one warp took 110 ns to issue a product of 38 ns.
    static constexpr int kWarpMma = 0, kWarpDq = 4, kDqWarps = 8, kWarpSoft = kWarpDq + kDqWarps, kSoftWarps = 4 * MT;
    static constexpr int kDqThreads = 32 * kDqWarps;
    static constexpr int kThreads = 32 * (kWarpSoft + kSoftWarps);
    // The warpgroups share the registers out anew: 32 + 2 * 56 + 2 * 168 = 5 * 96, or 56 + 2 * 112 + 184 < 4 * 128
    static constexpr int kRegMma = MT == 2 ? 32 : 56, kRegDq = MT == 2 ? 56 : 112, kRegSoft = MT == 2 ? 168 : 184;
    static constexpr int kQBytes = 128 * D * 2;  // one row tile
    static constexpr int kTile = KT * D * 2;     // K or V
    static constexpr int kStages = 2;
    static constexpr int kColO = MT * NS * KT;   // tensor memory: S buffers, then O
    static constexpr int kSmem = MT * kQBytes + 2 * kStages * kTile + 1024;
    static constexpr int kSlot = kRows * (D + 2);  // floats of a partial result: o[row][D], then m and l
};

struct Bars {
    uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2][2], s_free[2], drain[2];
    uint64_t o_full;     // one row tile: after each product with V but the last
    uint64_t o_done[2];  // after a row tile's last one
    uint32_t tmem;
    int abort;
    int nan_lo, nan_hi;   // first and last key with a value group that is not finite
    uint4 hide[8];        // of tiles j mod 8: keys (bits) whose page is outside the cache
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <class T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <class T>
__device__ __forceinline__ uint32_t pack2(float x, float y);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float x, float y) {
    return pack_h2(x, y);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float x, float y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// A pair of fp16 values, infinities as +-65,504; NaN stays.
__device__ __forceinline__ uint32_t finite2(uint32_t x) {
    return as_u32(__hmax2_nan(__hmin2_nan(as_h2(x), as_h2(0x7BFF7BFFu)), as_h2(0xFBFFFBFFu)));
}

// Whether scale and bias are finite: an exponent of all ones carries into bit 15 or 31.
__device__ __forceinline__ bool finite_affine(uint32_t af) { return !(((af & 0x7C007C00u) + 0x04000400u) & 0x80008000u); }

#define R8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])
#define W8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])

// 32 lanes x 32 columns of tensor memory, thread i lane (base + i)
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : W8(v, 0), W8(v, 8), W8(v, 16), W8(v, 24)
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::R8(v, 0),
        R8(v, 8), R8(v, 16), R8(v, 24), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15};" ::R8(v, 0),
        R8(v, 8), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];" : W8(v, 0) : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::R8(v, 0), "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 1 in one lane of a converged warp, always the same, 0 in the others. The whole warp goes
// through the issuing loops and this lane issues: the products' operands are then worked out in uniform
// registers. (One lane in a branch of its own, chosen by its number, took 1.62 ms where this takes 1.03.)
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one;
}

// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Descriptor of an operand [k][n] whose n runs along the 128-byte rows: chunks of
// 64 n lie n_stride bytes apart, groups of eight k 1024.
__device__ __forceinline__ uint64_t sw128_desc_n(uint32_t saddr, uint32_t n_stride) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(n_stride >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

using ptx::add2;
using ptx::f2;
using ptx::fma2;

template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// What a CTA works on.
struct Work {
    int first, n, len, b;  // the sequence: first q row, new tokens, keys, index
    int h, row0;           // kv head, first of its rows
    int k0, tiles;         // first key, and key tiles of this split
    bool any;              // there is such a piece of work
    bool whole;            // not split
};

// Row tile `item` (over all sequences and kv heads): its sequence, kv head and rows.
template <int D>
__device__ __forceinline__ Work find_rows(const KvAttend& a, unsigned item, int lane) {
    using S = PShape<D>;
    Work w{};
    w.h = (int)(item % (unsigned)a.c.H);
    int want = (int)(item / (unsigned)a.c.H);
    for (int base = 0; base < a.B; base += 32) {
        const int b = base + lane;
        int first = 0, n = 0, cnt = 0;
        if (b < a.B) {
            if (a.q_start) {
                first = min(max(a.q_start[b], 0), a.n_q);  // within q whatever q_start holds
                n = min(a.q_start[b + 1], a.n_q) - first;
            } else {
                first = b * a.T, n = a.T;
            }
            if (n > 0) cnt = (int)(((int64_t)n * a.G + S::kRows - 1) / S::kRows);
        }
        int inc = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned who = __ballot_sync(kFull, want >= inc - cnt && want < inc);
        if (who) {
            const int src = __ffs(who) - 1;
            w.b = base + src;
            w.first = __shfl_sync(kFull, first, src);
            w.n = __shfl_sync(kFull, n, src);
            // the last rows first: they see the most keys
            w.row0 = __shfl_sync(kFull, inc - 1 - want, src) * S::kRows;
            w.any = true;
            break;
        }
        want -= __shfl_sync(kFull, inc, 31);
    }
    return w;
}

template <int D>
__device__ __forceinline__ Work find_work(const KvAttend& a, int lane) {
    using S = PShape<D>;
    // the first a.full blocks take a row tile each, the others a split of one, a tile's side by side
    const bool whole = blockIdx.x < (unsigned)a.full;
    const unsigned y = whole ? 0 : blockIdx.x - (unsigned)a.full, split = y % (unsigned)a.splits;
    const int splits = whole ? 1 : a.splits;
    Work w = find_rows<D>(a, whole ? blockIdx.x : (unsigned)a.full + y / (unsigned)a.splits, lane);
    w.whole = splits == 1;
    if (!w.any) return w;
    w.len = max(0, min(*(a.kv_len + w.b), a.max_pages << a.c.page_shift));
    const int rows = min(S::kRows, w.n * a.G - w.row0);
    const int p0 = w.len - w.n + (int)a.by_g.div(w.row0), p1 = w.len - w.n + (int)a.by_g.div(w.row0 + rows - 1);
    const int lo = a.window && p0 >= a.window ? p0 - a.window + 1 : 0;
    const int hi = a.causal ? min(w.len, p1 + 1) : w.len;
    w.k0 = lo & ~15;
    const int tiles = hi > w.k0 ? (hi - w.k0 + S::KT - 1) / S::KT : 0;
    const int t0 = (int)((int64_t)tiles * split / splits), t1 = (int)((int64_t)tiles * (split + 1) / splits);
    w.k0 += t0 * S::KT;
    w.tiles = t1 - t0;
    return w;
}

template <int D, class T>
__global__ void __launch_bounds__(PShape<D>::kThreads, 1) kv_prompt_kernel(const __grid_constant__ KvAttend a) {
    using S = PShape<D>;
    constexpr int NG = S::NG, MT = S::MT, NS = S::NS, KT = S::KT, kRec = S::kRec;
    // operand tiles lie on 1 KB; at a place the compiler knows, so that their descriptors are constants
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char* const sq = smem;                              // [MT][NG chunks of 64 dims][128 rows][128 bytes]
    unsigned char* const sk = sq + MT * S::kQBytes;              // [stages][NG][KT][128 bytes]
    unsigned char* const sv = sk + S::kStages * S::kTile;
    Bars& B = *reinterpret_cast<Bars*>(sv + S::kStages * S::kTile);
    static_assert(sizeof(Bars) <= 1024);
    // the warp's index from lane 0, so that the compiler knows it to be the same in all lanes
    const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;

    if (tid == 0) {
        ptx::mbar_init(&B.q_full, 32 * S::kSoftWarps);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&B.k_full[i], S::kDqThreads);
            ptx::mbar_init(&B.v_full[i], S::kDqThreads);
            ptx::mbar_init(&B.k_empty[i], 1);
            ptx::mbar_init(&B.v_empty[i], 1);
            ptx::mbar_init(&B.s_free[i], 1);
            ptx::mbar_init(&B.drain[i], 1);
            ptx::mbar_init(&B.s_full[i], 1);
            for (int h = 0; h < 2; ++h) ptx::mbar_init(&B.p_full[i][h], 128);
            ptx::mbar_init(&B.o_done[i], 1);
        }
        ptx::mbar_init(&B.o_full, 1);
        B.abort = 0;
        for (int i = 0; i < 8; ++i) B.hide[i] = make_uint4(0, 0, 0, 0);
        B.nan_lo = 0x7FFFFFFF;
        B.nan_hi = -1;
    }
    ptx::fence_mbar_init();
    if (warp == S::kWarpMma) {
        ptx::tmem_alloc(&B.tmem, 512);
        ptx::tmem_relinquish();
    }
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const Work w = find_work<D>(a, lane);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    constexpr uint32_t tmem = 0;  // all 512 columns were allocated: they start at 0, checked below
    volatile int* const abortp = &B.abort;
    auto give_up = [&](unsigned code) {
        if (!*abortp) *(volatile unsigned*)a.err = code;
        *abortp = 1;
    };

    const bool based = B.tmem == tmem && (ptx::smem_addr(smem) & 1023) == 0;
    if (!based && tid == 0) give_up(1u << 21);
    if (!w.any || !based) {
    } else if (warp >= S::kWarpSoft) {
        more_registers<S::kRegSoft>();
        // ---------------- a row a thread: queries in, softmax, output ----------------
        const int mt = (warp - S::kWarpSoft) >> 2, r = tid & 127;
        const int row = w.row0 + mt * 128 + r;  // of the kv head's rows of this sequence
        const bool in = row < w.n * a.G;
        const int tk = in ? (int)a.by_g.div(row) : 0, hq = w.h * a.G + (in ? row - tk * a.G : 0);
        const int pos = w.len - w.n + tk;
        // rows past the last one see everything: they are not stored, and so cost no masking
        const int hi = !in ? 0x7FFFFFFF : a.causal ? min(w.len, pos + 1) : w.len;
        const int lo = in && a.window && pos >= a.window ? pos - a.window + 1 : 0;
        float c;  // scores in base 2 are c times S, c > 0
        {
            // A warp's 32 rows as they are, whole rows side by side (a row a thread would touch 32 lines a load), to
            // where each row belongs; then each thread scales its own there.
            constexpr int kChunks = D / 8, kRowsAt = 32 / kChunks, kPart = 16 < kChunks ? 16 : kChunks;
            const T* const mine = static_cast<const T*>(a.q) + (int64_t)(w.first + tk) * a.qt + (int64_t)hq * a.qh;
            const uint32_t rows = ptx::smem_addr(sq + mt * S::kQBytes);
            auto place = [&](int r, int i) { return rows + r * 128 + (i >> 3) * (128 * 128) + (((i & 7) ^ (r & 7)) << 4); };
            const unsigned there = __ballot_sync(kFull, in);
#pragma unroll
            for (int h = 0; h < 32; h += kPart * kRowsAt) {
                uint4 q[kPart];
#pragma unroll
                for (int i = 0; i < kPart; ++i) {
                    const int rr = h + i * kRowsAt + lane / kChunks;
                    const T* const row = reinterpret_cast<const T*>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(mine), rr));
                    q[i] = there >> rr & 1 ? *reinterpret_cast<const uint4*>(row + lane % kChunks * 8) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < kPart; ++i)
                    ptx::sts_u4(place((r & 96) + h + i * kRowsAt + lane / kChunks, lane % kChunks), q[i]);
            }
            __syncwarp();
            float top = 0.0f;
#pragma unroll 8
            for (int i = 0; i < kChunks; ++i) {
                const uint4 q = ptx::lds_u4(place(r, i));
                const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = unpack2<T>(u[e]);
                    top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
            }
            int ex = (int)((__float_as_uint(top) >> 23) & 255u) - 127;  // floor(log2 top)
            ex = top == 0.0f || ex == 128 ? 10 : min(max(ex, -100), 110);
            float f = __uint_as_float((uint32_t)(127 + 10 - ex) << 23);
            if (a.scale_log2 <= 0.0f) f = a.scale_log2 < 0.0f ? -f : 0.0f;
            c = a.scale_log2 == 0.0f ? 1.0f : fabsf(a.scale_log2) * __uint_as_float((uint32_t)(127 - 10 + ex) << 23);
#pragma unroll 8
            for (int i = 0; i < kChunks; ++i) {
                const uint4 q = ptx::lds_u4(place(r, i));
                const uint32_t u[4] = {q.x, q.y, q.z, q.w};
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 x = unpack2<T>(u[e]);
                    o[e] = pack_h2(x.x * f, x.y * f);
                }
                ptx::sts_u4(place(r, i), make_uint4(o[0], o[1], o[2], o[3]));
            }
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(&B.q_full);
        }
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t t_o = tmem + lanes + S::kColO + mt * D;
        float m = kNone, thr = kNone, l = 0.0f;  // bound, the S that passes it by kLazy, sum of weights
        bool ok = true;
        for (int j = 0; j < w.tiles; ++j) {
            const int sb = MT == 2 ? mt : j & 1;  // S buffer, and its barriers
            const uint32_t ph = MT == 2 ? j & 1 : (j >> 1) & 1;
            ok = __all_sync(kFull, ptx::mbar_wait_bounded(&B.s_full[sb], ph, abortp));
            if (!ok) {
                if (lane == 0) give_up(1u << 16);
                break;
            }
            ptx::tc_fence_after();
            const uint32_t t_s = tmem + lanes + sb * KT;
            const int key0 = w.k0 + j * KT;
            const uint4 hv = ptx::lds_u4(ptx::smem_addr(&B.hide[j & 7]));
            const uint32_t hide[4] = {hv.x, hv.y, hv.z, hv.w};
            const bool masked = !__all_sync(kFull, key0 >= lo && key0 + KT <= hi && !(hv.x | hv.y | hv.z | hv.w));
            uint32_t s[KT];
#pragma unroll
            for (int q = 0; q < KT / 32; ++q) tmem_ld32(t_s + 32 * q, s + 32 * q);
            ptx::tmem_ld_wait();
            if (masked) {
#pragma unroll
                for (int q = 0; q < KT / 32; ++q) {
                    // bit i: key key0 + 32 q + i is seen
                    const int up = hi - key0 - 32 * q, down = lo - key0 - 32 * q;
                    const uint32_t below = up >= 32 ? ~0u : (1u << max(up, 0)) - 1;
                    const uint32_t from = down >= 32 ? 0u : ~0u << max(down, 0);
                    const uint32_t seen = below & from & ~hide[q];
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (!(seen & (1u << i))) s[32 * q + i] = 0xFF800000u;  // -inf
                }
            }
            float top = kNone;
#pragma unroll
            for (int i = 0; i < KT; i += 2) top = fmaxf(top, fmaxf(__uint_as_float(s[i]), __uint_as_float(s[i + 1])));
            const bool over = top > thr;
            if (__any_sync(kFull, over)) {
                // some row of the warp passes its bound: its sums so far are rescaled
                const float mn = over ? fmaxf(m, top * c) : m;
                const float sc = over && m != kNone ? ex2(m - mn) : 1.0f;
                if (j > 0 && __any_sync(kFull, sc != 1.0f)) {
                    if (NS == 2) {
                        // the last product may still run; the one before it does not, as S could not have been
                        // made, and the next cannot start: so the phase waited for is the current one or the last
                        ok = __all_sync(kFull, ptx::mbar_wait_bounded(&B.o_full, (j - 1) & 1, abortp));
                        if (!ok) {
                            if (lane == 0) give_up(1u << 20);
                            break;
                        }
                        ptx::tc_fence_after();
                    }
#pragma unroll 1
                    for (int q = 0; q < D / 8; ++q) {  // few at a time: the scores are in registers
                        uint32_t o[8];
                        tmem_ld8(t_o + 8 * q, o);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * sc);
                        tmem_st8(t_o + 8 * q, o);
                    }
                }
                l *= sc;
                m = mn;
                if (over) thr = fmaxf((mn + kLazy) / c, top);
            }
            uint64_t sum = f2(0.0f, 0.0f);
            const uint64_t cc = f2(c, c), mm = f2(kHead - m, kHead - m);
#pragma unroll
            for (int q = 0; q < 2; ++q) {  // in halves, so that the product with V starts on the first
#pragma unroll
                for (int i = q * (KT / 2); i < (q + 1) * (KT / 2); i += 2) {
                    const float2 z = f2(fma2(f2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), cc, mm));
                    const float x = ex2(z.x), y = ex2(z.y);
                    sum = add2(sum, f2(x, y));
                    s[i / 2] = pack_h2(x, y);
                }
                if constexpr (KT == 128)
                    tmem_st32(t_s + 32 * q, s + 32 * q);
                else
                    tmem_st16(t_s + 16 * q, s + 16 * q);
                tmem_st_wait();
                ptx::tc_fence_before();
                ptx::mbar_arrive(&B.p_full[sb][q]);
            }
            const float2 x = f2(sum);
            l += x.x + x.y;
        }
        // ---- output ----
        if (ok && w.tiles > 0) {
            ok = __all_sync(kFull, ptx::mbar_wait_bounded(&B.o_done[mt], 0, abortp));
            if (!ok && lane == 0) give_up(1u << 17);
            ptx::tc_fence_after();
        }
        // NaN values are kept out of the products, where a weight of zero would spread them: the rows that see one
        // are NaN in its group. Which do is worked out from the records once more, 32 keys at a time (a microsecond or two),
        // between the first and the last such key that the CTA met.
        unsigned nan = 0;
        if (const int last = *(volatile int*)&B.nan_hi; last >= 0) {
            const int from = max((int)__reduce_min_sync(kFull, (unsigned)(in ? lo : 0x7FFFFFFF)), *(volatile int*)&B.nan_lo);
            const int to = min((int)__reduce_max_sync(kFull, (unsigned)(in ? max(hi, 0) : 0)), last + 1);
            const int32_t* const table = a.table + (int64_t)w.b * a.table_stride;
            for (int base = from; base < to; base += 32) {
                const int key = base + lane;
                const int page = key < to ? table[key >> a.c.page_shift] : -1;
                unsigned mine = 0;
                if ((unsigned)page < (unsigned)a.c.n_pages) {
                    const uint8_t* rec = a.c.pages + (((size_t)page * a.c.H + w.h) * (a.c.P >> 4) + ((key & (a.c.P - 1)) >> 4)) * kRec;
                    const uint32_t* ap = reinterpret_cast<const uint32_t*>(rec + kv_v_affine(D)) + (key & 15) * NG;
#pragma unroll
                    for (int g = 0; g < NG; ++g) mine |= (unsigned)!finite_affine(ap[g]) << g;
                }
                const int up = hi - base, down = lo - base;
                const uint32_t seen = (up >= 32 ? ~0u : (1u << max(up, 0)) - 1) & (down >= 32 ? 0u : ~0u << max(down, 0));
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    if (__ballot_sync(kFull, mine >> g & 1) & seen) nan |= 1u << g;
            }
        }
        float* const slot = a.part + (size_t)(blockIdx.x - (unsigned)a.full) * S::kSlot;
        if (ok) {
            // A row a thread would store 16 bytes of 32 lines at a time. The rows go through shared memory,
            // where this row tile's queries were: a warp's 32 rows of 2 D bytes, chunks of 16 swizzled, whole
            // rows of output or half rows of fp32 at a time.
            const bool whole = w.whole;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            constexpr int kChunks = D / 8, kRowsAt = 32 / kChunks < 1 ? 1 : 32 / kChunks;  // of a row; rows at a time
            const uint32_t stage = ptx::smem_addr(sq + mt * S::kQBytes) + (warp & 3) * (32 * D * 2);
            const unsigned stored = __ballot_sync(kFull, in);
            auto put = [&](int chunk, uint4 v) { ptx::sts_u4(stage + lane * (D * 2) + ((chunk ^ (lane & 7)) << 4), v); };
            T* const out = static_cast<T*>(a.out) + (int64_t)(w.first + tk) * a.ot + (int64_t)hq * a.oh;
            auto pass_on = [&](int half) {
                __syncwarp();
#pragma unroll 4
                for (int i = 0; i < 32; i += kRowsAt) {
                    const int rr = i + lane / kChunks, chunk = lane % kChunks;
                    const uint4 v = w.tiles > 0 ? ptx::lds_u4(stage + rr * (D * 2) + ((chunk ^ (rr & 7)) << 4)) : make_uint4(0, 0, 0, 0);
                    T* const row_out = reinterpret_cast<T*>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(out), rr));
                    if (!(stored >> rr & 1)) continue;
                    if (whole)
                        *reinterpret_cast<uint4*>(row_out + 8 * chunk) = v;
                    else
                        __stcg(reinterpret_cast<uint4*>(slot + (size_t)(mt * 128 + (warp & 3) * 32 + rr) * D + half * (D / 2)) + chunk, v);
                }
                __syncwarp();
            };
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
                uint32_t o[32];
                if (w.tiles > 0) {
                    tmem_ld32(t_o + 32 * q, o);
                    ptx::tmem_ld_wait();
                }
                const bool bad = nan >> (q / 2) & 1;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (w.tiles == 0 || l == 0.0f)
                        o[i] = 0;
                    else if (bad)
                        o[i] = 0x7FC00000u;
                if (w.tiles > 0 && whole) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t u[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            u[e] = pack2<T>(__uint_as_float(o[8 * i + 2 * e]) * inv, __uint_as_float(o[8 * i + 2 * e + 1]) * inv);
                        put(4 * q + i, make_uint4(u[0], u[1], u[2], u[3]));
                    }
                } else if (w.tiles > 0) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        put(8 * (q % (D / 64)) + i, make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]));
                }
                if (!whole && q % (D / 64) == D / 64 - 1) pass_on(q / (D / 64));
            }
            if (whole) pass_on(0);
            if (in && whole) {
                if (a.lse) a.lse[(int64_t)(w.first + tk) * a.Hq + hq] = l == 0.0f ? -INFINITY : 0.6931471805599453f * (m - kHead + log2f(l));
            } else if (in) {
                __stcg(slot + (size_t)S::kRows * D + mt * 128 + r, m);
                __stcg(slot + (size_t)S::kRows * (D + 1) + mt * 128 + r, l);
            }
        }
    } else if (warp >= S::kWarpDq) {
        fewer_registers<S::kRegDq>();
        // ---------------- dequantisation ----------------
        // A row's code bytes are kChunks pieces of 16; thread: piece t % kChunks of row t / kChunks, and so on
        constexpr int kChunks = D / 32, kPerIt = S::kDqThreads / kChunks, kIts = KT / kPerIt;
        const int t = tid - 32 * S::kWarpDq, piece = t % kChunks, r0 = t / kChunks;
        const int32_t* const table = a.table + (int64_t)w.b * a.table_stride;
        const uint8_t* const head = a.c.pages + (size_t)w.h * (a.c.P >> 4) * kRec;
        const size_t page_bytes = (size_t)a.c.H * (a.c.P >> 4) * kRec;
        // Of each of this thread's rows of a tile: the page id, and the record's offset, -1 where there
        // is none. The ids are asked for a tile before the records.
        int32_t page[kIts];
        int64_t at[kIts];
        uint4 kw[kIts], vw[kIts];
        uint32_t ka[kIts][NG], va[kIts][NG];
        auto ask = [&](int j) {
#pragma unroll
            for (int it = 0; it < kIts; ++it) {
                const int key = w.k0 + j * KT + it * kPerIt + r0;
                page[it] = key < w.len ? table[key >> a.c.page_shift] : -1;
            }
        };
        auto places = [&](int j) {
#pragma unroll
            for (int it = 0; it < kIts; ++it) {
                const int key = w.k0 + j * KT + it * kPerIt + r0;
                at[it] = -1;
                if ((unsigned)page[it] < (unsigned)a.c.n_pages)
                    at[it] = (int64_t)page[it] * page_bytes + (size_t)((key & (a.c.P - 1)) >> 4) * kRec;
                else if (key < w.len)
                    *(volatile unsigned*)a.bad = 1u;
            }
        };
        // side 0: keys, 1: values; rows that are not there read as zeros
        auto fetch = [&](int j, int side, uint4 (&cw)[kIts], uint32_t (&aw)[kIts][NG]) {
#pragma unroll
            for (int it = 0; it < kIts; ++it) {
                const int key = w.k0 + j * KT + it * kPerIt + r0, r = key & 15;
                cw[it] = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int g = 0; g < NG; ++g) aw[it][g] = 0;
                if (at[it] >= 0) {
                    const uint8_t* rec = head + at[it];
                    cw[it] = *(reinterpret_cast<const uint4*>(rec + (side ? kv_v_codes(D) : 0) + r * (D / 2)) + piece);
                    const uint32_t* ap = reinterpret_cast<const uint32_t*>(rec + (side ? kv_v_affine(D) : kv_k_affine(D))) + r * NG;
                    if constexpr (NG == 4) {
                        const uint4 x = *reinterpret_cast<const uint4*>(ap);
                        aw[it][0] = x.x, aw[it][1] = x.y, aw[it][2] = x.z, aw[it][3] = x.w;
                    } else if constexpr (NG == 2) {
                        const uint2 x = *reinterpret_cast<const uint2*>(ap);
                        aw[it][0] = x.x, aw[it][1] = x.y;
                    } else {
                        aw[it][0] = *(ap);
                    }
                }
            }
        };
        // Whether some value of these groups could lie past fp16's range: a bias of 2^15 or more or a scale of 2^11 or
        // more (below both, 15 scales and the bias stay under 65,504), infinities and NaN among them. Adding to the exponents
        // carries into bits 15 and 31.
        auto past = [&](const uint32_t (&aw)[kIts][NG]) {
            __half2 top = as_h2(0);
#pragma unroll
            for (int it = 0; it < kIts; ++it)
#pragma unroll
                for (int g = 0; g < NG; ++g) top = __hmax2_nan(top, __habs2(as_h2(aw[it][g])));
            return (((as_u32(top) & 0x7C007C00u) + 0x08001800u) & 0x80008000u) != 0;
        };
        // keys of tile j that are not there, for the softmax to leave out; and room for tile j + 2's, eight
        // tiles after its last use (the softmax is behind by three at most)
        auto note = [&](int j) {
            if (t == 0) B.hide[(j + 2) & 7] = make_uint4(0, 0, 0, 0);
            bool any = false;
#pragma unroll
            for (int it = 0; it < kIts; ++it) any |= at[it] < 0 && w.k0 + j * KT + it * kPerIt + r0 < w.len;
            if (!__any_sync(kFull, any)) return;
#pragma unroll
            for (int it = 0; it < kIts; ++it) {
                const int r = it * kPerIt + r0;
                if (at[it] < 0 && piece == 0 && w.k0 + j * KT + r < w.len)
                    atomicOr(reinterpret_cast<unsigned*>(&B.hide[j & 7]) + (r >> 5), 1u << (r & 31));
            }
        };
        auto at_word = [&](uint32_t base, int it, int x) {  // word 4 piece + x of row it: elements 8i .. 8i+7 of group g
            const int r = it * kPerIt + r0, g = (4 * piece + x) % NG, i = (4 * piece + x) / NG;
            return base + g * (KT * 128) + r * 128 + ((i ^ (r & 7)) << 4);
        };
        auto affine_at = [](const uint32_t (&a)[NG], int x) { return a[x % NG]; };
        auto put = [&](unsigned char* tile, const uint4 (&cw)[kIts], const uint32_t (&aw)[kIts][NG]) {
            const uint32_t base = ptx::smem_addr(tile);
#pragma unroll
            for (int it = 0; it < kIts; ++it) {
                const uint32_t words[4] = {cw[it].x, cw[it].y, cw[it].z, cw[it].w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t af = affine_at(aw[it], x);
                    const __half2 s2 = __half2half2(__ushort_as_half((unsigned short)(af & 0xFFFFu)));
                    const __half2 b2 = __half2half2(__ushort_as_half((unsigned short)(af >> 16)));
                    ptx::sts_u4(at_word(base, it, x), dequant8(words[x], s2, b2));
                }
            }
        };
        // A second pass over the few tiles that may hold a value past fp16's range. Finite ones (a scale rounded up
        // takes a group's largest to 65,624 at most) become its largest number: an infinity would make NaN of the products
        // with the weights of zero of rows that do not see it. Value groups that are not finite leave no trace in the tile but
        // are noted (see the epilogue).
        auto mend = [&](unsigned char* tile, const uint32_t (&aw)[kIts][NG], bool values, int j) {
            const uint32_t base = ptx::smem_addr(tile);
#pragma unroll
            for (int it = 0; it < kIts; ++it) {
                if (values && piece == 0)
#pragma unroll
                    for (int g = 0; g < NG; ++g)
                        if (!finite_affine(aw[it][g])) {
                            atomicMin(&B.nan_lo, w.k0 + j * KT + it * kPerIt + r0);
                            atomicMax(&B.nan_hi, w.k0 + j * KT + it * kPerIt + r0);
                        }
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t p = at_word(base, it, x);
                    uint4 v = ptx::lds_u4(p);
                    v = make_uint4(finite2(v.x), finite2(v.y), finite2(v.z), finite2(v.w));
                    if (values && !finite_affine(affine_at(aw[it], x))) v = make_uint4(0, 0, 0, 0);
                    ptx::sts_u4(p, v);
                }
            }
        };
        if (w.tiles > 0) {
            ask(0);
            places(0);
            fetch(0, 0, kw, ka);
            fetch(0, 1, vw, va);
            ask(1);
        }
        bool ok = true;
        for (int j = 0; j < w.tiles && ok; ++j) {
            const int st = j & 1;
            const uint32_t ph = ((j >> 1) & 1) ^ 1;
            const bool more = j + 1 < w.tiles;
            ok = __all_sync(kFull, ptx::mbar_wait_bounded(&B.k_empty[st], ph, abortp));
            if (!ok) break;
            note(j);
            put(sk + st * S::kTile, kw, ka);
            if (__any_sync(kFull, past(ka))) mend(sk + st * S::kTile, ka, false, j);
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(&B.k_full[st]);
            if (more) {
                places(j + 1);
                fetch(j + 1, 0, kw, ka);
                ask(j + 2);
            }
            ok = __all_sync(kFull, ptx::mbar_wait_bounded(&B.v_empty[st], ph, abortp));
            if (!ok) break;
            put(sv + st * S::kTile, vw, va);
            if (__any_sync(kFull, past(va))) mend(sv + st * S::kTile, va, true, j);
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(&B.v_full[st]);
            if (more) fetch(j + 1, 1, vw, va);
        }
        if (!ok && lane == 0) give_up(1u << 18);
    } else {
        fewer_registers<S::kRegMma>();
        if (warp < 2) {
            // ---------------- MMA issue ----------------
            // One warp with two row tiles: a warp for each would have products of both kinds (Q K^T from
            // shared memory, P V from tensor memory) alternate, and each change costs some 130 cycles
            // (1.53 ms against 1.08 for 4,096 tokens behind 12,288). With one row tile S in one, O in another.
            const uint32_t one = elect_one();
            const int tiles = __shfl_sync(kFull, w.tiles, 0);
            const uint32_t id_s = f16_idesc(128, KT), id_o = f16_idesc(128, D) | (1u << 16);  // V: n along the rows
            // descriptors: the low words hold the address, in 16-byte units, and never carry
            const uint64_t dq0 = sw128_desc(ptx::smem_addr(sq)), dk0 = sw128_desc(ptx::smem_addr(sk));
            const uint64_t dv0 = sw128_desc_n(ptx::smem_addr(sv), KT * 128);
            auto at = [](uint64_t d, uint32_t bytes) { return (d & ~0xFFFFFFFFull) | ((uint32_t)d + (bytes >> 4)); };
            auto wait = [&](uint64_t* bar, uint32_t ph) { return __all_sync(kFull, ptx::mbar_wait_bounded(bar, ph, abortp)); };
            auto qk = [&](int mt, int sb, int st) {  // S[sb] = Q[mt] K[st]^T
                if (one)
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const int chunk = k >> 2, in = k & 3;
                    ptx::mma_f16_ss(tmem + sb * KT, at(dq0, mt * S::kQBytes + chunk * (128 * 128) + in * 32),
                           at(dk0, st * S::kTile + chunk * (KT * 128) + in * 32), id_s, k > 0);
                }
            };
            // O[mt] += P[sb] V[st], over half the keys as soon as their weights are there
            auto pv = [&](int mt, int sb, int st, int j, uint32_t ph) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (!wait(&B.p_full[sb][half], ph)) return false;
                    ptx::tc_fence_after();  // P was written to tensor memory by other threads
                    if (one)
#pragma unroll
                    for (int k = half * (KT / 32); k < (half + 1) * (KT / 32); ++k)
                        mma_f16_ts(tmem + S::kColO + mt * D, tmem + sb * KT + 8 * k, at(dv0, st * S::kTile + k * 2048), id_o,
                               j > 0 || k > 0);
                }
                return true;
            };
            // Every commit's arrival is waited for by somebody, so none can reach a CTA that has ended.
            bool ok = tiles > 0;
            if (MT == 2 && warp == 0) {
                auto scores = [&](int mt, int j, int st) {  // S[mt] of tile j
                    qk(mt, mt, st);
                    if (one) ptx::mma_commit(&B.s_full[mt]);
                    if (one && mt == 1 && j + 2 < tiles) ptx::mma_commit(&B.k_empty[st]);
                };
                auto step = [&](int j, int st) {  // tile j, st = j & 1
                    const bool more = j + 1 < tiles;
                    if (!wait(&B.v_full[st], (j >> 1) & 1) || (more && !wait(&B.k_full[st ^ 1], ((j + 1) >> 1) & 1)))
                        return false;
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        if (!pv(mt, mt, st, j, j & 1)) return false;
                        if (more)
                            scores(mt, j + 1, st ^ 1);
                        else if (one)
                            ptx::mma_commit(&B.o_done[mt]);
                    }
                    if (one && j + 2 < tiles) ptx::mma_commit(&B.v_empty[st]);
                    return true;
                };
                ok = ok && wait(&B.q_full, 0) && wait(&B.k_full[0], 0);
                if (ok)
                    for (int mt = 0; mt < 2; ++mt) scores(mt, 0, 0);
                for (int j = 0; j < tiles && ok; j += 2) {
                    ok = step(j, 0);
                    if (ok && j + 1 < tiles) ok = step(j + 1, 1);
                }
            } else if (MT == 2) {
            } else if (warp == 0) {
                auto scores = [&](int j, int st) {  // S of tile j into buffer st = j & 1, once tile j - 2's P is used
                    if (j >= 2 && !wait(&B.s_free[st], ((j >> 1) & 1) ^ 1)) return false;
                    if (!wait(&B.k_full[st], (j >> 1) & 1)) return false;
                    qk(0, st, st);
                    if (one) ptx::mma_commit(&B.s_full[st]);
                    if (one && j + 2 < tiles) ptx::mma_commit(&B.k_empty[st]);
                    return true;
                };
                ok = ok && wait(&B.q_full, 0);
                for (int j = 0; j < tiles && ok; j += 2) {
                    ok = scores(j, 0);
                    if (ok && j + 1 < tiles) ok = scores(j + 1, 1);
                }
            } else {
                auto step = [&](int j, int st) {
                    const uint32_t ph = (j >> 1) & 1;
                    if (!wait(&B.v_full[st], ph) || !pv(0, st, st, j, ph)) return false;
                    if (one) ptx::mma_commit(j + 1 < tiles ? &B.o_full : &B.o_done[0]);
                    if (j + 2 < tiles) {
                        if (one) ptx::mma_commit(&B.v_empty[st]);
                        if (one) ptx::mma_commit(&B.s_free[st]);
                    }
                    return true;
                };
                for (int j = 0; j < tiles && ok; j += 2) {
                    ok = step(j, 0);
                    if (ok && j + 1 < tiles) ok = step(j + 1, 1);
                }
            }
            if (!ok && tiles > 0) {
                if (one) give_up(1u << 19);
                if (one) ptx::mma_commit(&B.drain[warp]);  // what was issued finishes before tensor memory is given back
                ptx::mbar_wait_bounded(&B.drain[warp], 0, nullptr);
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == S::kWarpMma) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(B.tmem, 512);
    }
}

// Adds the splits of a row tile's partial results; block (tile and kv head, row
// group of 8): a warp a row.
template <int D, class T>
__global__ void __launch_bounds__(256) kv_prompt_join_kernel(const __grid_constant__ KvAttend a) {
    using S = PShape<D>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const unsigned x = blockIdx.x / (S::kRows / 8), r = blockIdx.x % (S::kRows / 8) * 8 + warp;  // of the split tiles
    const Work w = find_rows<D>(a, (unsigned)a.full + x, lane);
    const int row = w.row0 + (int)r;
    if (!w.any || row >= w.n * a.G) return;
    const int first = w.first, tk = (int)a.by_g.div(row), hq = w.h * a.G + row - tk * a.G;
    const float* p0 = a.part + (size_t)x * a.splits * S::kSlot;
    float M = kNone, L = 0.0f;
    for (int p = lane; p < a.splits; p += 32) M = fmaxf(M, p0[(size_t)p * S::kSlot + (size_t)S::kRows * D + r]);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
    constexpr int E = D / 32;
    float y[E] = {};
#pragma unroll 4
    for (int p = 0; p < a.splits; ++p) {
        const float* s = p0 + (size_t)p * S::kSlot;
        const float wt = ex2(s[(size_t)S::kRows * D + r] - M);
        L = fmaf(wt, s[(size_t)S::kRows * (D + 1) + r], L);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 v = *reinterpret_cast<const float2*>(s + (size_t)r * D + lane * E + e);
            y[e] = fmaf(wt, v.x, y[e]), y[e + 1] = fmaf(wt, v.y, y[e + 1]);
        }
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + (int64_t)(first + tk) * a.ot + (int64_t)hq * a.oh + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = pack2<T>(y[e] * inv, y[e + 1] * inv);
    if (a.lse && lane == 0) a.lse[(int64_t)(first + tk) * a.Hq + hq] = L == 0.0f ? -INFINITY : 0.6931471805599453f * (M - kHead + log2f(L));
}

template <int D, class T>
cudaError_t launch_prompt(const KvAttend& a, int64_t work, cudaStream_t s, int* launched) {
    using S = PShape<D>;
    auto kernel = kv_prompt_kernel<D, T>;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), S::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t split = work - a.full;  // row tiles
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg =
        launch_config(dim3((unsigned)(a.full + split * a.splits)), dim3(S::kThreads), S::kSmem, s, true, &attr);
    e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e != cudaSuccess || a.splits == 1) return e;
    *launched = 2;
    const cudaLaunchConfig_t jcfg = launch_config(dim3((unsigned)(split * (S::kRows / 8))), dim3(256), 0, s, true, &attr);
    return cudaLaunchKernelEx(&jcfg, kv_prompt_join_kernel<D, T>, a);
}

template <int D>
cudaError_t launch_prompt_of(const KvAttend& a, int64_t work, moe_dtype t, cudaStream_t s, int* launched) {
    return t == MOE_BF16 ? launch_prompt<D, __nv_bfloat16>(a, work, s, launched) : launch_prompt<D, __half>(a, work, s, launched);
}

}  // namespace

// Row tiles (at most: the sequences' remainders are known on the device only), and how many of
// them are split how often: those that do not fill the SMs a last time, if they are at most half as many,
// four key tiles to a CTA at least. Where whole waves come first, the last wave's tiles are a
// causal prompt's first rows, and a split has to save more than the second kernel costs: they see 16 key
// tiles or more. 4,096 new tokens, 512 row tiles on 152 SMs, 56 of them in the fourth wave: behind 12,288
// keys 800 us whole, 728 with each split in two; alone, where the 56 see up to 448 keys, 139 and 151.
int64_t kv_prompt_plan(KvAttend& a, int d, int max_q, int max_len, int sms) {
    const int rows = d == 256 ? PShape<256>::kRows : PShape<128>::kRows, kt = d == 256 ? PShape<256>::KT : PShape<128>::KT;
    const int64_t tiles = a.q_start ? ((int64_t)a.n_q * a.G + (int64_t)a.B * (rows - 1)) / rows
                                    : (int64_t)a.B * (((int64_t)a.T * a.G + rows - 1) / rows);
    const int64_t work = tiles * a.c.H, rest = work % sms, full = work - rest;
    int64_t keys = max_len;  // that a tile to be split sees
    if (full && a.causal) keys = std::max<int64_t>(0, (int64_t)max_len - max_q) + (int64_t)max_q * rest / work;
    if (a.window) keys = std::min<int64_t>(keys, (int64_t)a.window + rows / a.G);
    const int64_t key_tiles = (keys + kt - 1) / kt;
    a.splits = 1;
    a.full = (int)work;
    if (rest > 0 && (full == 0 || key_tiles >= 16)) {
        a.splits = (int)std::max<int64_t>(1, std::min<int64_t>(sms / rest, (key_tiles + 3) / 4));
        if (a.splits > 1) a.full = (int)full;
    }
    return work;
}

cudaError_t launch_kv_prompt(const KvAttend& a, int d, moe_dtype t, int64_t work, cudaStream_t s, int* launched) {
    return d == 64    ? launch_prompt_of<64>(a, work, t, s, launched)
           : d == 128 ? launch_prompt_of<128>(a, work, t, s, launched)
                      : launch_prompt_of<256>(a, work, t, s, launched);
}

}  // namespace moe
