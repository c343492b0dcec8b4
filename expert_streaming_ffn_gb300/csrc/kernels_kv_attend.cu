// Attention of few query columns over the 4-bit cache (decode steps): the cache
// is read once, the codes go to the tensor cores as they are.
//
// Columns are (new token, query head of the kv head) pairs, 8 * NT to a tile; a
// segment is (sequence, kv head, column tile), its keys in blocks of 16 (one
// record each). All segments' blocks are laid end to end and cut into equal
// ranges, one per CTA, so ragged batches and single long sequences alike keep
// every SM reading; the fp32 partial results of a segment cut between CTAs are
// joined by a second kernel, in CTA order. (A join by the CTA that finishes last, in this
// kernel, took 5 us against 2.5, and its registers spilled the main loop's: 71 us against the
// 43 that the kernel took then, at 131,071 keys of 8 heads.)
//
// Within a CTA each of 8 warps takes every eighth chunk (4,608 bytes: 64, 32 or
// 16 tokens for head_dim 64, 128, 256) and owns a ring of bulk copies into
// shared memory, so no barrier but a piece's final merge is shared.
//
// Per chunk, with mma.sync m16n8k16 (fp16 inputs, fp32 sums):
//   scores  z[token][col] = c[col] * sum_g (s_tg * (codes . q)_g + b_tg * X_g[col])
//     where X_g is q's sum over group g. A nibble masked in place is an fp16
//     subnormal, code * 2^-24 (or * 2^-20 for the high nibble of a byte, whose
//     query element is divided by 16), so one AND makes two exact operands.
//   weights p = 2^(z - m), m a bound that moves only when some z passes it by 8
//     (so p <= 2^8), the sums then rescaled.
//   output  o[dim][col] = sum_t code_td w_tg + sum_t p f b_tg, w = p f s_tg: the
//     scale goes into the weights, one fp16 operand per group; f is a power of two, part of
//     the exponent's bound, that brings the largest scale to [2^5, 2^7) so that weights use
//     fp16's range whatever the values' magnitude. Rounding w to fp16 is the one
//     rounding beyond fp32: 2^-11, or where w is below fp16's normal range (2^-14) 2^-25, which is
//     2^-30 to 2^-32 of the warp's largest. A code being up to 15 times what a value varies by, it shows in
//     fp16 outputs (5.5e-4 off in all, 2.1e-4 of it their own rounding). For those the codes
//     count from 8: sum_t (code_td - 8) w_tg + sum_t p f (b_tg + 8 s_tg), the sum of the
//     rounded weights coming out of one product more a group (3.0e-4; 6 % slower, so not
//     for bf16, whose own rounding is 1.7e-3).
//
// What it measured, 32 query heads on 8 kv heads of 128 but where said, join included:
//   1 sequence, 131,071 keys, 151 MB of records: 39.3 us, 3.8 TB/s, 0.58 of the copy bandwidth
//     measured on this GPU, DRAM reads 1.00 of the records. About 7 us are the start (schedule, page
//     id, first chunk) and the join; in between 5.5 to 6.3 TB/s, 55 % of the cycles issuing.
//   64 ragged sequences to 8,192 keys, 307 MB: 73.4 us, 4.2 TB/s, 0.63; CTAs end 63 us in on average, the last 70.
//   head_dim 256, 16 query heads, 16 sequences, windows of 1,024, 35 MB: 19.6 us, 0.28: six rounds of
//     chunks for the 12 warps of a CTA. 100,000 keys, 8 columns: 59 us, 0.59.
//   1 sequence, 16 query heads, 333 keys: 7.3 us, the start alone; 512 keys 7.6, 8,192 10.9, 65,536 25.4.
#include <type_traits>

#include <cuda_bf16.h>

#include "kv_internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kMostWarps = 12;  // of a CTA
constexpr int kChunkBytes = 4608;
constexpr float kLazy = 8.0f;   // how far a score may pass the bound before it moves (log2)
constexpr float kNone = -3e38f;  // the bound before any score
// What a piece costs beside its blocks (merge, queries, the last chunks' latency), in blocks. 64
// ragged sequences to 8,192 keys, 100 to 3,000, 256 to 1,000, 8 heads of 128, us at 0, 12, 24, 48, 80:
// 94 83 76 75 77; 73 61 - 54 56; 89 70 61 62 64. Blocks of head_dim 256 are twice as
// long: at 0, 10, 20, 30, 40, 24 sequences to 6,000 keys, 100 to 3,000 and 64 to 1,000: 76 63 50 50 51; 128 116
// 104 101 103; 76 49 41 40 41.
constexpr int piece_cost(int d) { return d == 256 ? 30 : 40; }

constexpr int kPlanBytes = 2304;  // of the schedule, at least

template <int D, int NT>
struct Shape {
    static constexpr int NG = D / 64, W = D / 32;  // groups; code words of a row that one lane of four holds
    static constexpr int kRec = kv_record_bytes(D);
    static constexpr int SB = kChunkBytes / kRec;  // blocks of a chunk
    static constexpr int NC = 8 * NT;
    // Eight warps, two CTAs an SM. At head_dim 256 one CTA fills an SM's registers, and more at 12 warps of 168 than
    // at 8 of 208: 100,000 keys of 8 heads 61 us against 75.
    static constexpr int kWarps = D == 256 && NT == 1 ? 12 : 8, kThreads = 32 * kWarps;
    static constexpr int kCtas = NT == 1 && D <= 128 ? 2 : 1;  // per SM
    static constexpr int kStages = kCtas == 2 || D == 256 ? 2 : 3;
    static constexpr int kCol = D + 4;  // floats of a column in the merge buffer
    static constexpr int kRing = kWarps * kStages * kChunkBytes;
    static constexpr int kMaxGrid = 160 * kCtas;
    static constexpr int kMerge = kWarps * NC * kCol * 4;
    static constexpr int kSmall = (4 * kWarps * NC + 2 * NC + 4 * NC + 2 * (NG + 1) * NC + 2 * NT * W * 128) * 4;
    static constexpr size_t kSmem = kRing + kMerge + kSmall + kWarps * kStages * 8 + kPlanBytes;
    static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "the CTAs of an SM share its 228 KB, 1 KB of each taken by the system");
    static constexpr int kSlot = NC * (D + 2);  // floats of one partial result: m[NC], l[NC], o[NC][D]
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float2 affine_of(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// N consecutive 32-bit words of shared memory
template <int N>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&w)[N]) {
    if constexpr (N >= 4) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 v = ptx::lds_u4(a + 4 * i);
            w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
        }
    } else if constexpr (N == 2) {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a) : "memory");
    } else {
        w[0] = ptx::lds_u32(a);
    }
}

// The same, of a record of values. Four words: the lanes of a row four to a bank, so each begins with
// another word and puts them in order.
template <int N>
__device__ __forceinline__ void lds_turned(uint32_t a, int t, uint32_t (&w)[N]) {
    if constexpr (N == 4) {
        const uint32_t r0 = ptx::lds_u32(a + 4 * t), r1 = ptx::lds_u32(a + 4 * ((t + 1) & 3)),
                       r2 = ptx::lds_u32(a + 4 * ((t + 2) & 3)), r3 = ptx::lds_u32(a + 4 * ((t + 3) & 3));
        // ri is word (i + t) mod 4
        const bool odd = t & 1, two = t & 2;
        const uint32_t x0 = odd ? r3 : r0, x1 = odd ? r0 : r1, x2 = odd ? r1 : r2, x3 = odd ? r2 : r3;
        w[0] = two ? x2 : x0, w[1] = two ? x3 : x1, w[2] = two ? x0 : x2, w[3] = two ? x1 : x3;
    } else {
        lds_words<N>(a, w);
    }
}

template <class T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
    return affine_of(w);
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ void store4(__half* p, float4 v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_h2(v.x, v.y), pack_h2(v.z, v.w));
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// n / d, by 32-bit division where it will do.
__device__ __forceinline__ int64_t quot(int64_t n, int64_t d) {
    if ((uint64_t)(n | d) >> 32) return n / d;
    return (int64_t)((uint32_t)n / (uint32_t)d);
}

// One sequence as the schedule sees it.
struct Seq {
    int first, n, len, lo_blk, per, nct;  // first q row, new tokens, keys, first block seen, blocks of a segment, column tiles
};

__device__ __forceinline__ Seq seq_of(const KvAttend& a, int b, int NC) {
    Seq s;
    if (a.q_start) {
        s.first = min(max(*(a.q_start + b), 0), a.n_q);  // within q whatever q_start holds
        s.n = min(*(a.q_start + b + 1), a.n_q) - s.first;
    } else {
        s.first = b * a.T;
        s.n = a.T;
    }
    s.len = max(0, min(*(a.kv_len + b), a.max_pages << a.c.page_shift));
    const int pos0 = s.len - s.n;
    s.lo_blk = (a.window && pos0 >= a.window ? pos0 - a.window + 1 : 0) >> 4;
    s.per = max(1, ((s.len + 15) >> 4) - s.lo_blk);  // a segment without keys is one unit: its rows become zeros
    s.nct = s.n > 0 ? (int)quot((int64_t)s.n * a.G + NC - 1, NC) : 0;
    return s;
}

// How the segments' blocks are cut into the CTAs' ranges. Either (pad) a range
// holds one segment's blocks at most, a segment taking whole ranges; or segments
// lie end to end, each with some units before its blocks for what a piece costs beside
// them (piece_cost).
struct Cut {
    int64_t quota, total;
    int lead;  // units before a segment's blocks
    bool pad;
    __device__ __forceinline__ int64_t seg_units(int per) const {
        return pad ? quot(per + quota - 1, quota) * quota : per + lead;
    }
};

// A piece: the part of a segment that a CTA's range holds.
struct Piece {
    int first, n, len;   // the sequence: first q row, new tokens, keys
    int h, c0;           // kv head, first column
    int blk, nb;         // first block (of the sequence) and blocks; nb = 0 where there are no keys
    int parts;           // how many CTAs share the segment
    int start;           // 1: the piece holds the segment's first block
    int rot;             // which warp takes its first chunk
    int all_lo, all_hi;  // the keys that every column sees
    const int32_t* table;  // the sequence's page ids
    const uint8_t* head;   // the head's records of page 0
};

constexpr int kPieces = 32;  // pieces of one list

// What a block knows of the schedule, in shared memory.
struct Plan {
    Cut cut;
    int64_t w, w1;     // the CTA's range
    int64_t ex;        // where sequence b's units start
    int b, seg;        // the next piece's sequence, and its segment there
    Seq s;             // that sequence
    int count, more;   // pieces of the list; whether another list follows
    union {
        Piece piece[kPieces];
        struct {  // while the range is worked out, before any piece is listed
            int64_t scan[kMostWarps];
            int2 most[kMostWarps];
        };
    };
};

static_assert(sizeof(Plan) <= kPlanBytes);

// The piece of segment seg of sequence s (index b) that starts at block lo of the segment.
template <int NC, int kRec>
__device__ __forceinline__ Piece piece_of(const KvAttend& a, const Seq& s, int b, uint32_t seg, int lo, int nb, int rot,
                                          int parts) {
    Piece p;
    p.first = s.first, p.n = s.n, p.len = s.len;
    p.h = (int)(seg / (uint32_t)s.nct);
    p.c0 = (int)(seg - (uint32_t)p.h * (uint32_t)s.nct) * NC;
    p.blk = s.lo_blk + lo;
    p.nb = nb;
    p.parts = parts;
    p.start = lo == 0;
    p.rot = rot;
    const int pos0 = s.len - s.n, first = pos0 + (int)a.by_g.div(p.c0);
    const int last = pos0 + (int)a.by_g.div(min(p.c0 + NC, s.n * a.G) - 1);
    p.all_hi = a.causal ? min(s.len, first + 1) : s.len;
    p.table = a.table + (int64_t)b * a.table_stride;
    p.head = a.c.pages + (size_t)p.h * (a.c.P >> 4) * kRec;
    p.all_lo = a.window && last >= a.window ? last - a.window + 1 : 0;
    return p;
}

// Cuts U blocks in Sg segments of at most `most` blocks into ranges for the grid.
__device__ __forceinline__ Cut make_cut(const KvAttend& a, int64_t U, int64_t Sg, int most, int lead) {
    Cut c;
    const int grid = gridDim.x;
    c.lead = lead;
    c.total = U + Sg * lead;
    c.quota = quot(c.total + grid - 1, grid);
    c.pad = false;
    if (Sg <= grid) {  // fewer segments than CTAs: the same number of whole CTAs for each, unless that is too uneven
        const int per = (int)((uint32_t)grid / (uint32_t)max((int)Sg, 1));
        const int each = max(a.min_units, (int)((uint32_t)(most + per - 1) / (uint32_t)per));
        if (each <= max((int64_t)a.min_units, c.quota + lead)) c.quota = each, c.lead = 0, c.pad = true;
    }
    return c;
}

template <class I>
__device__ __forceinline__ I warp_inclusive(I x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const I y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// The CTA's range, and the sequence and segment that it starts in. 0: the range is
// empty; 1: its pieces are to be listed; 2: it is a single piece, listed already. Up to 32
// sequences, each warp works it out by itself and warp 0 writes it down; the block
// is not synchronised.
template <int NC, int kLead, int kRec, int kWarps>
__device__ __forceinline__ int make_plan(const KvAttend& a, Plan& P, int tid, int warp, int lane) {
    const int H = a.c.H;
    if (a.B <= 32) {
        Seq s{};
        if (lane < a.B) s = seq_of(a, lane, NC);
        const int64_t segs = (int64_t)H * s.nct;
        int64_t U = segs * s.per, Sg = segs;
        const int most = __reduce_max_sync(kFull, s.nct ? s.per : 0);
        if (a.B > 1) {
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                U += __shfl_xor_sync(kFull, U, o);
                Sg += __shfl_xor_sync(kFull, Sg, o);
            }
        } else {
            U = __shfl_sync(kFull, U, 0), Sg = __shfl_sync(kFull, Sg, 0);
        }
        Cut c = make_cut(a, U, Sg, most, kLead);
        const int64_t v = lane < a.B ? c.seg_units(s.per) * segs : 0;
        const int64_t inc = a.B > 1 ? warp_inclusive(v, lane) : v, e = inc - v;
        c.total = __shfl_sync(kFull, inc, a.B > 1 ? 31 : 0);
        const int64_t w = c.quota * blockIdx.x;
        if (w >= c.total) return 0;
        if (warp == 0 && e <= w && w < e + v && c.pad) {
            // a range can be as long as the page table is wide, so that offsets of ranges pass 32 bits
            const int units = (int)c.seg_units(s.per), seg = (int)quot(w - e, units);
            const int lo = (int)(w - e - (int64_t)seg * units), nb = s.len > 0 ? min((int)c.quota, s.per - lo) : 0;
            P.piece[0] = piece_of<NC, kRec>(a, s, lane, (uint32_t)seg, lo, nb, 0, (int)((uint32_t)units / (uint32_t)c.quota));
            P.count = 1, P.more = 0;
        } else if (warp == 0 && e <= w && w < e + v) {
            P.cut = c;
            P.w = w;
            P.w1 = min(c.total, w + c.quota);
            P.ex = e;
            P.b = lane;
            P.seg = (int)quot(w - e, c.seg_units(s.per));
            P.s = s;
        }
        __syncwarp();
        return c.pad ? 2 : 1;
    }
    int64_t U = 0, Sg = 0;
    int most = 0;
    for (int b = tid; b < a.B; b += 32 * kWarps) {
        const Seq s = seq_of(a, b, NC);
        const int64_t segs = (int64_t)H * s.nct;
        U += segs * s.per, Sg += segs;
        if (s.nct) most = max(most, s.per);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        U += __shfl_xor_sync(kFull, U, o);
        Sg += __shfl_xor_sync(kFull, Sg, o);
    }
    most = __reduce_max_sync(kFull, most);
    if (lane == 0) P.scan[warp] = U, P.most[warp] = make_int2(most, (int)min(Sg, (int64_t)1 << 30));
    __syncthreads();
    U = 0, Sg = 0, most = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) U += P.scan[i], most = max(most, P.most[i].x), Sg += P.most[i].y;
    Cut c = make_cut(a, U, Sg, most, kLead);
    const int64_t w = c.quota * blockIdx.x;
    int64_t run = 0;
    for (int base = 0; base < a.B; base += 32 * kWarps) {
        const int b = base + tid;
        Seq s{};
        if (b < a.B) s = seq_of(a, b, NC);
        const int64_t v = b < a.B ? c.seg_units(s.per) * H * s.nct : 0;
        const int64_t inc = warp_inclusive(v, lane);
        __syncthreads();
        if (lane == 31) P.scan[warp] = inc;
        __syncthreads();
        int64_t e = run + inc - v;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp) e += P.scan[i];
            run += P.scan[i];
        }
        if (e <= w && w < e + v) {
            P.ex = e;
            P.b = b;
            P.seg = (int)quot(w - e, c.seg_units(s.per));
            P.s = s;
        }
    }
    if (w >= run) return 0;
    if (tid == 0) {
        c.total = run;
        P.cut = c;
        P.w = w;
        P.w1 = min(run, w + c.quota);
    }
    __syncthreads();
    return 1;
}

// The next list of pieces, by one warp: lane p looks at the p-th segment from the list's first.
template <int NC, int SB, int kRec, int kWarps>
__device__ __forceinline__ void list_pieces(const KvAttend& a, Plan& P, int lane) {
    const Cut c = P.cut;
    int b = P.b;
    int64_t e = P.ex, seg = (int64_t)P.seg + lane;
    Seq s = P.s;
    int64_t u = c.seg_units(s.per), n = (int64_t)a.c.H * s.nct;
    while (seg >= n && b + 1 < a.B && e + n * u < P.w1) {
        seg -= n;
        e += n * u;
        s = seq_of(a, ++b, NC);
        u = c.seg_units(s.per);
        n = (int64_t)a.c.H * s.nct;
    }
    const int64_t at = e + seg * u + c.lead;  // the segment's first block
    const bool in = seg < n && at - c.lead < P.w1;
    const int lo = in ? (int)max((int64_t)0, min(P.w - at, (int64_t)s.per)) : 0;
    const int hi = in ? (int)max((int64_t)0, min(P.w1 - at, (int64_t)s.per)) : 0;
    const bool some = hi > lo;
    const unsigned who = __ballot_sync(kFull, some);
    const int nb = some && s.len > 0 ? hi - lo : 0;
    int chunks = (nb + SB - 1) / SB, rot = chunks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, rot, o);
        if (lane >= o) rot += x;
    }
    if (some)
        P.piece[__popc(who & ((1u << lane) - 1))] = piece_of<NC, kRec>(
            a, s, b, (uint32_t)seg, lo, nb, (int)((unsigned)(rot - chunks) % kWarps),
            (int)quot(at + s.per - 1, c.quota) - (int)quot(at, c.quota) + 1);
    // the next list starts at the segment behind lane 31's
    const bool more = __shfl_sync(kFull, in && at + s.per < P.w1, 31);
    __syncwarp();
    if (lane == 31) {
        P.b = b, P.ex = e, P.seg = (int)seg + 1, P.s = s;
        P.more = more;
    }
    if (lane == 0) P.count = __popc(who);
}

// Four sums of a column (its segment: first q row, kv head, first column), with
// its bound and sum of weights, to the output.
template <class T>
__device__ __forceinline__ void put_out(const KvAttend& a, int first, int h, int c0, int col, int dim, float4 x, float m,
                                        float l) {
    const int i = (int)a.by_g.div(c0 + col), hq = h * a.G + (c0 + col) - i * a.G;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    x.x *= inv, x.y *= inv, x.z *= inv, x.w *= inv;
    store4(static_cast<T*>(a.out) + (int64_t)(first + i) * a.ot + (int64_t)hq * a.oh + dim, x);
    if (a.lse && dim == 0)
        a.lse[(int64_t)(first + i) * a.Hq + hq] = l == 0.0f ? -INFINITY : 0.6931471805599453f * (m + log2f(l));
}

template <int D, int NT, class T>
__global__ void __launch_bounds__((Shape<D, NT>::kThreads), (Shape<D, NT>::kCtas))
    kv_decode_kernel(const __grid_constant__ KvAttend a) {
    using S = Shape<D, NT>;
    constexpr int NG = S::NG, W = S::W, SB = S::SB, NC = S::NC, kRec = S::kRec, kStages = S::kStages;
    constexpr int kWarps = S::kWarps, kThreads = S::kThreads;
    constexpr bool kCentre = std::is_same<T, __half>::value;
    extern __shared__ __align__(128) unsigned char smem[];
    unsigned char* ring = smem;
    float* merge = reinterpret_cast<float*>(smem + S::kRing);
    float* sm_stat = reinterpret_cast<float*>(smem + S::kRing + S::kMerge);  // [2][2][kWarps][NC]: by piece parity, bounds and sums
    float* sm_w = sm_stat + 4 * kWarps * NC;  // [2][NC]: the merged bound and sum
    int2* sm_see = reinterpret_cast<int2*>(sm_w + 2 * NC);            // [2][NC]: the keys [x, y) that a column sees
    float* sm_x = reinterpret_cast<float*>(sm_see + 2 * NC);           // [2][NG + 1][NC]: X_g, then cz (below)
    uint32_t* sm_q = reinterpret_cast<uint32_t*>(sm_x + 2 * (NG + 1) * NC);  // [2][NT][W][32][4]: query fragments
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm_q + 2 * NT * W * 128);
    Plan& plan = *reinterpret_cast<Plan*>(bars + kWarps * kStages);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    if (lane < kStages) ptx::mbar_init(bars + warp * kStages + lane, 1);
    ptx::fence_mbar_init();
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    if (tid == 0 && a.join) a.join[blockIdx.x].parts = 0;
    const int planned = make_plan<NC, piece_cost(D), kRec, kWarps>(a, plan, tid, warp, lane);
    if (!planned) return;

    uint32_t use_n = 0;  // chunks used
    uint32_t valid = 0;  // per stage, 4 bits: the blocks that were asked for; bit 16 + stage: in flight
    bool dead = false;   // a wait expired
    int parity = 0;
    uint64_t* const mybars = bars + warp * kStages;
    unsigned char* const myring = ring + warp * kStages * kChunkBytes;

#pragma unroll 1
  for (;;) {  // lists of pieces
    if (warp == 0 && planned == 1) list_pieces<NC, SB, kRec, kWarps>(a, plan, lane);
    __syncthreads();
    const int count = plan.count;

    // ---- loads: this warp's chunks, kStages ahead, and the page of the one after ----
    int ld_p = -1, ld_c = 1 << 20, ld_page = 0;  // piece, next chunk, this lane's page of it
    auto first_chunk = [&](int rot) { return warp >= rot ? warp - rot : warp - rot + kWarps; };
    auto find = [&]() {  // moves on to a piece with a chunk for this warp, and fetches its page id
        while ((ld_p < 0 || ld_c * SB >= plan.piece[ld_p].nb) && ++ld_p < count)
            ld_c = first_chunk(plan.piece[ld_p].rot);
        if (ld_p < count) {
            const Piece& p = plan.piece[ld_p];
            const int i = ld_c * SB + lane;
            if (lane < SB && i < p.nb) ld_page = *(p.table + ((p.blk + i) >> (a.c.page_shift - 4)));
        }
    };
    auto issue = [&](int st) {
        if (ld_p >= count || dead) return;
        const Piece& p = plan.piece[ld_p];
        const int i = ld_c * SB + lane;
        bool ok = lane < SB && i < p.nb;
        if (ok && (unsigned)ld_page >= (unsigned)a.c.n_pages) {
            *(volatile unsigned*)a.bad = 1u;
            ok = false;
        }
        const unsigned v = __ballot_sync(kFull, ok);
        if (lane == 0) ptx::mbar_arrive_expect_tx(mybars + st, __popc(v) * kRec);
        __syncwarp();
        if (ok) {
            const int in = (p.blk + i) & ((a.c.P >> 4) - 1);
            ptx::bulk_g2s(myring + st * kChunkBytes + lane * kRec,
                          p.head + ((size_t)ld_page * a.c.H * (a.c.P >> 4) + in) * kRec, kRec, mybars + st);
        }
        valid = (valid & ~(15u << (4 * st))) | (v << (4 * st)) | (65536u << st);
        ld_c += kWarps;
        find();
    };

    // row g of a score tile holds token pi(g) of its half block: 0 1 3 2 4 5 7 6, so that the
    // four lanes of a value fragment read rows of both parities (half as many bank conflicts)
    const int pg = g ^ ((g >> 1) & 1);

    // ---- a piece's queries: fp16 fragments in shared memory, each warp NT of its columns ----
    constexpr int E = D / 32;  // elements of a lane
    struct RawQ {
        uint32_t w[NT][E / 2];
    };
    auto fetch_q = [&](int i) {
        const Piece& p = plan.piece[i];
        RawQ r{};
        if (kWarps > 8 && warp >= 8) return r;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int c = p.c0 + nt * 8 + warp, tk = (int)a.by_g.div(c), hq = c - tk * a.G;
            const unsigned* qp = reinterpret_cast<const unsigned*>(
                static_cast<const T*>(a.q) + (int64_t)(p.first + tk) * a.qt + (int64_t)(p.h * a.G + hq) * a.qh + lane * E);
#pragma unroll
            for (int k = 0; k < E / 2; ++k) r.w[nt][k] = tk < p.n ? *(qp + k) : 0u;
        }
        return r;
    };
    // the next piece's queries into the cache while this one's chunks are worked on (held in registers
    // they would spill)
    auto touch_q = [&](int i) {
        const Piece& p = plan.piece[i];
        constexpr int kLines = (D * 2 + 127) / 128;  // of a row
        const int c = p.c0 + warp + lane / kLines * 8, tk = (int)a.by_g.div(c), hq = c - tk * a.G;
        if ((kWarps == 8 || warp < 8) && lane < NT * kLines && tk < p.n)
            asm volatile("prefetch.global.L1 [%0];" ::"l"(static_cast<const T*>(a.q) + (int64_t)(p.first + tk) * a.qt +
                                                          (int64_t)(p.h * a.G + hq) * a.qh + lane % kLines * 64));
    };
    // A row is scaled by a power of two to a largest element in [2^10, 2^11), and by the sign
    // of the scale; pairs 1 and 3 of a word are divided by 16 to meet codes times 16.
    auto prepare_q = [&](int i, int par, const RawQ& r) {
        const Piece& p = plan.piece[i];
        if (kWarps > 8 && warp >= 8) return;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int tk = (int)a.by_g.div(p.c0 + nt * 8 + warp);
            const bool in = tk < p.n;
            const uint32_t(&raw)[E / 2] = r.w[nt];
            float top = 0.0f;
#pragma unroll
            for (int k = 0; k < E / 2; ++k) {
                const float2 f = unpack2<T>(raw[k]);
                top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
            // non-negative floats compare as integers
            top = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(top)));
            int ex = (int)((__float_as_uint(top) >> 23) & 255u) - 127;  // floor(log2 top)
            ex = top == 0.0f || ex == 128 ? 10 : min(max(ex, -100), 110);
            float f = __uint_as_float((uint32_t)(127 + 10 - ex) << 23);
            if (a.scale_log2 <= 0.0f) f = a.scale_log2 < 0.0f ? -f : 0.0f;
            float xs = 0.0f;
#pragma unroll
            for (int k = 0; k < E / 2; ++k) {
                const int dim = lane * E + 2 * k, j = dim >> 6, w = ((dim & 63) >> 3) * NG + j, e = (dim & 7) >> 1;
                const float2 v = unpack2<T>(raw[k]);
                const float sc = (e & 1) ? f * 0.0625f : f;
                const uint32_t h = pack_h2(v.x * sc, v.y * sc);
                const float2 y = affine_of(h);
                xs += (y.x + y.y) * ((e & 1) ? 16.0f : 1.0f);
                // word w = t * W + k of the row: fragment k of lane (g = column, t)
                sm_q[((par * NT + nt) * W + w % W) * 128 + (warp * 4 + w / W) * 4 + e] = h;
            }
#pragma unroll
            for (int o = 32 / NG / 2; o; o >>= 1) xs += __shfl_xor_sync(kFull, xs, o);
            float* sx = sm_x + par * (NG + 1) * NC + nt * 8 + warp;
            if (lane % (32 / NG) == 0) sx[lane / (32 / NG) * NC] = xs * 0x1p-24f;
            if (lane == 0) {
                sx[NG * NC] = a.scale_log2 == 0.0f ? 1.0f
                                                   : fabsf(a.scale_log2) *
                                                         __uint_as_float((uint32_t)(127 - 10 + ex) << 23) * 16777216.0f;
                const int pos = p.len - p.n + tk;
                sm_see[par * NC + nt * 8 + warp] =
                    make_int2(a.window && pos >= a.window ? pos - a.window + 1 : 0,
                              in ? (a.causal ? min(p.len, pos + 1) : p.len) : 0);
            }
        }
    };
    // the first queries are asked for ahead of the cache, or they would queue behind it
    RawQ first_q{};
    if (count) first_q = fetch_q(0);
    find();
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) issue((int)((use_n + i) % kStages));
    if (count) prepare_q(0, parity, first_q);
    __syncthreads();

#pragma unroll 1
    for (int ip = 0; ip < count; ++ip, parity ^= 1) {
        const Piece& pc = plan.piece[ip];
        const int nb = pc.nb, blk0 = pc.blk;
        if (ip + 1 < count) touch_q(ip + 1);
        const float* const sx = sm_x + parity * (NG + 1) * NC + 2 * t;
        const uint32_t sq = ptx::smem_addr(sm_q + parity * NT * W * 128 + lane * 4);
        float cz[NT][2];  // scores are cz times the sums below, cz > 0
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float2 v = *reinterpret_cast<const float2*>(sx + NG * NC + nt * 8);
            cz[nt][0] = v.x, cz[nt][1] = v.y;
        }

        // The sums hold 2^(cz z - me): me = m - lf, m within kLazy of the largest cz z so far, 2^lf the
        // factor that keeps weight times scale within fp16's range. thr: the z that passes the bound; lim: the largest
        // scale (by magnitude) that 2^lf serves.
        float o[NT][D / 16][4], wsum[NT][4], bacc[NT][NG][2], thr[NT][2], me[NT][2], l[NT][2], lim = 0.0f, lf = 24.0f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) wsum[nt][e] = 0.0f;
#pragma unroll
            for (int j = 0; j < NG; ++j) bacc[nt][j][0] = bacc[nt][j][1] = 0.0f;
#pragma unroll
            for (int e = 0; e < 2; ++e) thr[nt][e] = me[nt][e] = kNone, l[nt][e] = 0.0f;
        }

#pragma unroll 1
        for (int c = first_chunk(pc.rot); c * SB < nb; c += kWarps) {
            const int st = (int)(use_n % kStages);
            if (!dead && !ptx::mbar_wait_bounded(mybars + st, (use_n / kStages) & 1, nullptr)) {
                dead = true;
                if (lane == 0) *(volatile unsigned*)a.err = 1024u;
            }
            dead = __any_sync(kFull, dead);
            if (dead) break;
            const uint32_t base = ptx::smem_addr(myring) + st * kChunkBytes;
            const unsigned v = (valid >> (4 * st)) & 15u;
            const int tok0 = (blk0 + c * SB) << 4;
            const bool whole = v == (1u << SB) - 1 && tok0 >= pc.all_lo && tok0 + 16 * SB <= pc.all_hi;

            // the query fragments and X come from shared memory once a chunk: held in registers they
            // would not leave room for two CTAs
            uint4 qf[NT][W];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < W; ++k) qf[nt][k] = ptx::lds_u4(sq + (nt * W + k) * 512);
            float z[SB][NT][4];
            uint32_t va[SB][2][NG];  // value affine words of tokens pi(g), pi(g) + 8
#pragma unroll
            for (int sb = 0; sb < SB; ++sb) {
                const uint32_t rec = base + sb * kRec;
                uint32_t kw[2][W], ka[2][NG];
                float2 X[NT][NG];
                lds_words<W>(rec + pg * (D / 2) + t * W * 4, kw[0]);
                lds_words<W>(rec + (pg + 8) * (D / 2) + t * W * 4, kw[1]);
                lds_words<NG>(rec + kv_k_affine(D) + pg * NG * 4, ka[0]);
                lds_words<NG>(rec + kv_k_affine(D) + (pg + 8) * NG * 4, ka[1]);
                lds_words<NG>(rec + kv_v_affine(D) + pg * NG * 4, va[sb][0]);
                lds_words<NG>(rec + kv_v_affine(D) + (pg + 8) * NG * 4, va[sb][1]);
                float acc[NG][NT][4];
#pragma unroll
                for (int j = 0; j < NG; ++j)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[j][nt][e] = 0.0f;
#pragma unroll
                for (int k = 0; k < W; ++k) {
                    const uint32_t x0 = kw[0][k], x1 = kw[1][k], y0 = x0 >> 8, y1 = x1 >> 8;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma(acc[k % NG][nt], x0 & 0x000F000Fu, x1 & 0x000F000Fu, x0 & 0x00F000F0u, x1 & 0x00F000F0u,
                            qf[nt][k].x, qf[nt][k].y);
                        mma(acc[k % NG][nt], y0 & 0x000F000Fu, y1 & 0x000F000Fu, y0 & 0x00F000F0u, y1 & 0x00F000F0u,
                            qf[nt][k].z, qf[nt][k].w);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < NG; ++j) X[nt][j] = *reinterpret_cast<const float2*>(sx + j * NC + nt * 8);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[sb][nt][e] = 0.0f;
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    const float2 r0 = affine_of(ka[0][j]), r1 = affine_of(ka[1][j]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        z[sb][nt][0] = fmaf(r0.x, acc[j][nt][0], fmaf(r0.y, X[nt][j].x, z[sb][nt][0]));
                        z[sb][nt][1] = fmaf(r0.x, acc[j][nt][1], fmaf(r0.y, X[nt][j].y, z[sb][nt][1]));
                        z[sb][nt][2] = fmaf(r1.x, acc[j][nt][2], fmaf(r1.y, X[nt][j].x, z[sb][nt][2]));
                        z[sb][nt][3] = fmaf(r1.x, acc[j][nt][3], fmaf(r1.y, X[nt][j].y, z[sb][nt][3]));
                    }
                }
            }
            if (!whole) {
#pragma unroll
                for (int sb = 0; sb < SB; ++sb) {
                    const int tk = tok0 + sb * 16 + pg;
                    const bool in = (v >> sb) & 1;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int k = tk + (e & 2) * 4;
                            const int2 see = sm_see[parity * NC + nt * 8 + 2 * t + (e & 1)];
                            if (!in || k < see.x || k >= see.y) z[sb][nt][e] = -INFINITY;
                        }
                    // places past the sequence's end hold anything: their scale must not move lf
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        if (!in || tk + 8 * r >= pc.len)
#pragma unroll
                            for (int j = 0; j < NG; ++j) va[sb][r][j] = 0;
                }
            }
            // does a score or a scale pass its bound?
            bool over = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float top = fmaxf(z[0][nt][e], z[0][nt][e + 2]);
#pragma unroll
                    for (int sb = 1; sb < SB; ++sb) top = fmaxf(top, fmaxf(z[sb][nt][e], z[sb][nt][e + 2]));
                    over |= top > thr[nt][e];
                }
            __half2 sm = __float2half2_rn(0.0f);
#pragma unroll
            for (int sb = 0; sb < SB; ++sb)
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int j = 0; j < NG; ++j)
                        sm = __hmax2(sm, __habs2(*reinterpret_cast<const __half2*>(&va[sb][r][j])));
            const float smax = __low2float(sm);
            over |= smax > lim;
            if (__any_sync(kFull, over)) {
                float top = smax;
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, x));
                if (top > lim) {  // the same in every lane
                    const int ex = min(max((int)(__float_as_uint(top) >> 23) - 127, -24), 15);
                    lf = (float)(5 - ex);  // the weights stay below 2^(kLazy + 5 + 2)
                    lim = __uint_as_float((uint32_t)(127 + 2 + ex) << 23);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = kNone;
#pragma unroll
                        for (int sb = 0; sb < SB; ++sb) mx = fmaxf(mx, fmaxf(z[sb][nt][e], z[sb][nt][e + 2]));
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, x));
                        mx = fmaxf(thr[nt][e] == kNone ? kNone : fmaf(thr[nt][e], cz[nt][e], -kLazy),
                                   mx == kNone ? kNone : mx * cz[nt][e]);
                        const float sc = ex2(me[nt][e] - (mx - lf));
                        thr[nt][e] = mx == kNone ? kNone : (mx + kLazy) / cz[nt][e];
                        me[nt][e] = mx - lf;
                        l[nt][e] *= sc;
                        if (kCentre) wsum[nt][e] *= sc;
#pragma unroll
                        for (int j = 0; j < NG; ++j) bacc[nt][j][e] *= sc;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) o[nt][i][e] *= sc, o[nt][i][e + 2] *= sc;
                    }
            }
#pragma unroll
            for (int sb = 0; sb < SB; ++sb) {
                const uint32_t rec = base + sb * kRec;
                // tokens pi(2t), pi(2t+1), and the same plus 8: k index 2t, 2t+1, 2t+8, 2t+9 of the product
                uint32_t vw[4][NG];
                const int ta = (2 * t) ^ (t & 1), tb = (2 * t + 1) ^ (t & 1);
                const uint32_t vr = rec + kv_v_codes(D) + g * NG * 4;
                lds_turned<NG>(vr + ta * (D / 2), t, vw[0]);
                lds_turned<NG>(vr + tb * (D / 2), t, vw[1]);
                lds_turned<NG>(vr + (ta + 8) * (D / 2), t, vw[2]);
                lds_turned<NG>(vr + (tb + 8) * (D / 2), t, vw[3]);
                float p[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[nt][e] = ex2(fmaf(z[sb][nt][e], cz[nt][e & 1], -me[nt][e & 1]));
                        l[nt][e & 1] += p[nt][e];
                    }
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    float2 r0 = affine_of(va[sb][0][j]), r1 = affine_of(va[sb][1][j]);
                    if (kCentre) {
                        r0.y = fmaf(8.0f, r0.x, r0.y), r1.y = fmaf(8.0f, r1.x, r1.y);
                        // a group that is not finite: this bias says so, and its weights would reach the other groups' sums
                        if (!(fabsf(r0.x) <= 65504.0f)) r0.x = 0.0f;
                        if (!(fabsf(r1.x) <= 65504.0f)) r1.x = 0.0f;
                    }
                    uint32_t pb[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float w0 = p[nt][0] * r0.x, w1 = p[nt][1] * r0.x, w2 = p[nt][2] * r1.x, w3 = p[nt][3] * r1.x;
                        if (whole) {
                            bacc[nt][j][0] = fmaf(p[nt][0], r0.y, fmaf(p[nt][2], r1.y, bacc[nt][j][0]));
                            bacc[nt][j][1] = fmaf(p[nt][1], r0.y, fmaf(p[nt][3], r1.y, bacc[nt][j][1]));
                        } else {  // an unseen value may be NaN or infinite
                            const float n = -INFINITY;
                            if (z[sb][nt][0] == n) w0 = 0.0f; else bacc[nt][j][0] = fmaf(p[nt][0], r0.y, bacc[nt][j][0]);
                            if (z[sb][nt][1] == n) w1 = 0.0f; else bacc[nt][j][1] = fmaf(p[nt][1], r0.y, bacc[nt][j][1]);
                            if (z[sb][nt][2] == n) w2 = 0.0f; else bacc[nt][j][0] = fmaf(p[nt][2], r1.y, bacc[nt][j][0]);
                            if (z[sb][nt][3] == n) w3 = 0.0f; else bacc[nt][j][1] = fmaf(p[nt][3], r1.y, bacc[nt][j][1]);
                        }
                        pb[nt][0] = transpose8x8(pack_h2(w0, w1));
                        pb[nt][1] = transpose8x8(pack_h2(w2, w3));
                    }
                    // two tokens' nibbles side by side: low halves hold elements 0, 2, 4, 6, high halves 1, 3, 5, 7
                    const uint32_t u0 = __byte_perm(vw[0][j], vw[1][j], 0x5410);
                    const uint32_t h0 = __byte_perm(vw[0][j], vw[1][j], 0x7632);
                    const uint32_t u1 = __byte_perm(vw[2][j], vw[3][j], 0x5410);
                    const uint32_t h1 = __byte_perm(vw[2][j], vw[3][j], 0x7632);
                    const uint32_t ones = g == j ? 0x3C003C00u : 0u;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if (kCentre) mma(wsum[nt], ones, 0u, ones, 0u, pb[nt][0], pb[nt][1]);
                        mma(o[nt][j * 4 + 0], u0 & 0x000F000Fu, h0 & 0x000F000Fu, u1 & 0x000F000Fu, h1 & 0x000F000Fu,
                            pb[nt][0], pb[nt][1]);
                        mma(o[nt][j * 4 + 1], u0 & 0x00F000F0u, h0 & 0x00F000F0u, u1 & 0x00F000F0u, h1 & 0x00F000F0u,
                            pb[nt][0], pb[nt][1]);
                        mma(o[nt][j * 4 + 2], (u0 >> 8) & 0x000F000Fu, (h0 >> 8) & 0x000F000Fu, (u1 >> 8) & 0x000F000Fu,
                            (h1 >> 8) & 0x000F000Fu, pb[nt][0], pb[nt][1]);
                        mma(o[nt][j * 4 + 3], (u0 >> 8) & 0x00F000F0u, (h0 >> 8) & 0x00F000F0u, (u1 >> 8) & 0x00F000F0u,
                            (h1 >> 8) & 0x00F000F0u, pb[nt][0], pb[nt][1]);
                    }
                }
            }
            ++use_n;
            valid &= ~(65536u << st);
            __syncwarp();
            issue(st);
        }

        if (ip + 1 < count) prepare_q(ip + 1, parity ^ 1, fetch_q(ip + 1));
        float* sm_m = sm_stat + parity * 2 * kWarps * NC;  // [kWarps][NC]
        float* sm_l = sm_m + kWarps * NC;
        // ---- merge the warps ----
        // o[nt][4j + i][e]: dim 64j + 8g + 2i + (e >> 1), column 8nt + 2t + (e & 1), in units of 2^-24
        // (odd i: 2^-20)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) {
                    l[nt][e] += __shfl_xor_sync(kFull, l[nt][e], x);
#pragma unroll
                    for (int j = 0; j < NG; ++j) bacc[nt][j][e] += __shfl_xor_sync(kFull, bacc[nt][j][e], x);
                }
                if (kCentre)
#pragma unroll
                    for (int j = 0; j < NG; ++j)
                        bacc[nt][j][e] = fmaf(-8.0f, __shfl_sync(kFull, wsum[nt][e], 4 * j + t), bacc[nt][j][e]);
                if (g == 0) {
                    sm_m[warp * NC + nt * 8 + 2 * t + e] = me[nt][e];
                    sm_l[warp * NC + nt * 8 + 2 * t + e] = l[nt][e];
                }
            }
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int col = nt * 8 + 2 * t + e;
                float M = kNone;
#pragma unroll
                for (int i = 0; i < kWarps; ++i) M = fmaxf(M, sm_m[i * NC + col]);
                const float wt = ex2(me[nt][e] - M);
                float* dst = merge + (warp * NC + col) * S::kCol + 8 * g;
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    float y[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float sc = (i & 1) ? 1048576.0f : 16777216.0f;
                        y[2 * i] = wt * fmaf(o[nt][j * 4 + i][e], sc, bacc[nt][j][e]);
                        y[2 * i + 1] = wt * fmaf(o[nt][j * 4 + i][e + 2], sc, bacc[nt][j][e]);
                    }
                    *reinterpret_cast<float4*>(dst + 64 * j) = make_float4(y[0], y[1], y[2], y[3]);
                    *reinterpret_cast<float4*>(dst + 64 * j + 4) = make_float4(y[4], y[5], y[6], y[7]);
                }
            }
        if (tid < NC) {
            float M = kNone, L = 0.0f;
            for (int i = 0; i < kWarps; ++i) M = fmaxf(M, sm_m[i * NC + tid]);
            for (int i = 0; i < kWarps; ++i) L += sm_l[i * NC + tid] * ex2(sm_m[i * NC + tid] - M);
            sm_w[tid] = M;
            sm_w[NC + tid] = L;
        }
        __syncthreads();

        const int parts = pc.parts, ncols = min(NC, pc.n * a.G - pc.c0);
        float* slot = a.part + (size_t)(2 * blockIdx.x + pc.start) * S::kSlot;
        for (int x = tid; x < ncols * (D / 4); x += kThreads) {
            const int col = x / (D / 4), dim = (x % (D / 4)) * 4;
            float4 y = *reinterpret_cast<const float4*>(merge + col * S::kCol + dim);
#pragma unroll
            for (int i = 1; i < kWarps; ++i) {
                const float4 q = *reinterpret_cast<const float4*>(merge + (i * NC + col) * S::kCol + dim);
                y.x += q.x, y.y += q.y, y.z += q.z, y.w += q.w;
            }
            if (parts == 1)
                put_out<T>(a, pc.first, pc.h, pc.c0, col, dim, y, sm_w[col], sm_w[NC + col]);
            else
                __stcg(reinterpret_cast<float4*>(slot + 2 * NC + col * D + dim), y);
        }
        if (parts > 1) {  // a segment cut between CTAs: kv_join_kernel adds its parts
            if (tid < 2 * NC) __stcg(slot + tid, sm_w[tid]);
            if (pc.start && tid == 0 && a.join) a.join[blockIdx.x] = KvJoin{parts, pc.first, pc.h, pc.c0, ncols};
        }
    }
    if (!plan.more) break;
    __syncthreads();  // the list is read no more
  }
    // a warp that gave up lets the copies already issued land before the CTA can exit
    if (dead)
        for (uint32_t n = use_n; n < use_n + kStages; ++n)
            if (valid >> (16 + n % kStages) & 1) ptx::mbar_wait_bounded(mybars + n % kStages, (n / kStages) & 1, nullptr);
}

// Adds the parts of the segment that starts in the range of CTA blockIdx.x and
// does not end there, if there is one: block y takes column y, D/4 threads times
// four groups of parts. Part 0 lies in that CTA's second slot, part p in the first
// slot of the p-th CTA after it.
template <int D, int NT, class T>
__global__ void __launch_bounds__(D) kv_join_kernel(const __grid_constant__ KvAttend a) {
    using S = Shape<D, NT>;
    constexpr int NC = S::NC, kLanes = D / 4, kGroups = 4, kThreads = D, kWarps = D / 32;
    __shared__ float w[S::kMaxGrid];
    __shared__ float4 sum[kThreads];
    __shared__ float warp_m[kWarps], warp_l[kWarps];
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const KvJoin j = a.join[blockIdx.x];
    const int tid = threadIdx.x, col = blockIdx.y;
    if (col >= j.cols || j.parts == 0) return;
    const float* p0 = a.part + (size_t)(2 * blockIdx.x + 1) * S::kSlot;
    auto part = [&](int p) { return p0 + (p == 0 ? 0 : (2 * p - 1) * S::kSlot); };
    // weights: 2^(bound - largest bound)
    float M = kNone;
    for (int p = tid; p < j.parts; p += kThreads) M = fmaxf(M, w[p] = part(p)[col]);
#pragma unroll
    for (int x = 16; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, x));
    if ((tid & 31) == 0) warp_m[tid >> 5] = M;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i) M = fmaxf(M, warp_m[i]);
    float L = 0.0f;
    for (int p = tid; p < j.parts; p += kThreads) {
        w[p] = ex2(w[p] - M);
        L += part(p)[NC + col] * w[p];
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) L += __shfl_xor_sync(kFull, L, x);
    if ((tid & 31) == 0) warp_l[tid >> 5] = L;
    __syncthreads();
    const int dim = tid % kLanes * 4, grp = tid / kLanes;
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int p = grp; p < j.parts; p += kGroups) {
        const float4 q = *reinterpret_cast<const float4*>(part(p) + 2 * NC + col * D + dim);
        y.x = fmaf(w[p], q.x, y.x), y.y = fmaf(w[p], q.y, y.y), y.z = fmaf(w[p], q.z, y.z), y.w = fmaf(w[p], q.w, y.w);
    }
    sum[tid] = y;
    __syncthreads();
    if (grp) return;
    L = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) L += warp_l[i];
#pragma unroll
    for (int i = 1; i < kGroups; ++i) {
        const float4 q = sum[i * kLanes + tid];
        y.x += q.x, y.y += q.y, y.z += q.z, y.w += q.w;
    }
    put_out<T>(a, j.first, j.h, j.c0, col, dim, y, M, L);
}

template <int D, int NT, class T>
cudaError_t launch_decode(const KvAttend& a, int sms, cudaStream_t s, int* launched) {
    using S = Shape<D, NT>;
    auto kernel = kv_decode_kernel<D, NT, T>;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), S::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    const int grid = min(S::kCtas * sms, S::kMaxGrid);
    const cudaLaunchConfig_t cfg = launch_config(dim3(grid), dim3(S::kThreads), S::kSmem, s, true, &attr);
    e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e != cudaSuccess || !a.join) return e;
    *launched = 2;
    const cudaLaunchConfig_t jcfg = launch_config(dim3(grid, S::NC), dim3(D), 0, s, true, &attr);
    return cudaLaunchKernelEx(&jcfg, kv_join_kernel<D, NT, T>, a);
}

// A tile of 16 columns reads the cache once for what two of 8 read twice, but at an odd number of
// eights half of the last one is idle. 100,000 keys of 8 heads, one sequence, us for tiles of 8
// and of 16 at 8, 16, 20 and 32 columns: head_dim 64: 23 31, 34 32, 44 53, 55 52; 128: 36 51,
// 54 52, 74 89, 94 89; 256: 59 91 at 8, 104 90 at 12, 104 91 at 16.
template <int D, class T>
cudaError_t launch_decode_cols(const KvAttend& a, int cols, int sms, cudaStream_t s, int* launched) {
    const bool wide = D == 256 ? cols > 8 : ((cols + 7) / 8 & 1) == 0 && cols > 8;
    return wide ? launch_decode<D, 2, T>(a, sms, s, launched) : launch_decode<D, 1, T>(a, sms, s, launched);
}

}  // namespace

cudaError_t launch_kv_attend(const KvAttend& a, int d, moe_dtype t, int cols, int sms, cudaStream_t s, int* launched) {
    const bool bf = t == MOE_BF16;
    if (d == 64)
        return bf ? launch_decode_cols<64, __nv_bfloat16>(a, cols, sms, s, launched) : launch_decode_cols<64, __half>(a, cols, sms, s, launched);
    if (d == 128)
        return bf ? launch_decode_cols<128, __nv_bfloat16>(a, cols, sms, s, launched) : launch_decode_cols<128, __half>(a, cols, sms, s, launched);
    return bf ? launch_decode_cols<256, __nv_bfloat16>(a, cols, sms, s, launched) : launch_decode_cols<256, __half>(a, cols, sms, s, launched);
}

}  // namespace moe
