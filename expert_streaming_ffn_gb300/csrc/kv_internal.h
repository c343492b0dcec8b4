// The 4-bit key/value cache: record layout, kernel parameters and launchers.
// Not part of the public ABI (include/moe.h describes the layout).
#pragma once

#include "moe_internal.h"

namespace moe {

constexpr int kKvBlock = 16;  // tokens of a record
MOE_HD constexpr int kv_record_bytes(int d) { return 18 * d; }

// Offsets within a record of the K codes (0), V codes, K and V affine words.
MOE_HD constexpr int kv_v_codes(int d) { return 8 * d; }
MOE_HD constexpr int kv_k_affine(int d) { return 16 * d; }
MOE_HD constexpr int kv_v_affine(int d) { return 17 * d; }

struct KvCache {
    uint8_t* pages;
    int H, P, page_shift;  // kv heads, tokens per page and its log2
    int n_pages;
    unsigned n_slots;  // n_pages * P
};

// n / d for 0 <= n < 2^31, as a multiply and a shift: with 2^(s-1) < d <= 2^s
// and m = ceil(2^(31+s) / d) < 2^32, floor(n m / 2^(31+s)) = floor(n / d).
struct FastDiv {
    uint32_t m, s, d;
    explicit FastDiv(uint32_t d_ = 1) : d(d_) {
        s = 0;
        while ((1ull << s) < d) ++s;
        m = (uint32_t)(((1ull << (31 + s)) + d - 1) / d);
    }
#ifdef __CUDACC__
    __device__ __forceinline__ uint32_t div(uint32_t n) const {
        return (uint32_t)(((uint64_t)n * m) >> (31 + s));
    }
#endif
};

struct KvRows {
    KvCache c;
    const int32_t* slots;
    unsigned n;  // rows: tokens * kv heads
    FastDiv by_head{1};
    // rows: element strides
    const void* k_in;
    const void* v_in;
    void* k_out;
    void* v_out;
    int64_t kt, kh, vt, vh;
    unsigned* bad;  // mapped word: a slot was outside the cache
};

cudaError_t launch_kv_append(const KvRows& a, int d, moe_dtype t, cudaStream_t s);
cudaError_t launch_kv_read(const KvRows& a, int d, moe_dtype t, cudaStream_t s);

// A segment cut between CTAs (parts = 0: none): how many have a part, its first
// q row, kv head, first column and columns.
struct KvJoin {
    int parts, first, h, c0, cols;
};

struct KvAttend {
    KvCache c;
    const void* q;
    void* out;
    float* lse;
    int64_t qt, qh, ot, oh;  // element strides
    const int32_t* table;
    int64_t table_stride;
    const int32_t* kv_len;
    const int32_t* q_start;  // or null
    int B, n_q, Hq, G, max_pages;
    FastDiv by_g{1};  // / G
    int T;  // tokens per sequence when q_start is null
    int causal, window;
    float scale_log2;  // scale * log2(e)
    unsigned* bad;
    unsigned* err;  // mapped word: a bounded wait expired
    // workspace of segments cut between CTAs: per CTA the segment that starts in its
    // range and ends in another's, and two partial results; null: none can be cut
    KvJoin* join;
    float* part;
    // prompts: row tiles of a CTA each, and how many CTAs share the keys of each other one
    int full, splits;
    int min_units;  // fewest blocks of 16 tokens that a CTA takes; a whole segment where none is cut
};

constexpr int kKvMaxCtas = 2;  // resident CTAs per SM of any of the kernels
// Floats of partial results per SM: one row tile's of the prompt kernel, 256 rows of
// 128 elements and two statistics; the decode kernel needs less.
constexpr size_t kKvPartFloats = 256 * (128 + 2);

// *launched gets the number of kernels. cols: query columns (new tokens * query heads per kv head) of a sequence, as the caller knows them
cudaError_t launch_kv_attend(const KvAttend& a, int d, moe_dtype t, int cols, int sms, cudaStream_t s, int* launched);

// The same for many columns a sequence. The plan sets a.full and a.splits and returns the row
// tiles; a call with splits > 1 uses the workspace.
int64_t kv_prompt_plan(KvAttend& a, int d, int max_q, int max_len, int sms);
cudaError_t launch_kv_prompt(const KvAttend& a, int d, moe_dtype t, int64_t work, cudaStream_t s, int* launched);

}  // namespace moe
