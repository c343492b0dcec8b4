// libmoe C ABI: the 4-bit key/value cache and the attention over it.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <new>

#include "kv_internal.h"

using namespace moe;

#define CUDA_TRY(call)                                                                                 \
    do {                                                                                               \
        cudaError_t e_ = (call);                                                                       \
        if (e_ != cudaSuccess)                                                                         \
            return set_error(MOE_ECUDA, "%s failed: %s (%s:%d)", #call, cudaGetErrorString(e_), __FILE__, \
                             __LINE__);                                                                \
    } while (0)

namespace moe {

// What the cache calls of a context keep: mapped words in which kernels note
// bad slots and page ids [0] and expired waits [1], and the attention's
// workspace, with the stream of the last call that uses it and an event behind
// that call.
struct KvState {
    unsigned* bad_host = nullptr;
    unsigned* bad_dev = nullptr;
    int sms = 0;
    unsigned char* ws = nullptr;
    cudaEvent_t ws_done = nullptr;
    unsigned long long ws_stream = 0;  // its id
    bool ws_used = false;
};

KvState* kv_state_create() {
    KvState* n = new (std::nothrow) KvState();
    if (!n) return nullptr;
    if (cudaHostAlloc(&n->bad_host, 2 * sizeof(unsigned), cudaHostAllocMapped) != cudaSuccess ||
        cudaHostGetDevicePointer(&n->bad_dev, n->bad_host, 0) != cudaSuccess) {
        cudaGetLastError();
        kv_state_destroy(n);
        return nullptr;
    }
    n->bad_host[0] = n->bad_host[1] = 0;
    return n;
}

void kv_state_destroy(KvState* st) {
    if (!st) return;
    cudaFreeHost(st->bad_host);
    cudaFree(st->ws);
    if (st->ws_done) cudaEventDestroy(st->ws_done);
    delete st;
}

// Most query columns a sequence (new tokens times query heads of a kv head) that the decode kernel
// takes: it reads the cache once a tile of columns, the prompt kernel once for 256 (128 at head_dim
// 256) whose tiles it fills in any case. us, decode and prompt kernel, one sequence of 16,511 keys and of
// 100,000, 16 of 4,000, 64 of 1,000, 8 heads: head_dim 64: 32 columns 17 22, 53 68, 42 49, 54 64; 48 columns 20 22,
// 72 68, 57 49, 74 64. head_dim 128: 32 columns 25 29, 90 91, 66 64, 83 86; 48 columns 30 29, 126 93, 92 64, 119 86.
// head_dim 256: 16 columns 26 33, 91 131, 72 94, 82 117; 20 columns 35 34, 149 132, 110 94, 137 119.
int decode_cols(int head_dim) { return head_dim == 256 ? 16 : 32; }

// Blocks of 16 tokens that a CTA of the decode kernel takes at least, as too few leave its warps
// without a chunk, and the sequence up to which a segment is left to one CTA, which saves the kernel
// that joins parts. 16 query heads on 8, one sequence, us for 16 and for 32 blocks: head_dim 64, 2,048 tokens:
// 8.5 8.8, 8,192: 9.3 10.5; 128: 9.0 10.3, 10.8 12.6; 256 (for 12 and 24), 1,500: 10.4 11.5. Cut into
// such pieces and whole: 64, 1,024 tokens: 8.6 7.4, 1,536: 8.7 9.0; 128, 512: 9.0 7.5, 640: 8.9 8.6, 768: 9.1 8.9,
// 1,024: 9.0 10.3; 256, 384: 9.8 9.0, 512: 9.7 10.4.
int decode_piece(int head_dim) { return head_dim == 256 ? 12 : 16; }
int decode_whole(int head_dim) { return head_dim == 256 ? 24 : head_dim == 128 ? 48 : 64; }

constexpr size_t kJoinBytes = 1024 * sizeof(KvJoin);  // for up to 1,024 CTAs

// The workspace of an attention call on s, made by the first of them.
moe_status ensure_workspace(KvState* S, int device, cudaStream_t s) {
    if (S->ws) return MOE_OK;
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    CUDA_TRY(cudaStreamIsCapturing(s, &cs));
    if (cs != cudaStreamCaptureStatusNone)  // an allocation would end the capture
        return set_error(MOE_ESTATE, "moe_kv_attend: a context's first attention call cannot be captured (it allocates)");
    int sms = 0;
    CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device));
    if ((size_t)sms * kKvMaxCtas * sizeof(KvJoin) > kJoinBytes)
        return set_error(MOE_ECUDA, "moe_kv_attend: %d SMs are more than it is made for", sms);
    const size_t bytes = kJoinBytes + (size_t)sms * kKvPartFloats * sizeof(float);
    if (!S->ws_done) CUDA_TRY(cudaEventCreateWithFlags(&S->ws_done, cudaEventDisableTiming));
    unsigned char* p = nullptr;
    if (cudaMalloc(&p, bytes) != cudaSuccess) {
        cudaGetLastError();
        return set_error(MOE_ENOMEM, "moe_kv_attend: workspace of %zu bytes failed", bytes);
    }
    S->sms = sms;
    S->ws = p;
    return MOE_OK;
}

// Orders a call on s behind the last call that used the workspace on another
// stream. A call being captured records no event outside its graph. Streams are told apart by
// their ids: a handle can come back after its stream was destroyed, whose work may
// still run, and the per-thread default stream's is the same in every thread.
moe_status workspace_begin(KvState* S, cudaStream_t s, bool* capturing) {
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    CUDA_TRY(cudaStreamIsCapturing(s, &cs));
    *capturing = cs != cudaStreamCaptureStatusNone;
    if (*capturing) return MOE_OK;
    unsigned long long id = 0;
    CUDA_TRY(cudaStreamGetId(s, &id));
    if (S->ws_used && S->ws_stream != id) CUDA_TRY(cudaStreamWaitEvent(s, S->ws_done, 0));
    S->ws_stream = id;
    return MOE_OK;
}

moe_status workspace_end(KvState* S, cudaStream_t s, bool capturing) {
    if (capturing) return MOE_OK;
    CUDA_TRY(cudaEventRecord(S->ws_done, s));
    S->ws_used = true;
    return MOE_OK;
}

}  // namespace moe

namespace {

bool shape_ok(const moe_kv_cache* c) {
    return c && c->n_kv_heads >= 1 && c->n_kv_heads <= 65536 &&
           (c->head_dim == 64 || c->head_dim == 128 || c->head_dim == 256) && c->page_tokens >= 16 &&
           c->page_tokens <= 256 && !(c->page_tokens & (c->page_tokens - 1)) && c->n_pages >= 1 &&
           (int64_t)c->n_pages * c->page_tokens < (int64_t)1 << 31;
}

moe_status check_cache(const char* who, const moe_kv_cache* c) {
    if (!shape_ok(c))
        return set_error(MOE_EINVAL, "%s: bad cache (n_kv_heads >= 1, head_dim 64, 128 or 256, page_tokens 16 to 256 "
                         "and a power of two, n_pages >= 1, n_pages * page_tokens < 2^31)", who);
    if (!c->pages || (reinterpret_cast<uintptr_t>(c->pages) & 15))
        return set_error(MOE_EINVAL, "%s: pages must be a 16-byte aligned device pointer", who);
    return MOE_OK;
}

KvCache view(const moe_kv_cache* c) {
    KvCache v;
    v.pages = static_cast<uint8_t*>(c->pages);
    v.H = c->n_kv_heads;
    v.P = c->page_tokens;
    v.page_shift = 0;
    while ((1 << v.page_shift) < v.P) ++v.page_shift;
    v.n_pages = c->n_pages;
    v.n_slots = (unsigned)c->n_pages * (unsigned)c->page_tokens;
    return v;
}

int type_size(moe_dtype t) { return t == MOE_F32 ? 4 : 2; }

bool rows_ok(const void* p, int64_t ts, int64_t hs, moe_dtype t) {
    const int64_t per = 16 / type_size(t);
    return !(reinterpret_cast<uintptr_t>(p) & 15) && ts % per == 0 && hs % per == 0;
}

moe_status expired(KvState* S) {
    const unsigned code = *(volatile unsigned*)(S->bad_host + 1);
    *(volatile unsigned*)(S->bad_host + 1) = 0;
    return set_error(MOE_ETIMEOUT, "a bounded device wait expired in an earlier attention call (code %u)", code);
}

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

moe_status rows_call(const char* who, moe_ctx* C, const moe_kv_cache* cache, const void* k, int64_t kt, int64_t kh,
                     const void* v, int64_t vt, int64_t vh, moe_dtype dtype, const int32_t* slots, int32_t n_tokens,
                     bool append, void* stream) {
    if (!C) return set_error(MOE_EINVAL, "%s: ctx is NULL", who);
    moe_status st = check_cache(who, cache);
    if (st != MOE_OK) return st;
    if (dtype != MOE_F32 && dtype != MOE_F16 && dtype != MOE_BF16)
        return set_error(MOE_EINVAL, "%s: dtype %d (MOE_F32, MOE_F16 or MOE_BF16)", who, (int)dtype);
    if (n_tokens < 0) return set_error(MOE_EINVAL, "%s: n_tokens = %d", who, n_tokens);
    if ((int64_t)n_tokens * cache->n_kv_heads >= (int64_t)1 << 31)
        return set_error(MOE_EINVAL, "%s: n_tokens * n_kv_heads must be below 2^31", who);
    if (n_tokens == 0) return MOE_OK;
    if (!k || !v || !slots) return set_error(MOE_EINVAL, "%s: NULL argument", who);
    if (!rows_ok(k, kt, kh, dtype) || !rows_ok(v, vt, vh, dtype))
        return set_error(MOE_EINVAL, "%s: rows of k and v must start on 16-byte boundaries", who);
    CUDA_TRY(cudaSetDevice(ctx_device(C)));
    std::lock_guard<std::mutex> lock(ctx_kv_mutex(C));
    KvState* const S = ctx_kv(C);
    KvRows a{};
    a.c = view(cache);
    a.slots = slots;
    a.n = (unsigned)n_tokens * (unsigned)cache->n_kv_heads;
    a.by_head = FastDiv((uint32_t)cache->n_kv_heads);
    if (append) {
        a.k_in = k;
        a.v_in = v;
    } else {
        a.k_out = const_cast<void*>(k);
        a.v_out = const_cast<void*>(v);
    }
    a.kt = kt, a.kh = kh, a.vt = vt, a.vh = vh;
    a.bad = S->bad_dev;
    const int d = cache->head_dim;
    const double bytes = (double)a.n * 2 * d * (type_size(dtype) + 0.5625) + 4.0 * n_tokens;
    cudaStream_t s = (cudaStream_t)stream;
    Launch l(C, append ? K_KV_APPEND : K_KV_READ, bytes, 0, s);
    CUDA_TRY(append ? launch_kv_append(a, d, dtype, s) : launch_kv_read(a, d, dtype, s));
    return MOE_OK;
}

}  // namespace

extern "C" size_t moe_kv_cache_bytes(const moe_kv_cache* c) {
    if (!shape_ok(c)) return 0;
    return (size_t)c->n_pages * c->n_kv_heads * (c->page_tokens / kKvBlock) * kv_record_bytes(c->head_dim);
}

extern "C" moe_status moe_kv_append(moe_ctx* C, const moe_kv_cache* cache, const void* k, int64_t kt, int64_t kh,
                                    const void* v, int64_t vt, int64_t vh, moe_dtype dtype, const int32_t* slots,
                                    int32_t n_tokens, void* stream) {
    return rows_call("moe_kv_append", C, cache, k, kt, kh, v, vt, vh, dtype, slots, n_tokens, true, stream);
}

extern "C" moe_status moe_kv_read(moe_ctx* C, const moe_kv_cache* cache, const int32_t* slots, int32_t n_tokens,
                                  void* k, int64_t kt, int64_t kh, void* v, int64_t vt, int64_t vh, moe_dtype dtype,
                                  void* stream) {
    return rows_call("moe_kv_read", C, cache, k, kt, kh, v, vt, vh, dtype, slots, n_tokens, false, stream);
}

extern "C" moe_status moe_kv_attend(moe_ctx* C, const moe_kv_cache* cache, const moe_kv_attend_args* p,
                                    void* stream) {
    const char* who = "moe_kv_attend";
    if (!C || !p) return set_error(MOE_EINVAL, "%s: NULL argument", who);
    moe_status st = check_cache(who, cache);
    if (st != MOE_OK) return st;
    if (p->dtype != MOE_F16 && p->dtype != MOE_BF16)
        return set_error(MOE_EINVAL, "%s: dtype %d (MOE_F16 or MOE_BF16)", who, (int)p->dtype);
    if (p->batch < 0 || p->n_q < 0 || p->max_pages < 0 || p->max_q < 0 || p->max_len < 0 || p->window < 0 ||
        (p->causal != 0 && p->causal != 1) || !isfinite(p->scale))
        return set_error(MOE_EINVAL, "%s: batch, n_q, max_pages, max_q, max_len and window must not be negative, causal "
                         "0 or 1 and scale finite", who);
    if (p->n_heads < 1 || p->n_heads % cache->n_kv_heads)
        return set_error(MOE_EINVAL, "%s: n_heads = %d must be a multiple of n_kv_heads = %d", who, p->n_heads,
                         cache->n_kv_heads);
    // kernels count the keys of tiles past a sequence's end in 32 bits
    if ((int64_t)p->max_pages * cache->page_tokens >= ((int64_t)1 << 31) - 1024 ||
        (int64_t)p->n_q * p->n_heads >= (int64_t)1 << 31)
        return set_error(MOE_EINVAL, "%s: max_pages * page_tokens must be below 2^31 - 1024, n_q * n_heads below 2^31", who);
    if (p->n_q == 0) return MOE_OK;
    if (p->batch == 0) return set_error(MOE_EINVAL, "%s: n_q = %d rows of no sequence", who, p->n_q);
    if (!p->q_start && p->n_q % p->batch)
        return set_error(MOE_EINVAL, "%s: without q_start, n_q = %d must be a multiple of batch = %d", who, p->n_q,
                         p->batch);
    if (!p->q || !p->out || !p->kv_len || (p->max_pages && !p->page_table))
        return set_error(MOE_EINVAL, "%s: NULL argument", who);
    if (!rows_ok(p->q, p->q_token_stride, p->q_head_stride, p->dtype) ||
        !rows_ok(p->out, p->out_token_stride, p->out_head_stride, p->dtype))
        return set_error(MOE_EINVAL, "%s: rows of q and out must start on 16-byte boundaries", who);
    CUDA_TRY(cudaSetDevice(ctx_device(C)));
    std::lock_guard<std::mutex> lock(ctx_kv_mutex(C));
    KvState* const S = ctx_kv(C);
    KvAttend a{};
    a.c = view(cache);
    a.q = p->q;
    a.out = p->out;
    a.lse = p->lse;
    a.qt = p->q_token_stride, a.qh = p->q_head_stride, a.ot = p->out_token_stride, a.oh = p->out_head_stride;
    a.table = p->page_table;
    a.table_stride = p->page_table_stride;
    a.kv_len = p->kv_len;
    a.q_start = p->q_start;
    a.B = p->batch, a.n_q = p->n_q, a.Hq = p->n_heads, a.G = p->n_heads / cache->n_kv_heads, a.max_pages = p->max_pages;
    a.by_g = FastDiv((uint32_t)a.G);
    a.T = p->q_start ? 0 : p->n_q / p->batch;
    a.causal = p->causal;
    // a window no shorter than any sequence hides nothing
    a.window = (int64_t)p->window >= (int64_t)p->max_pages * cache->page_tokens ? 0 : p->window;
    a.scale_log2 = p->scale * 1.4426950408889634f;
    a.bad = S->bad_dev;
    a.err = S->bad_dev + 1;
    if (*(volatile unsigned*)(S->bad_host + 1)) return expired(S);
    if ((st = ensure_workspace(S, ctx_device(C), (cudaStream_t)stream)) != MOE_OK) return st;
    a.part = reinterpret_cast<float*>(S->ws + kJoinBytes);
    const int d = cache->head_dim;
    cudaStream_t s = (cudaStream_t)stream;
    const bool prompt = (int64_t)p->max_q * a.G > decode_cols(cache->head_dim);
    const int cap = p->max_pages * cache->page_tokens, most = p->max_len && p->max_len < cap ? p->max_len : cap;
    // few short segments are never cut between CTAs, however long they turn out: such a call leaves the workspace alone
    const int64_t seen = a.window ? std::min<int64_t>(most, (int64_t)a.window + p->max_q + kKvBlock) : most;
    const int64_t segs = ((int64_t)p->n_q * a.G / 8 + p->batch) * cache->n_kv_heads;
    const int64_t work = prompt ? kv_prompt_plan(a, d, p->max_q, most, S->sms) : 0;
    const bool shared = prompt ? a.splits > 1 : seen > (int64_t)decode_whole(d) * kKvBlock || segs > S->sms;
    a.min_units = shared ? decode_piece(d) : std::max(1, cap / kKvBlock);
    if (shared) a.join = reinterpret_cast<KvJoin*>(S->ws);
    bool capturing = true;
    if (shared && (st = workspace_begin(S, s, &capturing)) != MOE_OK) return st;
    const double len = most;
    Launch l(C, K_KV_ATTEND, len * p->batch * cache->n_kv_heads * d * 1.125 + 4.0 * p->n_q * p->n_heads * d,
             4.0 * p->n_q * len * p->n_heads * d, s);
    int launched = 1;
    const cudaError_t launch = prompt ? launch_kv_prompt(a, d, p->dtype, work, s, &launched)
                                      : launch_kv_attend(a, d, p->dtype, p->max_q * a.G, S->sms, s, &launched);
    for (; launched > 1; --launched) ctx_count_launch(C);  // the first is counted already
    st = workspace_end(S, s, capturing);  // the first of two launches may have gone out before an error
    CUDA_TRY(launch);
    return st;
}

extern "C" moe_status moe_kv_check(moe_ctx* C) {
    if (!C) return set_error(MOE_EINVAL, "moe_kv_check: ctx is NULL");
    std::lock_guard<std::mutex> lock(ctx_kv_mutex(C));
    KvState* const S = ctx_kv(C);
    if (*(volatile unsigned*)(S->bad_host + 1)) return expired(S);
    if (*(volatile unsigned*)S->bad_host) {
        *(volatile unsigned*)S->bad_host = 0;
        return set_error(MOE_EINVAL, "an earlier cache call met a slot or page id outside its cache");
    }
    return MOE_OK;
}
