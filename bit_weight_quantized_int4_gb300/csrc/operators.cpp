// operators.cpp -- C-ABI host layer of the operators around the linears: the paged 8-bit
// key/value cache, attention over it, log probabilities and their gradient.  Everything that
// the host can see is checked here before anything is enqueued; index arrays live on the
// device and are checked by the kernels.
#include <algorithm>

#include "handle.h"

using q4lin::DeviceGuard;
using q4lin::make_ctx;
using q4lin::mul_ok;
using q4lin::overlaps;

namespace {

// Query rows (tokens x heads) per key/value head up to which a sequence's attention goes
// through the kernel that splits the keys (us, 8 key/value heads of 128, split / prompts' kernel,
// bf16: one sequence of 8192 keys, 32 rows 27.9 / 28.7, 64 rows 42.2 / 29.5; of 65536, 32 rows
// 96 / 86, 64 rows 174 / 88; 8 sequences of 2000, 32 rows 34 / 47, 64 rows 44 / 49; 32 of 4000,
// 32 rows 112 / 149, 64 rows 181 / 147; fp32, 8 of 2000: 31 / 47 and 41 / 48).
constexpr int64_t kSplitRows = 48;

bool aligned(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }
bool known_dtype(int dtype) { return dtype >= Q4LIN_DTYPE_F32 && dtype <= Q4LIN_DTYPE_BF16; }
int64_t size_of(int dtype) { return dtype == Q4LIN_DTYPE_F32 ? 4 : 2; }

// Bytes from the first to past the last element of [n0, n1, n2] with strides s0, s1 and 1.
bool extent(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t size, int64_t* bytes) {
    int64_t a, b, c;
    if (s0 < 0 || s1 < 0 || !mul_ok(n0 - 1, s0, &a) || !mul_ok(n1 - 1, s1, &b) ||
        __builtin_add_overflow(a, b, &c) || __builtin_add_overflow(c, n2, &c))
        return false;
    return mul_ok(c, size, bytes);
}

struct CacheBytes {
    int64_t codes, scales, table;
    // Whether [p, p + bytes) touches the codes or the scales.
    bool overlap(const q4lin_kv_cache_t& c, const void* p, int64_t bytes) const {
        return overlaps(p, bytes, c.k_codes, codes) || overlaps(p, bytes, c.v_codes, codes) ||
               overlaps(p, bytes, c.k_scales, scales) || overlaps(p, bytes, c.v_scales, scales);
    }
};

q4lin_status_t check_cache(const q4lin_kv_cache_t* c, CacheBytes* n) {
    if (!c || c->num_pages < 1 || c->kv_heads < 1 || c->batch < 0 || c->pages_per_sequence < 1 ||
        c->table_stride < c->pages_per_sequence)
        return Q4LIN_ERR_INVALID_ARG;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64) return Q4LIN_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return Q4LIN_ERR_UNSUPPORTED;
    if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales || (c->batch > 0 && !c->page_table))
        return Q4LIN_ERR_INVALID_ARG;
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 4) ||
        !aligned(c->v_scales, 4) || !aligned(c->page_table, 4))
        return Q4LIN_ERR_INVALID_ARG;
    int64_t t;
    if (!mul_ok(c->num_pages, c->kv_heads, &t) || !mul_ok(t, 4, &n->scales) ||
        !mul_ok(t, c->page_size * c->head_dim, &n->codes) ||
        !mul_ok(c->batch, c->table_stride, &t) || !mul_ok(t, 4, &n->table))
        return Q4LIN_ERR_INVALID_ARG;
    if (overlaps(c->k_codes, n->codes, c->v_codes, n->codes) ||
        overlaps(c->k_scales, n->scales, c->v_scales, n->scales) ||
        overlaps(c->k_codes, n->codes, c->k_scales, n->scales) ||
        overlaps(c->k_codes, n->codes, c->v_scales, n->scales) ||
        overlaps(c->v_codes, n->codes, c->k_scales, n->scales) ||
        overlaps(c->v_codes, n->codes, c->v_scales, n->scales))
        return Q4LIN_ERR_INVALID_ARG;
    // Grid and index limits of the kernels: positions and page numbers are 32 bits.
    if (c->kv_heads > 65535 || n->scales / 4 > 0x7FFFFFFF || c->batch > 0x7FFFFFFF / 8 ||
        c->pages_per_sequence > (0x7FFFFFFF - 64) / c->page_size)
        return Q4LIN_ERR_TOO_LARGE;
    return Q4LIN_OK;
}

q4lin_status_t check_rope(const q4lin_rope_t& r, int64_t head_dim, int64_t* bytes) {
    *bytes = 0;
    if (!r.cos) return Q4LIN_OK;
    if (!r.sin || r.positions < 1 || r.rotated < 8 || r.rotated > head_dim || r.rotated % 8 != 0 ||
        (r.interleaved != 0 && r.interleaved != 1) || !aligned(r.cos, 4) || !aligned(r.sin, 4) ||
        !mul_ok(r.positions, r.rotated / 2 * 4, bytes))
        return Q4LIN_ERR_INVALID_ARG;
    return Q4LIN_OK;
}

q4lin_status_t finish(cudaError_t err) {
    if (err == cudaSuccess) err = cudaGetLastError();
    return err == cudaSuccess ? Q4LIN_OK : Q4LIN_ERR_CUDA;
}

}  // namespace

extern "C" {

q4lin_status_t q4lin_run_kv_append(q4lin_handle_t h, const q4lin_kv_cache_t* cache,
                                   const q4lin_kv_append_t* a, void* stream) {
    if (!h || !a) return Q4LIN_ERR_INVALID_ARG;
    CacheBytes n;
    q4lin_status_t st = check_cache(cache, &n);
    if (st != Q4LIN_OK) return st;
    if (!known_dtype(a->dtype) || a->tokens < 0) return Q4LIN_ERR_INVALID_ARG;
    int64_t kb, vb, rb;
    if ((st = check_rope(a->rope, cache->head_dim, &rb)) != Q4LIN_OK) return st;
    if (a->tokens == 0 || cache->batch == 0) return Q4LIN_OK;
    const int64_t size = size_of(a->dtype);
    if (!a->k || !a->v || !a->offsets || !a->starts || !aligned(a->k, size) || !aligned(a->v, size) ||
        !aligned(a->offsets, 4) || !aligned(a->starts, 4))
        return Q4LIN_ERR_INVALID_ARG;
    if (!extent(a->tokens, a->k_token_stride, cache->kv_heads, a->k_head_stride, cache->head_dim, size, &kb) ||
        !extent(a->tokens, a->v_token_stride, cache->kv_heads, a->v_head_stride, cache->head_dim, size, &vb))
        return Q4LIN_ERR_INVALID_ARG;
    if (n.overlap(*cache, a->k, kb) || n.overlap(*cache, a->v, vb) ||
        n.overlap(*cache, a->offsets, (cache->batch + 1) * 4) ||
        n.overlap(*cache, a->starts, cache->batch * 4) ||
        n.overlap(*cache, cache->page_table, n.table) || n.overlap(*cache, a->rope.cos, rb) ||
        n.overlap(*cache, a->rope.sin, rb))
        return Q4LIN_ERR_INVALID_ARG;
    if (a->tokens > 0x7FFFFFFF) return Q4LIN_ERR_TOO_LARGE;
    DeviceGuard g(h->device);
    if (!g.ok()) return Q4LIN_ERR_CUDA;
    return finish(q4lin::kv_append_launch(*cache, *a, make_ctx(h, static_cast<cudaStream_t>(stream))));
}

q4lin_status_t q4lin_run_attention(q4lin_handle_t h, const q4lin_kv_cache_t* cache,
                                   const q4lin_attention_t* a, void* stream) {
    if (!h || !a) return Q4LIN_ERR_INVALID_ARG;
    CacheBytes n;
    q4lin_status_t st = check_cache(cache, &n);
    if (st != Q4LIN_OK) return st;
    if (!known_dtype(a->dtype) || a->tokens < 0 || a->heads < 1 || a->heads % cache->kv_heads != 0 ||
        a->window < 0 || (a->causal != 0 && a->causal != 1))
        return Q4LIN_ERR_INVALID_ARG;
    int64_t qb, ob, lb, rb, t;
    if ((st = check_rope(a->rope, cache->head_dim, &rb)) != Q4LIN_OK) return st;
    if (a->tokens == 0 || cache->batch == 0) return Q4LIN_OK;
    const int64_t size = size_of(a->dtype), D = cache->head_dim;
    // out is written 16 bytes at a time.
    if (a->max_query < 1 || !a->query || !a->out || !a->offsets || !a->lengths || !aligned(a->query, size) ||
        !aligned(a->out, 16) || !aligned(a->lse, 4) || !aligned(a->offsets, 4) || !aligned(a->lengths, 4))
        return Q4LIN_ERR_INVALID_ARG;
    if (!extent(a->tokens, a->q_token_stride, a->heads, a->q_head_stride, D, size, &qb) ||
        !mul_ok(a->tokens, a->heads, &t) || !mul_ok(t, D * size, &ob) || !mul_ok(t, a->lse ? 4 : 0, &lb))
        return Q4LIN_ERR_INVALID_ARG;
    const struct {
        const void* p;
        int64_t bytes;
    } inputs[] = {{a->query, qb},
                  {a->offsets, (cache->batch + 1) * 4},
                  {a->lengths, cache->batch * 4},
                  {cache->page_table, n.table},
                  {a->rope.cos, rb},
                  {a->rope.sin, rb}};
    for (const auto& in : inputs)
        if (overlaps(a->out, ob, in.p, in.bytes) || overlaps(a->lse, lb, in.p, in.bytes))
            return Q4LIN_ERR_INVALID_ARG;
    if (n.overlap(*cache, a->out, ob) || n.overlap(*cache, a->lse, lb) || overlaps(a->out, ob, a->lse, lb))
        return Q4LIN_ERR_INVALID_ARG;
    // The kernels count query rows in 32 bits, and the prompts' kernel keeps 32 bytes for each 256
    // rows of a key/value head in half of the workspace.
    constexpr int64_t kRowsMost = int64_t{1} << 27;
    static_assert(8 * (kRowsMost / 256) <= q4lin::kWsFloats / 3, "the pairs of row tiles fit");
    const int64_t group = a->heads / cache->kv_heads, max_query = std::min(a->max_query, a->tokens);
    int64_t rows_longest;
    if (t > 0x7FFFFFFF || t / cache->kv_heads > kRowsMost || !mul_ok(max_query, group, &rows_longest))
        return Q4LIN_ERR_TOO_LARGE;
    // One sequence of many rows goes to the prompts' kernel whatever its length; of several, each
    // kernel takes its own (lengths are on the device).
    const int64_t split_rows = h->attention_split_rows > 0 ? h->attention_split_rows : kSplitRows;
    const bool prompts = rows_longest > split_rows && q4lin::attention_prompt_eligible(*cache);
    const bool split = !prompts || cache->batch > 1;
    const int64_t split_most = prompts ? split_rows : INT64_MAX;
    q4lin_attention_t args = *a;
    args.max_query = max_query;
    // No sequence has more positions than its pages: a window of as many leaves every key.
    if (args.window >= cache->pages_per_sequence * cache->page_size) args.window = 0;
    if (split && !q4lin::attention_split_countable(*cache, args, split_most)) return Q4LIN_ERR_TOO_LARGE;
    DeviceGuard g(h->device);
    if (!g.ok()) return Q4LIN_ERR_CUDA;
    const q4lin::LaunchCtx c = make_ctx(h, static_cast<cudaStream_t>(stream));
    cudaError_t err = cudaSuccess;
    if (prompts) err = q4lin::attention_prompt_launch(*cache, args, split ? split_rows : 0, c);
    if (split && err == cudaSuccess) err = q4lin::attention_split_launch(*cache, args, split_most, c);
    return finish(err);
}

q4lin_status_t q4lin_run_logprobs(q4lin_handle_t h, const q4lin_logprobs_t* a, void* stream) {
    if (!h || !a) return Q4LIN_ERR_INVALID_ARG;
    if (!known_dtype(a->dtype) || a->rows < 0 || a->vocabulary < 1 || a->row_stride < 0 || a->top < 0 ||
        a->top > 32 || a->top > a->vocabulary)
        return Q4LIN_ERR_INVALID_ARG;
    if (a->rows == 0) return Q4LIN_OK;
    const int64_t size = size_of(a->dtype);
    if (!a->logits || !aligned(a->logits, size) || (a->top > 0 && (!a->top_tokens || !a->top_logprobs)) ||
        (a->tokens && !aligned(a->tokens, 4)))
        return Q4LIN_ERR_INVALID_ARG;
    int64_t xb, tb;
    if (!extent(a->rows, a->row_stride, 1, 0, a->vocabulary, size, &xb) || !mul_ok(a->rows, a->top * 4, &tb))
        return Q4LIN_ERR_INVALID_ARG;
    const int64_t rb = a->rows * 4;
    const struct {
        const void* p;
        int64_t bytes;
    } outs[] = {{a->logprob, rb},
                {a->entropy, rb},
                {a->lse, rb},
                {a->top > 0 ? a->top_tokens : nullptr, tb},
                {a->top > 0 ? a->top_logprobs : nullptr, tb}};
    for (const auto& o : outs) {
        if (!aligned(o.p, 4) || overlaps(o.p, o.bytes, a->logits, xb) || overlaps(o.p, o.bytes, a->tokens, rb))
            return Q4LIN_ERR_INVALID_ARG;
        for (const auto& other : outs)
            if (&other != &o && overlaps(o.p, o.bytes, other.p, other.bytes)) return Q4LIN_ERR_INVALID_ARG;
    }
    if (a->vocabulary > 0x7FFFFFFF || a->rows > 0x7FFFFFFF) return Q4LIN_ERR_TOO_LARGE;
    DeviceGuard g(h->device);
    if (!g.ok()) return Q4LIN_ERR_CUDA;
    return finish(q4lin::logprobs_launch(*a, make_ctx(h, static_cast<cudaStream_t>(stream))));
}

q4lin_status_t q4lin_run_logprobs_backward(q4lin_handle_t h, const q4lin_logprobs_backward_t* a,
                                           void* stream) {
    if (!h || !a) return Q4LIN_ERR_INVALID_ARG;
    if (!known_dtype(a->dtype) || a->rows < 0 || a->vocabulary < 1 || a->row_stride < 0 ||
        a->d_row_stride < a->vocabulary)
        return Q4LIN_ERR_INVALID_ARG;
    if (a->rows == 0) return Q4LIN_OK;
    const int64_t size = size_of(a->dtype);
    if (!a->logits || !a->d_logits || !a->lse || (a->d_logprob && !a->tokens) ||
        (a->d_entropy && !a->entropy) || !aligned(a->logits, size) || !aligned(a->d_logits, size))
        return Q4LIN_ERR_INVALID_ARG;
    int64_t xb, db;
    if (!extent(a->rows, a->row_stride, 1, 0, a->vocabulary, size, &xb) ||
        !extent(a->rows, a->d_row_stride, 1, 0, a->vocabulary, size, &db))
        return Q4LIN_ERR_INVALID_ARG;
    const bool in_place = a->d_logits == a->logits && a->d_row_stride == a->row_stride;
    if (!in_place && overlaps(a->d_logits, db, a->logits, xb)) return Q4LIN_ERR_INVALID_ARG;
    const int64_t rb = a->rows * 4;
    for (const void* p : {(const void*)a->tokens, (const void*)a->lse, (const void*)a->entropy,
                          (const void*)a->d_logprob, (const void*)a->d_entropy})
        if (!aligned(p, 4) || overlaps(a->d_logits, db, p, rb)) return Q4LIN_ERR_INVALID_ARG;
    if (a->vocabulary > 0x7FFFFFFF || a->rows > 0x7FFFFFFF / 64) return Q4LIN_ERR_TOO_LARGE;
    DeviceGuard g(h->device);
    if (!g.ok()) return Q4LIN_ERR_CUDA;
    return finish(q4lin::logprobs_backward_launch(*a, make_ctx(h, static_cast<cudaStream_t>(stream))));
}

}  // extern "C"
