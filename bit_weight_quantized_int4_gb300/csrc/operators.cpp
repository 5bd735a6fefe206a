// operators.cpp -- C-ABI host layer of the operators around the linears: the paged 8-bit and
// 4-bit key/value caches, attention over them, normalised and rotated queries and keys, log
// probabilities and their gradient.  Everything that
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
// Over a 4-bit cache the prompts' kernel is ahead earlier with bf16, whose products have one term
// each.  Kernel for few rows / for prompts, us, one sequence of 8192 keys, one of 65536, 8 of 2000, 32 of 4000:
//   bf16, 32 rows   heads of 64 21 / 25, 62 / 74, 30 / 44, 105 / 152   128 29 / 31, 97 / 89, 41 / 51, 175 / 183
//                   256 36 / 43, 148 / 139, 64 / 62, 294 / 285
//   bf16, 40 rows   64 31 / 26, 83 / 76, 44 / 46, 146 / 154   128 42 / 32, 129 / 90, 64 / 53, 238 / 187
//                   256 48 / 44, 179 / 140, 76 / 63, 366 / 284
//   fp16, 48 rows   64 32 / 29, 85 / 108, 46 / 53, 148 / 221   128 44 / 38, 131 / 146, 64 / 65, 245 / 283
//                   256 52 / 49, 210 / 217, 90 / 77, 422 / 401
//   fp16, 56 rows   64 30 / 29, 103 / 108, 42 / 54, 197 / 221   128 41 / 38, 161 / 147, 66 / 65, 317 / 284
//                   256 52 / 50, 240 / 217, 87 / 78, 488 / 401
//   fp32, 48 rows   64 30 / 31, 83 / 118, 44 / 56, 147 / 242   128 42 / 40, 128 / 157, 62 / 67, 243 / 312
//                   256 49 / 53, 206 / 234, 83 / 84, 416 / 494
constexpr int64_t kSplitRows4Bf16 = 32;

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

// bits: of a code. 8: one scale for a page and head, 4: one for each token of them.
q4lin_status_t check_cache(const q4lin_kv_cache_t* c, CacheBytes* n, int bits = 8) {
    if (!c || c->num_pages < 1 || c->kv_heads < 1 || c->batch < 0 || c->pages_per_sequence < 1 ||
        c->table_stride < c->pages_per_sequence)
        return Q4LIN_ERR_INVALID_ARG;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64) return Q4LIN_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return Q4LIN_ERR_UNSUPPORTED;
    if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales || (c->batch > 0 && !c->page_table))
        return Q4LIN_ERR_INVALID_ARG;
    const int64_t scale_bytes = bits == 8 ? 4 : 4 * c->page_size, scale_align = bits == 8 ? 4 : 16;
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, scale_align) ||
        !aligned(c->v_scales, scale_align) || !aligned(c->page_table, 4))
        return Q4LIN_ERR_INVALID_ARG;
    int64_t t, page_heads;
    if (!mul_ok(c->num_pages, c->kv_heads, &page_heads) || !mul_ok(page_heads, scale_bytes, &n->scales) ||
        !mul_ok(page_heads, c->page_size * c->head_dim * bits / 8, &n->codes) ||
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
    if (c->kv_heads > 65535 || page_heads > 0x7FFFFFFF || c->batch > 0x7FFFFFFF / 8 ||
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

// An append to a cache of `bits` bits, by `launch`.
template <typename Launch>
q4lin_status_t run_append(q4lin_handle_t h, const q4lin_kv_cache_t* cache, const q4lin_kv_append_t* a,
                          void* stream, int bits, Launch launch) {
    if (!h || !a) return Q4LIN_ERR_INVALID_ARG;
    CacheBytes n;
    q4lin_status_t st = check_cache(cache, &n, bits);
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
    return finish(launch(*cache, *a, make_ctx(h, static_cast<cudaStream_t>(stream))));
}

// Everything that the host can see of an attention's arguments; *idle: there is nothing to do.
q4lin_status_t check_attention(q4lin_handle_t h, const q4lin_kv_cache_t* cache, const q4lin_attention_t* a, int bits,
                               bool* idle) {
    *idle = false;
    if (!h || !a) return Q4LIN_ERR_INVALID_ARG;
    CacheBytes n;
    q4lin_status_t st = check_cache(cache, &n, bits);
    if (st != Q4LIN_OK) return st;
    if (!known_dtype(a->dtype) || a->tokens < 0 || a->heads < 1 || a->heads % cache->kv_heads != 0 ||
        a->window < 0 || (a->causal != 0 && a->causal != 1))
        return Q4LIN_ERR_INVALID_ARG;
    int64_t qb, ob, lb, rb, t;
    if ((st = check_rope(a->rope, cache->head_dim, &rb)) != Q4LIN_OK) return st;
    *idle = a->tokens == 0 || cache->batch == 0;
    if (*idle) return Q4LIN_OK;
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
    return Q4LIN_OK;
}

// [tokens, heads, head_dim] with contiguous channels, in bytes; strides of axes of length one (or
// none) are those of a contiguous array.
struct Rows {
    const void* p = nullptr;
    int64_t bytes = 0, token = 0, head = 0;
    int64_t span = 0;  // of one token's heads
    bool same(const Rows& o) const { return p == o.p && token == o.token && head == o.head; }
    // Whether no element lies in both: in ranges of their own, or in parts of their own of rows of
    // one length (slices of one array).
    bool apart(const Rows& o) const {
        if (!overlaps(p, bytes, o.p, o.bytes)) return true;
        if (token != o.token || span > token || o.span > token) return false;
        const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(o.p) - reinterpret_cast<uintptr_t>(p)) % token;
        const int64_t at = d < 0 ? d + token : d;
        return at >= span && at + o.span <= token;
    }
};
// False where pointer, strides or sizes are no array's.
bool rows_of(const void* p, int64_t tokens, int64_t token_stride, int64_t heads, int64_t head_stride, int64_t dim,
             int dtype, Rows* r) {
    *r = Rows();
    if (tokens == 0 || heads == 0) return true;
    const int64_t size = size_of(dtype);
    if (!p || !aligned(p, size)) return false;
    if (heads == 1) head_stride = dim;
    int64_t span;
    if (head_stride < 0 || !mul_ok(heads - 1, head_stride, &span) || __builtin_add_overflow(span, dim, &span)) return false;
    if (tokens == 1) token_stride = span;
    if (!extent(tokens, token_stride, heads, head_stride, dim, size, &r->bytes)) return false;
    if (!mul_ok(token_stride, size, &r->token) || !mul_ok(head_stride, size, &r->head)) return false;
    r->p = p, r->span = span * size;
    return true;
}
// Whether every element has a place of its own.
bool distinct(const Rows& r, int64_t tokens, int64_t heads, int64_t row) {
    if (!r.p) return true;
    if (r.head >= row && r.token >= r.span) return true;
    int64_t column;
    return r.token >= row && mul_ok(tokens - 1, r.token, &column) && r.head >= column + row;
}
// Whether `y` may be written while `x` is read row by row: it is x, or apart from it.
bool written_apart(const Rows& y, const Rows& x) { return y.same(x) || y.apart(x); }

struct NormRows {
    Rows x[2], y[2];  // queries, keys
    int64_t rope;
};
q4lin_status_t check_norm_rope(const q4lin_norm_rope_t& a, NormRows* n) {
    if (!known_dtype(a.dtype) || a.tokens < 0 || a.heads < 0 || a.kv_heads < 0 || a.heads + a.kv_heads < 1 ||
        !(a.eps >= 0.f) || a.eps > 3.4028235e38f)
        return Q4LIN_ERR_INVALID_ARG;
    if (a.head_dim != 64 && a.head_dim != 128 && a.head_dim != 256) return Q4LIN_ERR_UNSUPPORTED;
    const q4lin_status_t st = check_rope(a.rope, a.head_dim, &n->rope);
    if (st != Q4LIN_OK) return st;
    const int64_t D = a.head_dim, wb = D * 4, row = D * size_of(a.dtype);
    if (!aligned(a.q_weight, 4) || !aligned(a.k_weight, 4) || !aligned(a.positions, 4) ||
        !rows_of(a.q, a.tokens, a.q_token_stride, a.heads, a.q_head_stride, D, a.dtype, &n->x[0]) ||
        !rows_of(a.k, a.tokens, a.k_token_stride, a.kv_heads, a.k_head_stride, D, a.dtype, &n->x[1]) ||
        !rows_of(a.q_out, a.tokens, a.q_out_token_stride, a.heads, a.q_out_head_stride, D, a.dtype, &n->y[0]) ||
        !rows_of(a.k_out, a.tokens, a.k_out_token_stride, a.kv_heads, a.k_out_head_stride, D, a.dtype, &n->y[1]) ||
        !distinct(n->y[0], a.tokens, a.heads, row) || !distinct(n->y[1], a.tokens, a.kv_heads, row) ||
        (a.rope.cos && a.tokens > 0 && !a.positions))
        return Q4LIN_ERR_INVALID_ARG;
    int64_t pb;
    if (!mul_ok(a.tokens, 4, &pb)) return Q4LIN_ERR_INVALID_ARG;
    if (!n->y[0].apart(n->y[1]) || !n->y[0].apart(n->x[1]) || !n->y[1].apart(n->x[0])) return Q4LIN_ERR_INVALID_ARG;
    for (const Rows& y : n->y)
        if (overlaps(y.p, y.bytes, a.q_weight, wb) || overlaps(y.p, y.bytes, a.k_weight, wb) ||
            (a.rope.cos && (overlaps(y.p, y.bytes, a.positions, pb) || overlaps(y.p, y.bytes, a.rope.cos, n->rope) ||
                            overlaps(y.p, y.bytes, a.rope.sin, n->rope))))
            return Q4LIN_ERR_INVALID_ARG;
    // Heads and rows are counted in 64 bits; a token's heads in an int.
    if (a.heads > 0x7FFFFFF || a.kv_heads > 0x7FFFFFF || a.tokens > 0x7FFFFFFF) return Q4LIN_ERR_TOO_LARGE;
    return Q4LIN_OK;
}

// Attention over a cache of `bits` bits by its kernels.
template <typename Countable, typename Prompt, typename Split>
q4lin_status_t run_attention(q4lin_handle_t h, const q4lin_kv_cache_t* cache, const q4lin_attention_t* a, void* stream,
                             int bits, Countable countable, Prompt prompt_launch, Split split_launch) {
    bool idle;
    const q4lin_status_t st = check_attention(h, cache, a, bits, &idle);
    if (st != Q4LIN_OK || idle) return st;
    const int64_t t = a->tokens * a->heads;
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
    const int64_t by_rule = bits == 4 && a->dtype == Q4LIN_DTYPE_BF16 ? kSplitRows4Bf16 : kSplitRows;
    const int64_t split_rows = h->attention_split_rows > 0 ? h->attention_split_rows : by_rule;
    // (Heads of 256 have a record for each 128 rows: where those would not fit, the other kernel takes all.)
    const bool eligible = bits == 4 ? cache->head_dim <= 128 || t / cache->kv_heads <= kRowsMost / 2
                                    : q4lin::attention_prompt_eligible(*cache);
    const bool prompts = rows_longest > split_rows && eligible;
    const bool split = !prompts || cache->batch > 1;
    const int64_t split_most = prompts ? split_rows : INT64_MAX;
    q4lin_attention_t args = *a;
    args.max_query = max_query;
    // No sequence has more positions than its pages: a window of as many leaves every key.
    if (args.window >= cache->pages_per_sequence * cache->page_size) args.window = 0;
    if (split && !countable(*cache, args, split_most)) return Q4LIN_ERR_TOO_LARGE;
    DeviceGuard g(h->device);
    if (!g.ok()) return Q4LIN_ERR_CUDA;
    const q4lin::LaunchCtx c = make_ctx(h, static_cast<cudaStream_t>(stream));
    cudaError_t err = cudaSuccess;
    if (prompts) err = prompt_launch(*cache, args, split ? split_rows : 0, c);
    if (split && err == cudaSuccess) err = split_launch(*cache, args, split_most, c);
    return finish(err);
}

}  // namespace

extern "C" {

q4lin_status_t q4lin_run_kv_append(q4lin_handle_t h, const q4lin_kv_cache_t* cache,
                                   const q4lin_kv_append_t* a, void* stream) {
    return run_append(h, cache, a, stream, 8, q4lin::kv_append_launch);
}

q4lin_status_t q4lin_run_attention(q4lin_handle_t h, const q4lin_kv_cache_t* cache,
                                   const q4lin_attention_t* a, void* stream) {
    return run_attention(h, cache, a, stream, 8, q4lin::attention_split_countable, q4lin::attention_prompt_launch,
                         q4lin::attention_split_launch);
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

q4lin_status_t q4lin_run_kv4_append(q4lin_handle_t h, const q4lin_kv4_cache_t* cache,
                                    const q4lin_kv_append_t* a, void* stream) {
    return run_append(h, cache, a, stream, 4, q4lin::kv4_append_launch);
}

q4lin_status_t q4lin_run_kv4_read(q4lin_handle_t h, const q4lin_kv4_cache_t* cache, const q4lin_kv_read_t* a,
                                  void* stream) {
    if (!h || !a) return Q4LIN_ERR_INVALID_ARG;
    CacheBytes n;
    q4lin_status_t st = check_cache(cache, &n, 4);
    if (st != Q4LIN_OK) return st;
    if (!known_dtype(a->dtype) || a->tokens < 0) return Q4LIN_ERR_INVALID_ARG;
    if (a->tokens == 0 || cache->batch == 0) return Q4LIN_OK;
    int64_t ob;
    if ((!a->k && !a->v) || !a->offsets || !a->starts || !aligned(a->k, 16) || !aligned(a->v, 16) ||
        !aligned(a->offsets, 4) || !aligned(a->starts, 4) ||
        !mul_ok(a->tokens, cache->kv_heads * cache->head_dim * size_of(a->dtype), &ob))
        return Q4LIN_ERR_INVALID_ARG;
    for (const void* out : {a->k, a->v})
        if (n.overlap(*cache, out, ob) || overlaps(out, ob, cache->page_table, n.table) ||
            overlaps(out, ob, a->offsets, (cache->batch + 1) * 4) || overlaps(out, ob, a->starts, cache->batch * 4))
            return Q4LIN_ERR_INVALID_ARG;
    if (overlaps(a->k, ob, a->v, ob)) return Q4LIN_ERR_INVALID_ARG;
    if (a->tokens > 0x7FFFFFFF) return Q4LIN_ERR_TOO_LARGE;
    DeviceGuard g(h->device);
    if (!g.ok()) return Q4LIN_ERR_CUDA;
    return finish(q4lin::kv4_read_launch(*cache, *a, make_ctx(h, static_cast<cudaStream_t>(stream))));
}

q4lin_status_t q4lin_run_kv4_attention(q4lin_handle_t h, const q4lin_kv4_cache_t* cache,
                                       const q4lin_attention_t* a, void* stream) {
    return run_attention(h, cache, a, stream, 4, q4lin::kv4_attention_split_countable,
                         q4lin::kv4_attention_prompt_launch, q4lin::kv4_attention_split_launch);
}

q4lin_status_t q4lin_run_norm_rope(q4lin_handle_t h, const q4lin_norm_rope_t* a, void* stream) {
    if (!h || !a) return Q4LIN_ERR_INVALID_ARG;
    NormRows n;
    const q4lin_status_t st = check_norm_rope(*a, &n);
    if (st != Q4LIN_OK || a->tokens == 0) return st;
    if (!written_apart(n.y[0], n.x[0]) || !written_apart(n.y[1], n.x[1])) return Q4LIN_ERR_INVALID_ARG;
    DeviceGuard g(h->device);
    if (!g.ok()) return Q4LIN_ERR_CUDA;
    return finish(q4lin::norm_rope_launch(*a, make_ctx(h, static_cast<cudaStream_t>(stream))));
}

q4lin_status_t q4lin_run_norm_rope_backward(q4lin_handle_t h, const q4lin_norm_rope_backward_t* b, void* stream) {
    if (!h || !b) return Q4LIN_ERR_INVALID_ARG;
    const q4lin_norm_rope_t& a = b->forward;
    NormRows n;
    q4lin_status_t st = check_norm_rope(a, &n);
    if (st != Q4LIN_OK) return st;
    if (!aligned(b->d_q_weight, 4) || !aligned(b->d_k_weight, 4)) return Q4LIN_ERR_INVALID_ARG;
    const int64_t wb = a.head_dim * 4;
    Rows d[2];
    if (!rows_of(b->d_q_out, a.tokens, b->d_q_out_token_stride, a.heads, b->d_q_out_head_stride, a.head_dim, a.dtype, &d[0]) ||
        !rows_of(b->d_k_out, a.tokens, b->d_k_out_token_stride, a.kv_heads, b->d_k_out_head_stride, a.head_dim, a.dtype, &d[1]) ||
        overlaps(b->d_q_weight, wb, b->d_k_weight, wb))
        return Q4LIN_ERR_INVALID_ARG;
    for (int i = 0; i < 2; ++i) {
        if (!written_apart(n.y[i], n.x[i]) || !written_apart(n.y[i], d[i]) || !n.y[i].apart(d[1 - i]))
            return Q4LIN_ERR_INVALID_ARG;
        float* dw = i ? b->d_k_weight : b->d_q_weight;
        for (const Rows* r : {&n.x[0], &n.x[1], &n.y[0], &n.y[1], &d[0], &d[1]})
            if (overlaps(dw, wb, r->p, r->bytes)) return Q4LIN_ERR_INVALID_ARG;
        if (overlaps(dw, wb, a.q_weight, wb) || overlaps(dw, wb, a.k_weight, wb) ||
            (a.rope.cos && (overlaps(dw, wb, a.positions, a.tokens * 4) || overlaps(dw, wb, a.rope.cos, n.rope) ||
                            overlaps(dw, wb, a.rope.sin, n.rope))))
            return Q4LIN_ERR_INVALID_ARG;
    }
    DeviceGuard g(h->device);
    if (!g.ok()) return Q4LIN_ERR_CUDA;
    const q4lin::LaunchCtx c = make_ctx(h, static_cast<cudaStream_t>(stream));
    if (a.tokens > 0) return finish(q4lin::norm_rope_backward_launch(*b, c));
    cudaError_t e = cudaSuccess;
    if (b->d_q_weight) e = cudaMemsetAsync(b->d_q_weight, 0, wb, c.stream);
    if (b->d_k_weight && e == cudaSuccess) e = cudaMemsetAsync(b->d_k_weight, 0, wb, c.stream);
    return finish(e);
}

}  // extern "C"
