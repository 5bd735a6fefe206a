/*
 * q4lin.h -- C ABI of the GB300 (sm_103a) 4-bit group-symmetric weight-quantized linear.
 *
 *   out[m,n] = bias[n] + sum_k x[m,k] * (nib(W)[n,k] - 8) * scale[k / group_size, n]
 *
 * Sources of the operation ("[ExecuTorch][WebGPU] ..." pull-request pages):
 *   - "Add linear_qcs4w op (et_vk.linear_qcs4w)", Solution and Constraints (2)-(4): the
 *     per-term formula in[m,k] * (unpack_int4(w) - 8) * scale, the grouped scale index
 *     (k / group_size) * N + n, the +8-shifted signed int4, the packed [N, K/2] uint8
 *     weight whose LOW nibble holds the even k (the q4gsw packer's "(odd << 4) | even"),
 *     the per-output-channel case (one scale per n, i.e. group_size = K), and the
 *     fail-loud argument guards (K_packed == ceil(K/2), enough scales).
 *   - "Add fp32 matmul ops ... (linear_q4gsw_backward)", #20943: dequant = (code - 8) *
 *     scale with [num_groups, N] scales; the K == 0 guard of the sibling ops.
 *   - "Add optimized linear_fp32 op", Implementation: the optional bias (a dummy binding
 *     when absent) added once in the epilogue, v = v + bias[n].
 *   - "Add 256-thread steel q4gsw prefill GEMM", Solution/Implementation: M = 1 routes to
 *     a GEMV, M > 1 to GEMM kernels chosen by a fail-closed eligibility check.
 *
 * Conventions for every entry point:
 *   - Every buffer is owned by the caller.  q4lin_run allocates nothing, never
 *     synchronizes the device and only enqueues kernels on the given stream.  A handle
 *     owns its options, a 4-byte device status word and 64 MiB of device scratch plus
 *     64 KiB of counters (partial sums of launches that split K or the rows across CTAs:
 *     decode GEMV, tensor-core GEMM, small-M tensor-core GEMM, input gradient, attention,
 *     log probabilities; the fp16 copy of x of the fp16 tensor-core path), all allocated
 *     by q4lin_create.
 *   - Status codes, never exceptions, aborts or prints.  Arguments are validated before
 *     any launch: a non-OK status from validation means nothing was enqueued.
 *   - All device pointers must be device-accessible memory of the handle's device.
 *   - The handle's scratch is shared by its calls: calls on one handle must be ordered on
 *     the GPU (one stream, or streams ordered by events).  Use one handle per stream for
 *     calls that run concurrently.  q4lin_set_option must not race with q4lin_run on the
 *     same handle.
 */
#ifndef Q4LIN_H
#define Q4LIN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define Q4LIN_API __attribute__((visibility("default")))
#else
#define Q4LIN_API
#endif

typedef struct q4lin_handle* q4lin_handle_t;

typedef enum {
    Q4LIN_OK = 0,
    Q4LIN_ERR_INVALID_ARG = 1, /* bad pointer, size, alignment, overlap or option     */
    Q4LIN_ERR_UNSUPPORTED = 2, /* device is not sm_103, or a forced path cannot run   */
    Q4LIN_ERR_CUDA = 3,        /* a CUDA runtime call or launch failed                 */
    Q4LIN_ERR_TIMEOUT = 4,     /* a bounded device-side wait gave up (see status word) */
    Q4LIN_ERR_NO_DEVICE = 5,   /* no CUDA device with that ordinal                     */
    Q4LIN_ERR_TOO_LARGE = 6    /* exceeds a fixed capacity (q4lin_run_static_scratch),
                                  or what the operators around the linears can index   */
} q4lin_status_t;

/* Element type of the scales array. */
typedef enum { Q4LIN_SCALE_F32 = 0, Q4LIN_SCALE_F16 = 1 } q4lin_scale_dtype_t;

/* Kernel families.  AUTO picks by M and shape (measured crossover); the others force. */
typedef enum {
    Q4LIN_PATH_AUTO = 0,
    Q4LIN_PATH_GEMV = 1,    /* CUDA-core GEMV family: TMA-fed decode GEMV (M = 1),
                               TMA-fed multi-row GEMV (2 <= M <= 4, >= 10 M weights),
                               else the row-streaming kernel (small M)                */
    Q4LIN_PATH_FFMA = 2,    /* generic CUDA-core kernel: any K, group size, alignment  */
    Q4LIN_PATH_TC = 3,      /* tcgen05 tensor-core GEMM (TMEM accumulators)            */
    Q4LIN_PATH_TC_SMALL = 4 /* tcgen05 GEMM for 2 <= M <= 32 activation rows: persistent
                               CTAs over 128-row weight blocks, each weight read once,
                               x resident in shared memory or streamed for long K
                               (K % 32 == 0, 16-byte aligned x and qweight; grouped
                               scales: a power-of-two multiple of 32 as group size and a
                               scale row of whole 16-byte units); on fewer blocks
                               than half the SMs it splits K and adds the parts
                               through the handle's workspace (deterministic order);
                               tensor-core tolerance.  AUTO takes it for 3..32 rows
                               where it measured fastest (large matrices, and with
                               the K split most smaller ones from 5 rows) */
} q4lin_path_t;

/* Options for q4lin_set_option / q4lin_get_option. */
typedef enum {
    /* q4lin_path_t; default AUTO.  A forced path that cannot run the shape makes
     * q4lin_run return Q4LIN_ERR_UNSUPPORTED. */
    Q4LIN_OPT_FORCE_PATH = 1,
    /* 0 (default): the low nibble of byte j holds k = 2j (the q4gsw packer).
     * 1: the high nibble holds k = 2j (the qcs4w AOT packer's "(even << 4) | odd"
     * order, "Add linear_qcs4w op", Constraints (2)). */
    Q4LIN_OPT_NIBBLE_EVEN_HIGH = 2,
    /* Time limit, in nanoseconds of the GPU's global timer, of every bounded
     * device-side wait (mbarrier polls) of the TMA-fed kernels (decode and multi-row
     * GEMV, tensor-core GEMM, input gradient, attention); <= 0 restores the default
     * (2 s).  When a wait runs out the kernel records code 1 in the handle's status word, stops issuing
     * work, lets its own copies (and MMAs) in flight finish, frees its tensor memory and
     * returns; its output is then undefined. */
    Q4LIN_OPT_WAIT_LIMIT = 3,
    /* 1: launch with programmatic dependent launch, so a kernel may start streaming
     * its weights while the previous kernel on the stream drains (default 0).  The
     * preceding kernel must not write this call's qweight or scales.  This is the linears'
     * option.  Of the operators around them the norms, their gradient, the 4-bit cache's
     * append and read and its attention of few query rows may always begin while the previous
     * kernel drains, whatever it says: they wait for that kernel's end on the device before
     * they touch memory, and let the next one begin no sooner than after that wait.  The
     * others start when the previous call has ended. */
    Q4LIN_OPT_PDL = 4,
    /* Test hook, default 0.  1: the tensor-core kernel's copy engine skips the first
     * pipeline stage, the multi-row GEMV's copy engine issues nothing, and the attention
     * kernels' barriers expect keys that do not come, so the barrier their consumers wait
     * on is never completed and their bounded waits run out (exercises the timeout path
     * without faulting the GPU). */
    Q4LIN_OPT_TC_SKIP_FIRST_COPY = 5,
    /* 1: the tensor-core GEMM multiplies fp16 operands (x and the dequantized weights
     * (code - 8) * scale rounded to IEEE binary16, fp32 accumulation: tcgen05.mma
     * kind::f16, twice the tf32 rate) instead of tf32 (default 0).  Each product carries a
     * relative error below 2^-10, inside the tensor-core path's 4e-3 * sum|x*w| bar.
     * Values outside the fp16 range (|x| >= 65520, or a scale with |scale| > 8188) make
     * the call record code 2 in the status word; its output is then undefined.  x is
     * first converted into the handle's scratch (M * K * 2 bytes); a problem whose copy
     * does not fit there runs in tf32. */
    Q4LIN_OPT_TC_F16 = 6,
    /* Operands of the small-M tensor-core GEMM (Q4LIN_PATH_TC_SMALL).  Up to 8 rows, with
     * x resident in shared memory, K > 256 and room for an even weight ring of >= 4 stages,
     * it can multiply bf16 operands: the dequantized weights rounded to bf16, and x as the
     * two bf16 terms bf16(x) and bf16(x - bf16(x)), taken by the same MMA as extra columns;
     * each product then carries a relative error below 2^-9 + 2^-16, inside the tensor-core
     * path's 4e-3 * sum|x*w| bar, and bf16 keeps fp32's exponent range.  0 (default): bf16
     * where it applies and the matrix has >= 100 blocks of 128 rows (measured faster there),
     * else tf32; 1: tf32 always; 2: bf16 wherever it applies. */
    Q4LIN_OPT_TC_SMALL_OPERANDS = 7,
    /* Query rows (tokens x heads of one key/value head) up to which a sequence's attention
     * goes through the kernel that splits the keys over the SMs; longer ones go through the
     * prompts' tcgen05 kernel (head_dim 64 and 128).  0 (default): the measured crossover. */
    Q4LIN_OPT_ATTENTION_SPLIT_ROWS = 8
} q4lin_option_t;

/* Create a handle for CUDA device `device`.  Queries the SM count and shared-memory
 * limit and allocates the 4-byte device status word and the handle's scratch.  Q4LIN_ERR_NO_DEVICE if the
 * ordinal does not exist, Q4LIN_ERR_UNSUPPORTED if it is not compute capability 10.3.
 * The caller's current device is left unchanged. */
Q4LIN_API q4lin_status_t q4lin_create(q4lin_handle_t* handle, int device);

/* Release the handle, its status word and its scratch.  NULL is accepted (no-op). */
Q4LIN_API q4lin_status_t q4lin_destroy(q4lin_handle_t handle);

/* out = x @ dequant(W)^T (+ bias), enqueued on `stream` (a cudaStream_t; NULL = the
 * legacy default stream).
 *
 *   x        float32 [M, K], row-major, contiguous, 4-byte aligned.
 *   qweight  uint8 [N, ceil(K/2)], row-major: byte (n, j) holds codes for k = 2j and
 *            k = 2j+1 (low/high nibble by default, see Q4LIN_OPT_NIBBLE_EVEN_HIGH);
 *            signed weight = code - 8.  For odd K the last high nibble is never read.
 *   scales   [ceil(K / group_size), N] row-major, float32 (scale_dtype 0, 4-byte
 *            aligned) or IEEE binary16 (scale_dtype 1, 2-byte aligned).  Per-channel
 *            (qcs4w) weights use group_size = K with a [1, N] (= [N]) array.
 *   bias     float32 [N], 4-byte aligned, or NULL for no bias.
 *   out      float32 [M, N], row-major, 4-byte aligned; must not overlap any input.
 *   M >= 0, N >= 0, K >= 1, group_size >= 1.  M == 0 or N == 0 returns Q4LIN_OK and
 *   launches nothing; K == 0 is Q4LIN_ERR_INVALID_ARG.
 * Any K, group size and alignment beyond the element alignment above is accepted;
 * shapes a fast kernel cannot take run on a slower one (never an error under AUTO).
 * Accumulation is fp32.  Q4LIN_ERR_CUDA reports a failed launch
 * (cudaGetLastError after enqueueing). */
Q4LIN_API q4lin_status_t q4lin_run(q4lin_handle_t handle, const float* x,
                                   const uint8_t* qweight, const void* scales,
                                   const float* bias, float* out, int64_t M, int64_t N,
                                   int64_t K, int64_t group_size, int scale_dtype,
                                   void* stream);

/* One problem of q4lin_run_grouped: the arguments of one q4lin_run call. */
typedef struct q4lin_problem {
    const float* x;
    const uint8_t* qweight;
    const void* scales;
    const float* bias; /* may be NULL */
    float* out;
    int64_t M, N, K, group_size;
    int scale_dtype;
} q4lin_problem_t;

/* Run `count` problems on `stream`; the result is that of calling q4lin_run on each in
 * order.  Consecutive M = 1 problems that read the same x with the same K, group size and
 * scale dtype (for example the q, k and v projections of a decoder layer, or its gate
 * and up projections) run as one launch, up to 4 per launch, when none of their outputs
 * overlaps another problem's buffers; everything else runs one call at a time.  This is
 * the fused decode launch that the pages' MLC fusion passes produce before the GEMV
 * schedule ("dlight.gpu.GEMV" notice: "fusion passes -> LowBatchGemvSpecialize").
 * Every problem is validated before anything is enqueued (same rules and status codes
 * as q4lin_run); `problems` is read during the call only.  count == 0 is Q4LIN_OK. */
Q4LIN_API q4lin_status_t q4lin_run_grouped(q4lin_handle_t handle,
                                           const q4lin_problem_t* problems, int count,
                                           void* stream);

/* Decode GEMV (M = 1) for callers that cannot allocate device memory.
 *
 * No counterpart on the pages: this entry point exists for callers that may not call
 * cudaMalloc -- code that runs while a stream is being captured into a CUDA graph in a
 * mode that forbids allocation, code inside a custom allocator or memory pool (where
 * allocating would recurse), and real-time paths where an allocation's latency or
 * failure is not allowed.  Such callers cannot create a handle (q4lin_create allocates),
 * so this call needs none: it runs the same decode GEMV as q4lin_run with M = 1, whose
 * split-K partial sums and counters live in a fixed array of about 537 KB that the
 * library reserves in the device code image; every GPU that loads the library holds it
 * until the process exits.  Nothing is allocated: no cudaMalloc, cudaFree or allocating
 * library routine.
 *
 *   Arguments as q4lin_run with M = 1 (x is [K], out is [N]); default nibble order, no
 *   PDL.  N must be at most 16384: larger N returns Q4LIN_ERR_TOO_LARGE and runs nothing.
 *   Shapes the TMA-fed GEMV cannot take (K % 32 != 0, K < 512, N < 32, x or qweight not
 *   16-byte aligned, group_size neither a multiple of 32 nor >= K) return
 *   Q4LIN_ERR_UNSUPPORTED.
 *   The first call on a device looks up the array's device address (once per device, on
 *   the current device); make that first call before any stream capture.  A device reset
 *   (cudaDeviceReset) destroys the array with the context: the next call on that device
 *   sees the new context and looks the address up again, so after a reset, too, make the
 *   first call before any capture.
 *   Every call shares the array and it keeps the last call's contents: each call clears
 *   the counters it needs (an asynchronous memset on `stream`) before its kernel.  Calls
 *   that overlap on the GPU race on the array: order them (one stream, or events).
 *   A bounded device-side wait that runs out is not reported by this entry point (the
 *   output is then undefined); the kernel still returns. */
Q4LIN_API q4lin_status_t q4lin_run_static_scratch(const float* x, const uint8_t* qweight,
                                                  const void* scales, const float* bias,
                                                  float* out, int64_t N, int64_t K,
                                                  int64_t group_size, int scale_dtype,
                                                  void* stream);

/* Input gradient of the linear on the same packed weights (the frozen 4-bit base of
 * adapter training):
 *
 *   d_x[m,k] = sum_n d_out[m,n] * (nib(W)[n,k] - 8) * scale[k / group_size, n]
 *
 * "[ExecuTorch][WebGPU] Add fp32 matmul ops ... (linear_q4gsw_backward)", #20943:
 * d_x[M,K] = d_out[M,N] @ dequant(W)[N,K], contracting over N, with the forward's weight
 * and scale layout.
 *   d_out   device fp32 [M, N] row-major (4-byte aligned)
 *   qweight, scales, K, group_size, scale_dtype: exactly as q4lin_run (the handle's
 *           Q4LIN_OPT_NIBBLE_EVEN_HIGH applies)
 *   d_x     device fp32 [M, K] row-major (4-byte aligned); must not overlap any input
 * Summation order over n is not specified (fp32 accumulation; results within
 * 1e-5 * sum_n |d_out * w| + 1e-7 of the fp64 definition), but it is fixed for a given
 * shape: repeated calls give identical bits.  M == 0 is Q4LIN_OK (nothing runs); N == 0
 * writes zeros to d_x.  Uses the handle's workspace when the rows are split over CTAs
 * (calls on one handle must be ordered on the GPU).  Validated before anything is
 * enqueued; same status codes as q4lin_run. */
Q4LIN_API q4lin_status_t q4lin_run_backward_dx(q4lin_handle_t handle, const float* d_out,
                                               const uint8_t* qweight, const void* scales,
                                               float* d_x, int64_t M, int64_t N, int64_t K,
                                               int64_t group_size, int scale_dtype,
                                               void* stream);

/* Straight-through re-quantisation of fp32 latent weights to packed 4-bit codes with
 * frozen scales, in the layout q4lin_run reads:
 *
 *   code[n,k] = clamp(round(latent[n,k] / scale[k / group_size, n]), -8, 7) + 8
 *
 * "[ExecuTorch][WebGPU] Add fp32 matmul ops ... (q4gsw_requant)", #20945: a zero scale
 * gives code 8.  The quotient is the IEEE fp32 quotient, round() rounds half to even,
 * a NaN quotient gives code 8, and for odd K the padding nibble of each row's last byte
 * is 8.  Bit-exact (integer output).
 *   latent  device fp32 [N, K] row-major (4-byte aligned)
 *   scales  device fp32 or fp16 [ceil(K/group_size), N], as q4lin_run
 *   qweight device uint8 [N, ceil(K/2)] output (low nibble = even k, or swapped when the
 *           handle's Q4LIN_OPT_NIBBLE_EVEN_HIGH is set); must not overlap any input
 * N == 0 is Q4LIN_OK (nothing runs).  Validated before anything is enqueued. */
Q4LIN_API q4lin_status_t q4lin_run_requant(q4lin_handle_t handle, const float* latent,
                                           const void* scales, uint8_t* qweight, int64_t N,
                                           int64_t K, int64_t group_size, int scale_dtype,
                                           void* stream);

/* ------------------------------------------------------------------------------------
 * Operators around the linears: a paged 8-bit key/value cache, attention over it, and the
 * log probabilities of the vocabulary head's output with their gradient.
 *
 * Every index array (page table, offsets, starts, lengths, tokens) is read on the device
 * only.  An index that points outside its array (a page >= num_pages or < 0, a position
 * past the page table or the rotation table, offsets that decrease or pass `tokens`, a
 * token >= vocabulary) makes the kernel leave out what it would have touched and record
 * code 4 in the handle's status word; nothing out of range is read or written.
 *
 * Sizes whose rows, pages or positions the kernels cannot count (2^31 rows of queries or
 * logits, 2^27 query rows of one key/value head; for the attention of up to 256 sequences at
 * a time that do not go through the prompts' kernel, 2^31 tiles of 64 keys times query rows
 * in eights times key/value heads, by the width of the page table) return
 * Q4LIN_ERR_TOO_LARGE. */

/* Element type of keys, values, queries, attention outputs and logits. */
typedef enum { Q4LIN_DTYPE_F32 = 0, Q4LIN_DTYPE_F16 = 1, Q4LIN_DTYPE_BF16 = 2 } q4lin_dtype_t;

/* A key/value cache in pages of page_size tokens.  A code c (one byte) of page p and head h
 * stands for (c - 128) * scale[p, h], scale >= 0.
 *   k_codes   uint8 [num_pages, kv_heads, page_size, head_dim], 16-byte aligned
 *   v_codes   uint8 [num_pages, kv_heads, head_dim, page_size], 16-byte aligned (values
 *             are kept transposed within a page, so that both products of the attention
 *             read 16 consecutive bytes along the axis that they sum over)
 *   k_scales, v_scales  float32 [num_pages, kv_heads]
 *   page_table int32 [batch, table_stride]: entry (b, j) is the page of tokens
 *             [j * page_size, (j + 1) * page_size) of sequence b, j < pages_per_sequence.
 *             Entries past a sequence's length are not read (they may be -1), nor are
 *             those wholly before the window of an attention's queries.
 * page_size: 16, 32 or 64.  head_dim: 64, 128 or 256.  A page belongs to one sequence
 * while that sequence is appended to (full pages may be shared). */
typedef struct q4lin_kv_cache {
    uint8_t* k_codes;
    float* k_scales;
    uint8_t* v_codes;
    float* v_scales;
    const int32_t* page_table;
    int64_t num_pages, kv_heads, page_size, head_dim;
    int64_t batch, pages_per_sequence, table_stride;
} q4lin_kv_cache_t;

/* Position rotation of the first `rotated` channels (a multiple of 8, at most head_dim) of a
 * head; cos and sin are float32 [positions, rotated / 2], contiguous, indexed by the
 * token's position in its sequence.  With i < rotated / 2, the pair (a, b) of channels
 * (i, i + rotated / 2), or (2i, 2i + 1) when interleaved is 1, becomes
 * (a cos - b sin, b cos + a sin).  cos == NULL: no rotation. */
typedef struct q4lin_rope {
    const float* cos;
    const float* sin;
    int64_t positions, rotated;
    int interleaved;
} q4lin_rope_t;

typedef struct q4lin_kv_append {
    const void* k; /* [tokens, kv_heads, head_dim], channels contiguous */
    const void* v;
    int64_t k_token_stride, k_head_stride, v_token_stride, v_head_stride; /* elements */
    int dtype;              /* q4lin_dtype_t of k and v */
    int64_t tokens;         /* new tokens of all sequences */
    const int32_t* offsets; /* [batch + 1]: sequence b's are rows offsets[b] .. offsets[b+1] */
    const int32_t* starts;  /* [batch]: tokens that sequence b holds before the call */
    q4lin_rope_t rope;      /* of the keys */
} q4lin_kv_append_t;

/* Append keys (rotated on the way) and values to the cache.
 *
 * For each page that receives tokens and each head, with amax the largest finite |x| of
 * the new tokens in that page (keys after the rotation, in fp32) and s0 the page's scale
 * if it holds earlier tokens of the sequence, else 0:
 *   s    = max(s0, amax * fl(1/127))          (a scale below 2^-126 is 0)
 *   code = clamp(rint(x * fl(1/s)), -127, 127) + 128, or 128 when s is 0
 * and where s > s0 > 0 the page's earlier codes are rounded again,
 *   code = rint((code - 128) * fl(s0/s)) + 128.
 * rint rounds half to even, and every product, sum and quotient is rounded to fp32 once, in
 * the order written, so the bytes are determined by the inputs.  An infinity becomes 1 or
 * 255, a NaN 128, and either records code 3 in the status word.  The caller keeps the
 * lengths: sequence b holds starts[b] + offsets[b+1] - offsets[b] tokens afterwards.
 * k and v may be slices of one larger array (strides).  tokens == 0 or batch == 0 is
 * Q4LIN_OK (nothing runs).  No input may overlap the cache. */
Q4LIN_API q4lin_status_t q4lin_run_kv_append(q4lin_handle_t handle,
                                             const q4lin_kv_cache_t* cache,
                                             const q4lin_kv_append_t* args, void* stream);

typedef struct q4lin_attention {
    const void* query; /* [tokens, heads, head_dim], channels contiguous */
    int64_t q_token_stride, q_head_stride; /* elements */
    void* out;              /* [tokens, heads, head_dim], contiguous, of the query's type,
                               16-byte aligned */
    float* lse;             /* [tokens, heads], or NULL */
    int dtype;              /* q4lin_dtype_t of query and out */
    int64_t tokens, heads;  /* heads: a multiple of kv_heads */
    int64_t max_query;      /* no sequence has more query tokens than this (<= tokens) */
    const int32_t* offsets; /* [batch + 1], as in q4lin_kv_append_t */
    const int32_t* lengths; /* [batch]: tokens in the cache, those of the queries included */
    float scale;            /* of the scores, usually 1 / sqrt(head_dim) */
    int causal;             /* 1: a query sees keys up to its own position; 0: all of them */
    int64_t window;         /* > 0: only the last `window` of those (its own included); 0: off */
    q4lin_rope_t rope;      /* of the queries (the keys were rotated when appended) */
} q4lin_attention_t;

/* Attention of queries over the cache.  Query i of the t = offsets[b+1] - offsets[b] of
 * sequence b has position q = lengths[b] - t + i, and reads the keys j < lengths[b] with
 * j <= q (causal) and j > q - window (window > 0); head h reads key/value head
 * h / (heads / kv_heads):
 *   x_j = scale * sum_d q_d K[j,d],  out_d = sum_j e^(x_j) V[j,d] / sum_j e^(x_j),
 *   lse = ln sum_j e^(x_j).
 * A query that sees no key (an empty sequence; causal and a negative position) gets out = 0
 * and lse = -infinity; another one with a NaN or an infinity gets NaN.  Queries at negative
 * positions are not rotated.  Codes are exact in the tensor cores' fp16 operands; queries and
 * probabilities enter them as two fp16 terms (22 bits), and everything is summed in fp32.
 * Sequences with many query rows go through a tcgen05 kernel (whose bfloat16 outputs take
 * probabilities of one fp16 term, 11 bits; which reads values relative to the largest value
 * scale of the keys that its 256 rows read; and whose sums cut off what fp32 has no room for:
 * about 4e-6 of the outputs' norm for float32, 6e-5 for float16 and, at 131072 keys, 2e-4
 * for bfloat16), the others through one that splits the keys evenly over the SMs (partial
 * results joined in a fixed order through the handle's workspace), so a batch may mix
 * prompts and single tokens (Q4LIN_OPT_ATTENTION_SPLIT_ROWS).  The same call gives the same
 * bits; where a walk is cut goes by the whole call, so a sequence's last bits may differ with
 * the rest of its batch.  tokens == 0 or batch == 0 is Q4LIN_OK.  Sequences of more than
 * max_query tokens record code 4, and their outputs are not written; where offsets decrease,
 * other sequences' outputs may not be written either. */
Q4LIN_API q4lin_status_t q4lin_run_attention(q4lin_handle_t handle,
                                             const q4lin_kv_cache_t* cache,
                                             const q4lin_attention_t* args, void* stream);

typedef struct q4lin_logprobs {
    const void* logits; /* [rows, vocabulary], entries of a row contiguous */
    int64_t row_stride; /* elements */
    int dtype;          /* q4lin_dtype_t of the logits */
    int64_t rows, vocabulary;
    const int32_t* tokens; /* [rows]; -1: no token (its log probability is 0); may be NULL */
    float* logprob;        /* [rows], or NULL */
    float* entropy;        /* [rows], or NULL */
    float* lse;            /* [rows], or NULL */
    int64_t top;           /* alternatives, 0..32 and <= vocabulary */
    int32_t* top_tokens;   /* [rows, top] (NULL when top is 0) */
    float* top_logprobs;   /* [rows, top] (NULL when top is 0) */
} q4lin_logprobs_t;

/* Of each row x of logits, in one pass: lse = ln sum_v e^(x_v), logprob = x_token - lse,
 * entropy = -sum_v p_v ln p_v with p = e^(x - lse), and the `top` largest entries in
 * descending order (equal ones: lowest index first) with their log probabilities.
 * -infinity stands for an excluded entry (p = 0, no part in the entropy).  A row of
 * nothing else has lse = -infinity, logprob and top_logprobs -infinity and entropy 0.  A
 * row with a NaN has lse NaN, one with a +infinity and no NaN has lse +infinity; in both,
 * entropy, logprob and top_logprobs are NaN (but -infinity for an excluded entry where
 * there is no NaN).  The order of the top entries takes a NaN as the largest. */
Q4LIN_API q4lin_status_t q4lin_run_logprobs(q4lin_handle_t handle, const q4lin_logprobs_t* args,
                                            void* stream);

typedef struct q4lin_logprobs_backward {
    const void* logits; /* as in q4lin_logprobs_t */
    int64_t row_stride;
    int dtype;
    int64_t rows, vocabulary;
    const int32_t* tokens;  /* [rows], or NULL when d_logprob is NULL */
    const float* lse;       /* [rows], as q4lin_run_logprobs wrote it */
    const float* entropy;   /* [rows], ditto (may be NULL when d_entropy is NULL) */
    const float* d_logprob; /* [rows], or NULL for zeros */
    const float* d_entropy; /* [rows], or NULL for zeros */
    void* d_logits;         /* [rows, vocabulary], of the logits' type */
    int64_t d_row_stride;   /* elements */
} q4lin_logprobs_backward_t;

/* Gradient of q4lin_run_logprobs' logprob and entropy for the logits:
 *   d_x_v = d_logprob (1[v = token] - p_v) - d_entropy p_v (ln p_v + entropy).
 * Entries with p = 0 get 0 (beyond the token's term).  A row with token -1 has no logprob
 * term; a row whose lse is -infinity gets zeros.  d_logits may be the logits' own array
 * (same pointer and stride), else it must not overlap any input. */
Q4LIN_API q4lin_status_t q4lin_run_logprobs_backward(q4lin_handle_t handle,
                                                     const q4lin_logprobs_backward_t* args,
                                                     void* stream);

/* ------------------------------------------------------------------------------------
 * A decoder layer over a cache in 4 bits: queries and keys normalised per head and rotated,
 * keys and values quantised into the cache, read back, and attended to.  Index arrays are
 * read and checked on the device as above. */

/* Norm of each head of queries and keys, and the position rotation, in one pass:
 *   r = 1 / sqrt(sum_d x_d^2 / head_dim + eps),   y = rotation(x r w),
 * the rotation as in q4lin_rope_t, by the token's entry of `positions`.  Everything is fp32
 * up to the one rounding to the type.  Rows whose squares leave fp32's range are scaled by a
 * power of two first, so finite rows have finite results (but for zeros with eps 0, which are
 * NaN).  A NaN or an infinity stays in its row. */
typedef struct q4lin_norm_rope {
    const void* q; /* [tokens, heads, head_dim], channels contiguous */
    const void* k; /* [tokens, kv_heads, head_dim] */
    int64_t q_token_stride, q_head_stride, k_token_stride, k_head_stride; /* elements */
    const float* q_weight; /* [head_dim], or NULL for ones */
    const float* k_weight;
    void* q_out; /* as q and k; may be them (same pointer and strides) */
    void* k_out;
    int64_t q_out_token_stride, q_out_head_stride, k_out_token_stride, k_out_head_stride;
    int dtype;                      /* q4lin_dtype_t of all four */
    int64_t tokens, heads, kv_heads; /* either number of heads may be 0 */
    int64_t head_dim;               /* 64, 128 or 256 */
    const int32_t* positions;       /* [tokens]; not read without a rotation */
    q4lin_rope_t rope;
    float eps; /* finite, >= 0 */
} q4lin_norm_rope_t;

/* No two elements of an output may share memory, nor an output with an input or the other
 * output, but q_out with q and k_out with k.  A token whose position is outside the rotation
 * table records code 4 and its outputs are not written.  tokens == 0 is Q4LIN_OK. */
Q4LIN_API q4lin_status_t q4lin_run_norm_rope(q4lin_handle_t handle, const q4lin_norm_rope_t* args,
                                             void* stream);

typedef struct q4lin_norm_rope_backward {
    q4lin_norm_rope_t forward; /* its inputs; q_out, k_out and their strides are d_q and d_k, the
                                  gradients for q and k */
    const void* d_q_out; /* gradients for q_out and k_out, of the same shapes and type; any strides */
    const void* d_k_out; /* (0 for a gradient that is the same for all tokens or heads) */
    int64_t d_q_out_token_stride, d_q_out_head_stride, d_k_out_token_stride, d_k_out_head_stride;
    float* d_q_weight; /* [head_dim], or NULL */
    float* d_k_weight;
} q4lin_norm_rope_backward_t;

/* Gradients of q4lin_run_norm_rope.  With g the rotation undone on a row of d_q_out (d_k_out)
 * and u = x r:
 *   d_w = sum over tokens and heads of g u,   d_x = r (g w - u sum_d(g w u) / head_dim).
 * Sums are fp32 in a fixed order (the same call gives the same bits).  d_q may be q or
 * d_q_out (same pointer and strides), d_k may be k or d_k_out; no other memory may be shared.
 * A token whose position is outside the rotation table records code 4, has no part in d_w
 * and its d_q and d_k are not written.  tokens == 0 writes zeros to d_q_weight and
 * d_k_weight.  Uses the handle's workspace. */
Q4LIN_API q4lin_status_t q4lin_run_norm_rope_backward(q4lin_handle_t handle,
                                                      const q4lin_norm_rope_backward_t* args,
                                                      void* stream);

/* A key/value cache of 4-bit codes in pages of page_size tokens, with a scale for each token
 * and head.  The members of q4lin_kv_cache_t, which mean here:
 *   k_codes, v_codes    uint8 [num_pages, kv_heads, page_size, head_dim / 2], 16-byte aligned;
 *             the low four bits are the even channel's (as in packed weights), and a code c
 *             stands for (c - 8) * scale
 *   k_scales, v_scales  float32 [num_pages, kv_heads, page_size], 16-byte aligned, >= 0
 * page_table, page_size (16, 32 or 64) and head_dim (64, 128 or 256) as there.  Slots of a
 * page behind a sequence's length are never read as numbers: their codes and scales may be
 * anything. */
typedef q4lin_kv_cache_t q4lin_kv4_cache_t;

/* Append keys (rotated on the way, if args->rope says so) and values.  Of each new token and
 * head, with amax the largest finite |x| of its head_dim channels (keys after the rotation):
 *   s    = amax * fl(1/7.5)                            (a scale below 2^-126 is 0)
 *   code = clamp(rint(x * fl(1/s)), -8, 7) + 8, or 8 when s is 0.
 * All 16 codes are used and no finite x is further than about s / 2 from what its code stands
 * for.  Rounding as in q4lin_run_kv_append: the bytes are determined by the inputs.  An
 * infinity becomes code 15 or 0, a NaN 8, and either records code 3 in the status word.
 * Tokens that the cache held before are not touched.  The arguments, their checks and the
 * lengths as there. */
Q4LIN_API q4lin_status_t q4lin_run_kv4_append(q4lin_handle_t handle,
                                              const q4lin_kv4_cache_t* cache,
                                              const q4lin_kv_append_t* args, void* stream);

typedef struct q4lin_kv_read {
    void* k; /* [tokens, kv_heads, head_dim], contiguous, 16-byte aligned; or NULL */
    void* v;
    int dtype;              /* q4lin_dtype_t of k and v */
    int64_t tokens;         /* tokens read, of all sequences */
    const int32_t* offsets; /* [batch + 1]: sequence b's are rows offsets[b] .. offsets[b+1] */
    const int32_t* starts;  /* [batch]: the first token of sequence b that is read */
} q4lin_kv_read_t;

/* Read tokens back: (code - 8) * scale in fp32, rounded once to the type.  Token
 * starts[b] + i of sequence b becomes row offsets[b] + i; rows of no sequence are left as they
 * are.  A token without a page in the table records code 4 and its row is left as well.
 * tokens == 0 or batch == 0 is Q4LIN_OK.  No output may overlap an input or the other one. */
Q4LIN_API q4lin_status_t q4lin_run_kv4_read(q4lin_handle_t handle, const q4lin_kv4_cache_t* cache,
                                            const q4lin_kv_read_t* args, void* stream);

/* Attention over a 4-bit cache: as q4lin_run_attention in its arguments, checks, masks and
 * results.  Codes are exact in the tensor cores' fp16 operands here too; the keys' scales
 * multiply the scores and the values' scales the probabilities, in fp32, and these products
 * enter as two terms that leave 2^-22 of the largest one among keys that the row sees: neither
 * the scales of keys that it does not see nor those of values that are zero matter.  (In the
 * kernel for many query rows, down to 2^-80 of the largest value scale among the keys that its
 * 256 rows, 128 of heads of 256, read.)  One exception: where bfloat16 outputs come from that
 * kernel, probabilities take one term, 11 bits, and while those value scales are within 2^24 of
 * one another a value times its scale (over a power of two near the largest) is rounded to fp16
 * once, 11 bits too. */
Q4LIN_API q4lin_status_t q4lin_run_kv4_attention(q4lin_handle_t handle,
                                                 const q4lin_kv4_cache_t* cache,
                                                 const q4lin_attention_t* args, void* stream);

/* The path q4lin_run would take for these arguments (no launch, no device access);
 * *path_out receives a q4lin_path_t other than AUTO.  Same validation and status codes
 * as q4lin_run.  For M == 0 or N == 0, *path_out is Q4LIN_PATH_AUTO (nothing runs). */
Q4LIN_API q4lin_status_t q4lin_plan(q4lin_handle_t handle, const float* x,
                                    const uint8_t* qweight, const void* scales,
                                    const float* bias, const float* out, int64_t M,
                                    int64_t N, int64_t K, int64_t group_size,
                                    int scale_dtype, int* path_out);

/* Kernels behind the paths (what q4lin_plan_kernel reports). */
typedef enum {
    Q4LIN_KERNEL_NONE = 0,      /* M == 0 or N == 0: nothing runs                          */
    Q4LIN_KERNEL_GEMV_TMA = 1,  /* TMA-fed decode GEMV (M = 1)                             */
    Q4LIN_KERNEL_MULTIROW = 2,  /* TMA-fed multi-row GEMV (2 <= M <= 4)                    */
    Q4LIN_KERNEL_ROWSTREAM = 3, /* row-streaming CUDA-core kernel (small M)                */
    Q4LIN_KERNEL_GENERIC = 4,   /* generic CUDA-core kernel (any K, group size, alignment) */
    Q4LIN_KERNEL_TC = 5,        /* tcgen05 tensor-core GEMM, tf32 operands                 */
    Q4LIN_KERNEL_TC_F16 = 6,    /* the same with fp16 operands (Q4LIN_OPT_TC_F16)          */
    Q4LIN_KERNEL_GEMV_TMA_FIXED = 7, /* the decode GEMV with exact fixed-point arithmetic: x as
                                      * 32-bit fixed point per 32-k chunk, codes times x by
                                      * dp4a; chosen when its CTAs take >= 2 row blocks each */
    Q4LIN_KERNEL_TC_SMALL = 8,  /* tcgen05 GEMM for 2 <= M <= 32 (Q4LIN_PATH_TC_SMALL), tf32 */
    Q4LIN_KERNEL_TC_SMALL_BF16 = 9 /* the same with bf16 operands (up to 8 rows, see
                                    * Q4LIN_OPT_TC_SMALL_OPERANDS) */
} q4lin_kernel_t;

/* The kernel q4lin_run would launch for these arguments (no launch, no device access);
 * *kernel_out receives a q4lin_kernel_t.  Same arguments, validation and status codes as
 * q4lin_plan; for M == 0 or N == 0, *kernel_out is Q4LIN_KERNEL_NONE. */
Q4LIN_API q4lin_status_t q4lin_plan_kernel(q4lin_handle_t handle, const float* x,
                                           const uint8_t* qweight, const void* scales,
                                           const float* bias, const float* out, int64_t M,
                                           int64_t N, int64_t K, int64_t group_size,
                                           int scale_dtype, int* kernel_out);

/* Set / read one q4lin_option_t.  Q4LIN_ERR_INVALID_ARG for an unknown option or an
 * out-of-range value. */
Q4LIN_API q4lin_status_t q4lin_set_option(q4lin_handle_t handle, int option,
                                          int64_t value);
Q4LIN_API q4lin_status_t q4lin_get_option(q4lin_handle_t handle, int option,
                                          int64_t* value);

/* Read and clear the handle's device status word after synchronizing `stream`.
 * *code_out = 0 if no kernel recorded a problem since the last call; otherwise the
 * first recorded code (1 = a bounded device-side wait ran out; 2 = a value outside the
 * fp16 range on the fp16 tensor-core path; 3 = a non-finite key or value was appended to a
 * cache; 4 = an index outside its array, see the operators around the linears).
 * The word is shared by every call on the handle.
 * Returns Q4LIN_ERR_TIMEOUT when the code is non-zero, Q4LIN_OK otherwise. */
Q4LIN_API q4lin_status_t q4lin_check_device_status(q4lin_handle_t handle, void* stream,
                                                   int* code_out);

/* Static, never-NULL description of a status code. */
Q4LIN_API const char* q4lin_status_string(q4lin_status_t status);

#ifdef __cplusplus
}
#endif

#endif /* Q4LIN_H */
