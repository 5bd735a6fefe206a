// attention_split.cuh -- what the kernels that split keys evenly over the GPU's warps share
// (attention.cu for the 8-bit cache, kv4_attention.cu for the 4-bit one): the list of 64-key tiles
// of all sequences and heads, the pieces that a warp takes of it, and the kernel that joins the
// heads whose keys were cut.
#pragma once

#include <algorithm>

#include "q4lin_internal.h"
#include "serving.cuh"

namespace q4lin {
namespace {
using namespace ptx;
using namespace serving;

constexpr int kTile = 64;        // keys per tile
constexpr int kMaxBatch = 256;   // sequences per launch
constexpr float kShift = 14.f;   // probabilities are kept as 2^14 p: fp16's range downwards
// Undone before a logarithm, whose error grows with its distance from 0.
constexpr float kUnshift = 1.f / 16384.f;
constexpr int64_t kDrainNs = 4000000000LL;
constexpr uint32_t kTooMany = 0x7FFFFFFF;

struct SplitArgs {
    q4lin_kv_cache_t cache;
    q4lin_attention_t a;
    int page_shift;
    int64_t rows_max;
    int q_vec;
    int workers;    // warps of the launch
    float unshift;      // of the parts' sums of weights, before a logarithm
    int64_t join_each;  // tokens of a sequence that the joining kernel has CTAs for; 0: one for every token
    float* parts;   // [workers][2][R (D + 2)]: a warp's first and last piece, if unfinished
    int* list;      // [batch + 1]: the share, then where each sequence begins in the list
    int* status;
    int64_t wait_ns;
    uint32_t missing;  // test hook: bytes that the copies' barriers wait for in vain
};

// Per query row of a piece.
struct RowInfo {
    float factor;        // of the MMA's scores, without the keys' scale, in powers of two
    int limit, low;      // keys [low, limit] are seen
    int index;           // token * heads + head (below 2^31), or -1
};

struct Sequence {
    int tq, len, tile0, tiles, row_tiles;
};

// What one sequence asks of this kernel; nothing where its indices are bad or its rows are
// too many for it.  tq is -1 where its offsets decrease.
template <int R>
__device__ __forceinline__ Sequence sequence_of(const SplitArgs& g, int64_t b, bool* bad) {
    Sequence s;
    const int64_t o0 = __ldg(g.a.offsets + b), o1 = __ldg(g.a.offsets + b + 1);
    const int64_t group = g.a.heads / g.cache.kv_heads;
    s.len = __ldg(g.a.lengths + b);
    s.tq = (int)(o1 - o0);
    *bad = o0 < 0 || o1 < o0 || o1 > g.a.tokens || s.tq > g.a.max_query ||
           (int64_t)s.len > g.cache.pages_per_sequence << g.page_shift ||
           (g.a.rope.cos && s.len > g.a.rope.positions);
    if (o1 < o0)
        s.tq = -1;
    else if (*bad || s.tq * group > g.rows_max)
        s.tq = 0;
    if (s.len < 0) s.len = 0;
    const int64_t first = g.a.window > 0 ? (int64_t)s.len - s.tq - g.a.window + 1 : 0;
    s.tile0 = first > 0 ? (int)(first / kTile) : 0;
    s.tiles = max((s.len + kTile - 1) / kTile - s.tile0, 1);
    s.row_tiles = (int)((s.tq * group + R - 1) / R);
    return s;
}

// An unfinished piece: [R][D] sums, then R maxima and R sums of weights.
template <int D, int R>
__device__ __forceinline__ float* part_at(const SplitArgs& g, int worker, bool begins) {
    constexpr int kPart = R * (D + 2);
    return g.parts + ((int64_t)worker * 2 + begins) * kPart;
}

// Inclusive scan of the sequences' tiles by a CTA of W warps: prefix[b] is where sequence b begins
// in the list, and the result its length.  prefix[0] is 0 already.  Sums stop at kTooMany: the host
// has counted on offsets that rise, and where one decreases (which is reported) sequences may
// overlap and have more tiles than 32 bits hold.
template <int R, int W>
__device__ __forceinline__ uint32_t scan_tiles(const SplitArgs& g, int* prefix, uint32_t* sums) {
    constexpr int T = 32 * W;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int batch = (int)g.cache.batch, Hkv = (int)g.cache.kv_heads;
    uint32_t sum = 0;
    for (int b0 = 0; b0 < batch; b0 += T) {
        const int b = b0 + tid;
        uint32_t v = 0;
        if (b < batch) {
            bool bad;
            const Sequence s = sequence_of<R>(g, b, &bad);
            v = s.tq < 0 ? kTooMany : (uint32_t)(s.tiles * s.row_tiles * Hkv);
            if (bad && blockIdx.x == 0) atomicCAS(g.status, 0, kStatusIndex);
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t n = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v = min(v + n, kTooMany);
        }
        if (b0 > 0) __syncthreads();
        if (lane == 31) sums[warp] = v;
        __syncthreads();
        uint32_t before = sum;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            sum = min(sum + sums[w], kTooMany);
            if (w + 1 == warp) before = sum;
        }
        if (b < batch) prefix[b + 1] = (int)min(before + v, kTooMany);
    }
    __syncthreads();
    return sum;
}

// A warp's share of one head's keys: tiles [k0, k0 + n) of `tiles`, of row tile row0 / R of head h
// of sequence b.
struct Piece {
    int b, len, tq, h, row0, k0, n, tiles, tile0;
};
// The piece that begins at `pos` of the list and goes no further than `end`.
template <int R>
__device__ __forceinline__ Piece piece_of(const SplitArgs& g, const int* prefix, int pos, int end) {
    const int batch = (int)g.cache.batch;
    int lo = 0, hi = batch;  // prefix[lo] <= pos < prefix[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= pos)
            lo = mid;
        else
            hi = mid;
    }
    bool bad;
    const Sequence s = sequence_of<R>(g, lo, &bad);
    const int local = pos - prefix[lo], seg = local / s.tiles;
    Piece p;
    p.b = lo, p.len = s.len, p.tq = s.tq, p.tiles = s.tiles, p.tile0 = s.tile0;
    p.k0 = local - seg * s.tiles;
    p.h = seg / s.row_tiles, p.row0 = (seg - p.h * s.row_tiles) * R;
    p.n = min(s.tiles - p.k0, end - pos);
    return p;
}

// The rows of heads that were cut: one CTA per query row, its warps taking parts in turn.
template <int D, int R, int kJoinWarps, int kAhead>
__global__ void __launch_bounds__(32 * kJoinWarps) attention_join_kernel(const SplitArgs g) {
    constexpr int kVec = D == 256 ? 2 : 1;  // 16-byte units per lane
    __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
    __shared__ float4 s_o[kJoinWarps][D / 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t at_token = blockIdx.x / g.a.heads;
    const int head = (int)(blockIdx.x - at_token * g.a.heads);
    const int group = (int)(g.a.heads / g.cache.kv_heads), h = head / group;
    // (Offsets and lengths are the caller's inputs, not the first kernel's results.)
    int64_t b;
    if (g.join_each)
        b = at_token / g.join_each;
    else
        b = find_sequence(g.cache.batch, at_token, [&](int64_t i) { return (int64_t)__ldg(g.a.offsets + i); });
    bool bad;
    const Sequence s = sequence_of<R>(g, b, &bad);
    const int64_t o0 = __ldg(g.a.offsets + b), token = g.join_each ? o0 + at_token - b * g.join_each : at_token;
    griddep_wait();
    if (token < o0 || token >= o0 + s.tq) return;
    const int row = (int)(token - o0) * group + head - h * group, r = row % R;
    const int share = __ldcg(g.list), at = __ldcg(g.list + 1 + b) + (h * s.row_tiles + row / R) * s.tiles;
    const int c0 = at / share, c1 = (at + s.tiles - 1) / share;
    if (c0 == c1) return;
    float mx = -INFINITY, l = 0.f;
    float4 o[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v) o[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool on = lane < D / 4;
    for (int c = c0 + warp; c <= c1; c += kJoinWarps * kAhead) {
        float pm[kAhead], pl[kAhead];
        float4 po[kAhead][kVec];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int w = c + k * kJoinWarps;
            pm[k] = -INFINITY, pl[k] = 0.f;
            if (w <= c1) {
                const float* src = part_at<D, R>(g, w, w == c0);
                pm[k] = __ldcg(src + R * D + r), pl[k] = __ldcg(src + R * D + R + r);
#pragma unroll
                for (int v = 0; v < kVec; ++v)
                    if (on) po[k][v] = __ldcg(reinterpret_cast<const float4*>(src + r * D) + lane + 32 * v);
            }
        }
        float top = mx;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) top = fmaxf(top, pm[k]);
        const float from = top == -INFINITY ? 0.f : top, old = ex2(mx - from);
        l *= old, mx = top;
#pragma unroll
        for (int v = 0; v < kVec; ++v) o[v].x *= old, o[v].y *= old, o[v].z *= old, o[v].w *= old;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (c + k * kJoinWarps > c1) continue;
            const float w = ex2(pm[k] - from);
            l = fmaf(pl[k], w, l);
#pragma unroll
            for (int v = 0; v < kVec; ++v) {
                o[v].x = fmaf(po[k][v].x, w, o[v].x), o[v].y = fmaf(po[k][v].y, w, o[v].y);
                o[v].z = fmaf(po[k][v].z, w, o[v].z), o[v].w = fmaf(po[k][v].w, w, o[v].w);
            }
        }
    }
    if (lane == 0) s_m[warp] = mx, s_l[warp] = l;
#pragma unroll
    for (int v = 0; v < kVec; ++v)
        if (on) s_o[warp][lane + 32 * v] = o[v];
    __syncthreads();
    if (warp != 0 || !on) return;
    mx = -INFINITY, l = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) mx = fmaxf(mx, s_m[w]);
    const float from = mx == -INFINITY ? 0.f : mx;
    float f[kJoinWarps];
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) f[w] = ex2(s_m[w] - from), l = fmaf(s_l[w], f[w], l);
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const int64_t index = token * g.a.heads + head;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            const float4 p = s_o[w][lane + 32 * v];
            a.x = fmaf(p.x, f[w], a.x), a.y = fmaf(p.y, f[w], a.y);
            a.z = fmaf(p.z, f[w], a.z), a.w = fmaf(p.w, f[w], a.w);
        }
        const int d = (lane + 32 * v) * 4;
        if (g.a.dtype == Q4LIN_DTYPE_F32)
            *reinterpret_cast<float4*>(static_cast<float*>(g.a.out) + index * D + d) =
                make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
        else
            *reinterpret_cast<uint2*>(static_cast<unsigned short*>(g.a.out) + index * D + d) =
                make_uint2(to_16x2(a.x * inv, a.y * inv, g.a.dtype), to_16x2(a.z * inv, a.w * inv, g.a.dtype));
    }
    if (lane == 0 && g.a.lse) g.a.lse[index] = l != 0.f ? (from + lg2(l * g.unshift)) * kLn2 : -INFINITY;
}

// What a launch may have to do.
struct SplitSize {
    int rows;          // query rows of a row tile
    int64_t segments;  // row tiles of all key/value heads
    int64_t tiles;     // of keys, of each
};
// Row tiles of `least` rows, or twice, four times as many up to 16 (8 with 256 channels) where a
// sequence may have more.
inline SplitSize split_size(const q4lin_kv_cache_t& cache, const q4lin_attention_t& a, int64_t rows_max, int64_t batch,
                            int least) {
    const int64_t group = a.heads / cache.kv_heads, rows = std::min(rows_max, a.max_query * group);
    const int most = cache.head_dim == 256 ? 8 : 16;
    SplitSize s;
    s.rows = least;
    while (s.rows < most && s.rows < rows) s.rows *= 2;
    const int64_t R = s.rows;
    const int64_t row_tiles =
        std::min((a.tokens * group + R - 1) / R + batch, ((rows + R - 1) / R) * batch);
    s.segments = row_tiles * cache.kv_heads;
    s.tiles = (cache.pages_per_sequence * cache.page_size + kTile - 1) / kTile;
    return s;
}
// Whether a launch's list of tiles is short enough for 32 bits.
inline bool split_countable(const q4lin_kv_cache_t& cache, const q4lin_attention_t& a, int64_t rows_max, int least) {
    const SplitSize s = split_size(cache, a, rows_max, std::min<int64_t>(kMaxBatch, cache.batch), least);
    int64_t units;
    // (The kernel rounds the list up to its warps, of which there are fewer than 2^16.)
    return !__builtin_mul_overflow(s.segments, s.tiles, &units) && units <= 0x7FFFFFFF - 0xFFFF;
}

// The joining kernel, behind the one that left the parts.
template <int D, int R>
cudaError_t join_launch(SplitArgs& g, const SplitSize& size, const LaunchCtx& c) {
    // CTAs for the tokens that a sequence of this kernel may have, or for every token, whichever are
    // fewer (among 2403 tokens of three prompts, none of them this kernel's, 77000 idle CTAs took 140 us).
    const int64_t each = std::min(g.a.max_query, std::max<int64_t>(1, g.rows_max / (g.a.heads / g.cache.kv_heads)));
    g.join_each = each <= g.a.tokens / g.cache.batch ? each : 0;
    const int64_t rows = g.join_each ? each * g.cache.batch : g.a.tokens;
    // The second kernel's launch overlaps the first's work; it waits for its end on the device.
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    // Warps per row by the parts that a row may have (64 sequences x 8 heads on 1216 warps: 2 or 3
    // parts, two warps 3 us less for the whole call than four; 9 x 4 heads x 3 row tiles on 1064:
    // about 10, eight warps 21 us, two 24; one sequence x 8 heads: 152).
    const int64_t parts = g.workers / size.segments;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * g.a.heads));
    cfg.stream = c.stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (parts <= 4) {
        cfg.blockDim = dim3(64);
        return cudaLaunchKernelEx(&cfg, attention_join_kernel<D, R, 2, 4>, g);
    }
    if (parts <= 32) {
        cfg.blockDim = dim3(256);
        return cudaLaunchKernelEx(&cfg, attention_join_kernel<D, R, 8, 4>, g);
    }
    cfg.blockDim = dim3(512);
    return cudaLaunchKernelEx(&cfg, attention_join_kernel<D, R, 16, D == 256 ? 4 : 10>, g);
}

// run(arguments, size) for sequences in groups that a launch's list holds.
template <typename Run>
cudaError_t in_groups(const q4lin_kv_cache_t& cache, const q4lin_attention_t& a, int64_t rows_max, int least,
                      const LaunchCtx& c, Run run) {
    cudaError_t err = cudaSuccess;
    for (int64_t b = 0; b < cache.batch && err == cudaSuccess; b += kMaxBatch) {
        SplitArgs g;
        g.cache = cache;
        g.a = a;
        g.cache.batch = std::min<int64_t>(kMaxBatch, cache.batch - b);
        g.cache.page_table += b * cache.table_stride;
        g.a.offsets += b;
        g.a.lengths += b;
        g.page_shift = cache.page_size == 16 ? 4 : cache.page_size == 32 ? 5 : 6;
        g.rows_max = rows_max;
        g.unshift = kUnshift;
        g.q_vec = reinterpret_cast<uintptr_t>(a.query) % (4 * dtype_size(a.dtype)) == 0 &&
                  a.q_token_stride % 4 == 0 && a.q_head_stride % 4 == 0;
        g.status = c.status_word;
        g.wait_ns = c.wait_limit_ns;
        g.missing = c.tc_skip_first_copy ? 16 : 0;
        err = run(g, split_size(cache, a, rows_max, g.cache.batch, least));
    }
    return err;
}

}  // namespace
}  // namespace q4lin
