// kv4_attention.cu -- attention over the paged cache of 4-bit codes.
//
// One CTA for a query row (token and head): its threads take keys in turn for the scores, then
// channels for the outputs, 256 keys at a time, with the running maximum and sum of a softmax.
#include <algorithm>

#include "q4lin_internal.h"
#include "serving.cuh"

namespace q4lin {
namespace {
using namespace serving;

constexpr int kThreads = 256;

struct Args {
    q4lin_kv4_cache_t cache;
    q4lin_attention_t a;
    int page_shift;
    int* status;
};

__global__ void __launch_bounds__(kThreads) kv4_attention_kernel(const Args g) {
    __shared__ float q[256], p[kThreads], part[8], o_part[kThreads];
    __shared__ int64_t place[kThreads];
    const q4lin_kv4_cache_t& C = g.cache;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, D = (int)C.head_dim, ps = g.page_shift;
    const int64_t token = blockIdx.x / g.a.heads, head = blockIdx.x - token * g.a.heads;
    const int64_t h = head / (g.a.heads / C.kv_heads);
    if (blockIdx.x == 0)
        for (int64_t b = tid; b < C.batch; b += kThreads) {
            const int o0 = __ldg(g.a.offsets + b), o1 = __ldg(g.a.offsets + b + 1);
            if (o0 < 0 || o1 < o0 || o1 > g.a.tokens) atomicCAS(g.status, 0, kStatusIndex);
        }
    const int64_t b = find_sequence(C.batch, token, [&](int64_t i) { return (int64_t)__ldg(g.a.offsets + i); });
    const int64_t o0 = __ldg(g.a.offsets + b), o1 = __ldg(g.a.offsets + b + 1);
    int64_t len = __ldg(g.a.lengths + b);
    if (token < o0 || token >= o1) return;
    if (o0 < 0 || o1 > g.a.tokens || o1 - o0 > g.a.max_query || len > C.pages_per_sequence << ps ||
        (g.a.rope.cos && len > g.a.rope.positions)) {
        if (tid == 0) atomicCAS(g.status, 0, kStatusIndex);
        return;
    }
    if (len < 0) len = 0;
    const int64_t position = len - (o1 - o0) + (token - o0);
    if (tid < D / 8) {
        bool turned;
        int lo, hi;
        float x[8];
        rope_channels(g.a.rope, tid, &turned, &lo, &hi);
        const int64_t at = token * g.a.q_token_stride + head * g.a.q_head_stride;
        load_four(g.a.query, g.a.dtype, at + lo, false, x);
        load_four(g.a.query, g.a.dtype, at + hi, false, x + 4);
        if (turned && position >= 0) rope_unit(g.a.rope, position, tid, x);
        for (int e = 0; e < 8; ++e) q[e < 4 ? lo + e : hi + e - 4] = x[e];
    }
    __syncthreads();
    int64_t end = g.a.causal ? position + 1 : len, low = g.a.window > 0 ? position - g.a.window + 1 : 0;
    end = max((int64_t)0, min(end, len)), low = max((int64_t)0, low);
    // A power of two keeps the sums of products in fp32's range.
    float most = 0.f;
    for (int i = 0; i < D; ++i) most = fmaxf(most, fabsf(q[i]));
    const int ex = min(max((int)(__float_as_uint(most) >> 23), 30), 254) - 127;
    // (With an infinity all scores become NaN: one of -infinity would look masked.)
    const float up = most == INFINITY ? NAN : __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
    const float factor = g.a.scale * kLog2e * __uint_as_float((uint32_t)(127 - 14 + ex) << 23);
    float m = -INFINITY, l = 0.f, o = 0.f;
    const int groups = kThreads / D, d = tid % D;  // groups of keys for the outputs
    for (int64_t k0 = low; k0 < end; k0 += kThreads) {
        const int64_t key = k0 + tid;
        float s = -INFINITY;
        place[tid] = -1;
        if (key < end) {
            int64_t page = __ldg(C.page_table + b * C.table_stride + (key >> ps));
            if (page < 0 || page >= C.num_pages) {
                atomicCAS(g.status, 0, kStatusIndex);
                page = 0;
            }
            const int64_t row = ((page * C.kv_heads + h) << ps) + (key & ((1 << ps) - 1));
            place[tid] = row;
            const uint8_t* codes = C.k_codes + row * (D / 2);
            float dot = 0.f;
            for (int c = 0; c < D / 2; ++c) {
                const int w = __ldg(codes + c);
                dot = fmaf(q[2 * c] * up, (float)((w & 15) - 8), dot);
                dot = fmaf(q[2 * c + 1] * up, (float)((w >> 4) - 8), dot);
            }
            s = dot * __ldg(C.k_scales + row) * factor;
        }
        float mx = s;
        for (int i = 16; i; i >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, i));
        if (lane == 0) part[warp] = mx;
        __syncthreads();
        mx = m;
        for (int i = 0; i < kThreads / 32; ++i) mx = fmaxf(mx, part[i]);
        const float base = mx == -INFINITY ? 0.f : mx, alpha = exp2f(m - base);
        m = mx;
        p[tid] = key < end ? exp2f(s - base) : 0.f;
        __syncthreads();
        l *= alpha, o *= alpha;
        const int n = (int)min((int64_t)kThreads, end - k0);
        for (int i = 0; i < n; ++i) l += p[i];
        for (int i = tid / D; i < n; i += groups) {
            const int w = __ldg(C.v_codes + place[i] * (D / 2) + d / 2);
            o = fmaf(p[i] * __ldg(C.v_scales + place[i]), (float)((d & 1 ? w >> 4 : w & 15) - 8), o);
        }
        __syncthreads();
    }
    o_part[tid] = o;
    __syncthreads();
    if (tid >= D) return;
    for (int i = 1; i < groups; ++i) o += o_part[i * D + tid];
    const int64_t row = token * g.a.heads + head;
    store_one(g.a.out, g.a.dtype, row * D + tid, l > 0.f ? o / l : l == 0.f ? 0.f : NAN);
    if (tid == 0 && g.a.lse)
        g.a.lse[row] = l != 0.f ? ((m == -INFINITY ? 0.f : m) + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace

cudaError_t kv4_attention_launch(const q4lin_kv4_cache_t& cache, const q4lin_attention_t& a, const LaunchCtx& c) {
    Args g;
    g.cache = cache;
    g.a = a;
    g.page_shift = cache.page_size == 16 ? 4 : cache.page_size == 32 ? 5 : 6;
    g.status = c.status_word;
    kv4_attention_kernel<<<(unsigned)(a.tokens * a.heads), kThreads, 0, c.stream>>>(g);
    return cudaGetLastError();
}

}  // namespace q4lin
