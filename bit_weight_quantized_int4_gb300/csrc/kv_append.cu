// kv_append.cu -- keys and values appended to the paged 8-bit cache, keys rotated on the way.
//
// One CTA per (page that receives tokens, head, keys or values).  It holds the page's new
// tokens in registers between the two steps of the quantisation (the largest |x|, then the
// codes), so they are read once; each unit of a thread is eight channels of one token, and a
// thread's units are eight consecutive tokens of the same channels, so that the transposed
// values leave as eight consecutive bytes per channel.
//
// Bound: memory traffic (size + 1 bytes per element) for prompts, the chain of dependent
// loads (offset -> page -> old scale) for single tokens.  The old codes of a page are read
// and written only where its scale grows.
#include "q4lin_internal.h"
#include "serving.cuh"

namespace q4lin {
namespace {
using namespace serving;

constexpr int kUnits = 8;  // tokens per thread

struct AppendArgs {
    q4lin_kv_cache_t cache;
    q4lin_kv_append_t a;
    int page_shift;
    int by_token;  // blockIdx.x counts tokens (few per sequence), else page slots
    int k_vec, v_vec;
    int* status;
};

// Page slots of sequence b: offsets[b] / page + 2 b up to the same of b + 1.  A sequence of
// n tokens touches at most (n - 1) / page + 2 pages, which never exceeds that difference.
__device__ __forceinline__ int64_t first_slot(const AppendArgs& g, int64_t b) {
    return ((int64_t)__ldg(g.a.offsets + b) >> g.page_shift) + 2 * b;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) kv_append_kernel(const AppendArgs g) {
    __shared__ float s_amax[THREADS / 32];
    const q4lin_kv_cache_t& C = g.cache;
    const int D = (int)C.head_dim, P = (int)C.page_size, units = D / 8;
    const int h = blockIdx.y;
    const bool keys = blockIdx.z == 0;

    // Which tokens: rows [first, first + n) of the call, slots [at, at + n) of their page.
    int64_t b;
    if (g.by_token) {
        b = find_sequence(C.batch, blockIdx.x, [&](int64_t i) { return (int64_t)__ldg(g.a.offsets + i); });
    } else {
        b = find_sequence(C.batch, blockIdx.x, [&](int64_t i) { return first_slot(g, i); });
    }
    const int64_t o0 = __ldg(g.a.offsets + b), o1 = __ldg(g.a.offsets + b + 1);
    const int64_t start = __ldg(g.a.starts + b);
    if (o0 < 0 || o1 > g.a.tokens || start < 0) {
        if (threadIdx.x == 0) atomicCAS(g.status, 0, kStatusIndex);
        return;
    }
    if (o1 <= o0) return;
    int64_t page0;  // first position of the page
    if (g.by_token) {
        const int64_t position = start + blockIdx.x - o0;
        if (blockIdx.x < o0 || blockIdx.x >= o1) return;
        if (blockIdx.x != o0 && (position & (P - 1)) != 0) return;  // another token's page
        page0 = position & ~(int64_t)(P - 1);
    } else {
        const int64_t j = blockIdx.x - first_slot(g, b);
        if (j < 0) return;
        page0 = ((start >> g.page_shift) + j) << g.page_shift;
    }
    const int64_t end = start + (o1 - o0);
    if (page0 >= end) return;
    const int64_t p0 = page0 > start ? page0 : start;             // first new position
    const int64_t p1 = page0 + P < end ? page0 + P : end;         // past the last
    const int at = (int)(p0 - page0), n = (int)(p1 - p0);
    const int64_t first = o0 + (p0 - start);
    const int64_t column = page0 >> g.page_shift;
    const bool turn = keys && g.a.rope.cos != nullptr;
    int64_t page = -1;
    if (column < C.pages_per_sequence) page = __ldg(C.page_table + b * C.table_stride + column);
    if (page < 0 || page >= C.num_pages || (turn && p1 > g.a.rope.positions)) {
        if (threadIdx.x == 0) atomicCAS(g.status, 0, kStatusIndex);
        return;
    }
    const int64_t head = page * C.kv_heads + h;
    uint8_t* codes = (keys ? C.k_codes : C.v_codes) + head * ((int64_t)D << g.page_shift);
    float* scale = (keys ? C.k_scales : C.v_scales) + head;
    const float s0 = at > 0 ? *scale : 0.f;

    // Thread (u, q): channels of unit u, slots 8 q .. 8 q + 7 of the page.
    const int u = threadIdx.x % units, q = threadIdx.x / units;
    const void* src = keys ? g.a.k : g.a.v;
    const int64_t ts = keys ? g.a.k_token_stride : g.a.v_token_stride;
    const int64_t hs = keys ? g.a.k_head_stride : g.a.v_head_stride;
    const bool vec = keys ? g.k_vec : g.v_vec;
    bool turned = false;
    int lo = 8 * u, hi = 8 * u + 4;
    if (keys) rope_channels(g.a.rope, u, &turned, &lo, &hi);
    float x[kUnits][8];
    float amax = 0.f;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int r = q * kUnits + i - at;  // new token
        const bool in = r >= 0 && r < n;
        if (in) {
            const int64_t e = (first + r) * ts + h * hs;
            float a[4], c[4];
            load_four(src, g.a.dtype, e + lo, vec, a);
            load_four(src, g.a.dtype, e + hi, vec, c);
#pragma unroll
            for (int d = 0; d < 4; ++d) x[i][d] = a[d], x[i][4 + d] = c[d];
        } else {
#pragma unroll
            for (int d = 0; d < 8; ++d) x[i][d] = 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int r = q * kUnits + i - at;
        if (turned && r >= 0 && r < n) rope_unit(g.a.rope, p0 + r, u, x[i]);
#pragma unroll
        for (int d = 0; d < 8; ++d) {
            const float m = fabsf(x[i][d]);
            const bool finite = m <= 3.4028235e38f;
            amax = fmaxf(amax, finite ? m : 0.f);
            odd |= !finite;
        }
    }
    if (__any_sync(0xffffffffu, odd) && (threadIdx.x & 31) == 0) atomicCAS(g.status, 0, kStatusNonFinite);
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((threadIdx.x & 31) == 0) s_amax[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) amax = fmaxf(amax, s_amax[w]);
    float s = fmaxf(s0, __fmul_rn(amax, (float)(1.0 / 127.0)));
    if (!(s >= 1.17549435e-38f)) s = 0.f;
    const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
    // (Every thread has read s0; the barrier above orders that before the store.)
    if (threadIdx.x == 0) *scale = s;

    if (s > s0 && s0 > 0.f) {
        // Earlier tokens, rounded again to the larger scale, a word of codes at a time.
        const float ratio = __fdiv_rn(s0, s);
        uint32_t* words = reinterpret_cast<uint32_t*>(codes);
        const int count = keys ? at * D / 4 : D << (g.page_shift - 2);
        for (int w = threadIdx.x; w < count; w += THREADS) {
            const int slot = (4 * w) & (P - 1);  // values: the slot of the word's first byte
            if (!keys && slot >= at) continue;
            const uint32_t old = words[w];
            uint32_t now = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = (int)((old >> (8 * e)) & 0xFF);
                const bool held = keys || slot + e < at;
                const int r = (int)rintf(__fmul_rn((float)(c - 128), ratio)) + 128;
                now |= (uint32_t)(held ? r : c) << (8 * e);
            }
            words[w] = now;
        }
        __syncthreads();  // before new codes are stored into the same words
    }

    // Codes.  x * inv may be an infinity (clamped) or a NaN (code 128).
    uint32_t code[kUnits][2];
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            uint32_t v = 0;
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const float y = rintf(__fmul_rn(x[i][4 * w + d], inv));
                const int c = y == y ? (int)fminf(fmaxf(y, -127.f), 127.f) : 0;
                v |= (uint32_t)(c + 128) << (8 * d);
            }
            code[i][w] = v;
        }
    if (keys) {
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int slot = q * kUnits + i, r = slot - at;
            if (r < 0 || r >= n) continue;
            *reinterpret_cast<uint32_t*>(codes + slot * D + lo) = code[i][0];
            *reinterpret_cast<uint32_t*>(codes + slot * D + hi) = code[i][1];
        }
        return;
    }
    const int slot0 = q * kUnits;
    const bool whole = slot0 >= at && slot0 + kUnits <= at + n;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        if (whole) {
            // 4 x 4 byte transposes: word i of channel d holds slots 4 i .. 4 i + 3.
            uint32_t t[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t a = code[4 * i][w], b4 = code[4 * i + 1][w], c = code[4 * i + 2][w],
                               d = code[4 * i + 3][w];
                const uint32_t ab0 = ptx::prmt(a, b4, 0x5140u), ab1 = ptx::prmt(a, b4, 0x7362u);
                const uint32_t cd0 = ptx::prmt(c, d, 0x5140u), cd1 = ptx::prmt(c, d, 0x7362u);
                t[i][0] = ptx::prmt(ab0, cd0, 0x5410u), t[i][1] = ptx::prmt(ab0, cd0, 0x7632u);
                t[i][2] = ptx::prmt(ab1, cd1, 0x5410u), t[i][3] = ptx::prmt(ab1, cd1, 0x7632u);
            }
#pragma unroll
            for (int d = 0; d < 4; ++d)
                *reinterpret_cast<uint2*>(codes + (((w ? hi : lo) + d) << g.page_shift) + slot0) =
                    make_uint2(t[0][d], t[1][d]);
        } else {
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
                const int r = slot0 + i - at;
                if (r < 0 || r >= n) continue;
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    codes[(((w ? hi : lo) + d) << g.page_shift) + slot0 + i] =
                        (uint8_t)(code[i][w] >> (8 * d));
            }
        }
    }
}

bool vector_rows(const void* p, int dtype, int64_t token_stride, int64_t head_stride) {
    return reinterpret_cast<uintptr_t>(p) % (4 * dtype_size(dtype)) == 0 && token_stride % 4 == 0 &&
           head_stride % 4 == 0;
}

}  // namespace

cudaError_t kv_append_launch(const q4lin_kv_cache_t& cache, const q4lin_kv_append_t& a,
                             const LaunchCtx& c) {
    AppendArgs g;
    g.cache = cache;
    g.a = a;
    g.page_shift = cache.page_size == 16 ? 4 : cache.page_size == 32 ? 5 : 6;
    g.k_vec = vector_rows(a.k, a.dtype, a.k_token_stride, a.k_head_stride);
    g.v_vec = vector_rows(a.v, a.dtype, a.v_token_stride, a.v_head_stride);
    g.status = c.status_word;
    // One CTA per token that opens a page's share (every token is looked at), or per page
    // slot, whichever are fewer.
    const int64_t slots = a.tokens / cache.page_size + 2 * cache.batch;
    g.by_token = a.tokens <= slots;
    const dim3 grid((unsigned)(g.by_token ? a.tokens : slots), (unsigned)cache.kv_heads, 2);
    const int64_t threads = cache.head_dim / 8 * (cache.page_size / kUnits);
    if (threads <= 64)
        kv_append_kernel<64><<<grid, 64, 0, c.stream>>>(g);
    else if (threads <= 128)
        kv_append_kernel<128><<<grid, 128, 0, c.stream>>>(g);
    else
        kv_append_kernel<256><<<grid, 256, 0, c.stream>>>(g);
    return cudaGetLastError();
}

}  // namespace q4lin
