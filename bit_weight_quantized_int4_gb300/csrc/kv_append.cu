// kv_append.cu -- keys and values appended to the paged 8-bit cache, keys rotated on the way.
//
// Two kernels.  Prompts: one CTA per (page that receives tokens, head, keys or values).  It
// holds the page's new tokens in registers between the two steps of the quantisation (the
// largest |x|, then the codes), so they are read once; a thread's units are eight consecutive
// tokens of the same eight channels, so that the values are transposed in registers; a whole
// page's codes leave through shared memory.  Few tokens a sequence: one warp per (page, head, keys or values).
//
// Bound: memory traffic (size + 1 bytes per element) for prompts, the chain of dependent
// loads (offset -> page -> old scale) for single tokens; what does not depend on the last
// load is asked for with it.  The old codes of a page are read and written only where its
// scale grows.
//
// Measured: prompts of 8 k tokens, 48.5 MB, 12.7 us where the linears have just written them (in
// L2), 18.8 us from memory: 2.6 TB/s, 0.38 of a copy's bandwidth.  1344 CTAs of one page and head
// each in three rounds, loads, maximum, codes and stores one after the other: without the last
// two 13.2 us from memory, without the angles 3 less.  (Elements in shared memory, six CTAs an
// SM: 20.8 us; heads side by side: 19.5; angles asked for with the keys: 18.4, but 13.3 from
// L2; five CTAs an SM: 18.8 and 13.2.)  One token 2.5 us, one for each of 64 sequences 3.6 us.
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
    int k_vec, v_vec;
    int* status;
};

// Page slots of sequence b: offsets[b] / page + 2 b up to the same of b + 1.  A sequence of
// n tokens touches at most (n - 1) / page + 2 pages, which never exceeds that difference.
__device__ __forceinline__ int64_t first_slot(const AppendArgs& g, int64_t b, int64_t offset) {
    return (offset >> g.page_shift) + 2 * b;
}

// Whether one of the offsets that this CTA looks at (all CTAs of a blockIdx.x range together look
// at every one) decreases or passes the tokens; the searches below need not come across it.
__device__ __forceinline__ bool offsets_bad(const AppendArgs& g) {
    bool bad = false;
    for (int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; b < g.cache.batch;
         b += (int64_t)gridDim.x * blockDim.x) {
        const int o0 = __ldg(g.a.offsets + b), o1 = __ldg(g.a.offsets + b + 1);
        bad |= o0 < 0 || o1 < o0 || o1 > g.a.tokens;
    }
    return bad;
}

// New tokens of one page: rows [first, first + n) of the call, positions from p0, slots [at,
// at + n).  n is 0 where there are none.
struct Share {
    int64_t b, first, p0, column;
    int at, n;
};

// The share of page slot (or, by token, of the page that token opens for the call) `id`.  The
// sequence is found by a 32-way search of the warp, which brings its three indices along.
template <bool BY_TOKEN>
__device__ __forceinline__ Share find_share(const AppendArgs& g, int64_t id) {
    const int lane = threadIdx.x & 31, P = 1 << g.page_shift;
    int64_t lo = 0, n = g.cache.batch, o0 = 0, o1 = 0, start = 0;
    while (true) {
        const int64_t step = (n + 31) / 32, b = lo + lane * step;
        const bool in = lane * step < n;
        const int64_t o = in ? __ldg(g.a.offsets + b) : 0;
        const int next = in && step == 1 ? __ldg(g.a.offsets + b + 1) : 0;
        const int st = in && step == 1 ? __ldg(g.a.starts + b) : 0;
        const unsigned m = __ballot_sync(0xffffffffu, in && (BY_TOKEN ? o : first_slot(g, b, o)) <= id);
        const int last = m ? 31 - __clz(m) : 0;
        lo += last * step;
        if (step == 1) {
            o0 = __shfl_sync(0xffffffffu, (int)o, last), o1 = __shfl_sync(0xffffffffu, next, last);
            start = __shfl_sync(0xffffffffu, st, last);
            break;
        }
        n = n - last * step < step ? n - last * step : step;
    }
    Share s = {lo, 0, 0, 0, 0, 0};
    if (o0 < 0 || o1 > g.a.tokens || (start < 0 && o1 > o0)) {
        if (threadIdx.x == 0) atomicCAS(g.status, 0, kStatusIndex);
        return s;
    }
    int64_t page0;  // first position of the page
    if (BY_TOKEN) {
        if (id < o0 || id >= o1) return s;
        const int64_t position = start + id - o0;
        if (id != o0 && (position & (P - 1)) != 0) return s;  // another token's page
        page0 = position & ~(int64_t)(P - 1);
    } else {
        const int64_t j = id - first_slot(g, lo, o0);
        if (j < 0) return s;
        page0 = ((start >> g.page_shift) + j) << g.page_shift;
    }
    const int64_t end = start + (o1 - o0);
    if (page0 >= end) return s;
    s.p0 = page0 > start ? page0 : start;                 // first new position
    const int64_t p1 = page0 + P < end ? page0 + P : end;  // past the last
    s.at = (int)(s.p0 - page0), s.n = p1 > s.p0 ? (int)(p1 - s.p0) : 0;
    s.first = o0 + (s.p0 - start);
    s.column = page0 >> g.page_shift;
    return s;
}
// The share's page, -1 where its index or its positions are out of range.
__device__ __forceinline__ int64_t page_of(const AppendArgs& g, const Share& s, bool keys) {
    const q4lin_kv_cache_t& C = g.cache;
    const int64_t page =
        s.column < C.pages_per_sequence ? __ldg(C.page_table + s.b * C.table_stride + s.column) : -1;
    const bool ok = page >= 0 && page < C.num_pages &&
                    !(keys && g.a.rope.cos && s.p0 + s.n > g.a.rope.positions);
    return ok ? page : -1;
}

// The page's scale from that of its earlier tokens (0: none) and the new tokens' largest |x|.
__device__ __forceinline__ float new_scale(float s0, float amax) {
    const float s = fmaxf(s0, __fmul_rn(amax, (float)(1.0 / 127.0)));
    return s >= 1.17549435e-38f ? s : 0.f;
}
// Largest |x|, and whether all are finite: 0 x is 0 only then.
__device__ __forceinline__ void largest(const float (&x)[8], float& amax, float& zero) {
#pragma unroll
    for (int d = 0; d < 8; ++d) amax = fmaxf(amax, fabsf(x[d])), zero = fmaf(x[d], 0.f, zero);
}
__device__ __forceinline__ float largest_finite(const float (&x)[8], float amax) {
#pragma unroll
    for (int d = 0; d < 8; ++d) {
        const float m = fabsf(x[d]);
        amax = m <= 3.4028235e38f ? fmaxf(amax, m) : amax;
    }
    return amax;
}
// Four codes.  Finite x: |x inv| rounds to 127 at most, and adding 1.5 2^23 + 128 rounds it to a
// whole number, half to even, whose low byte is the code.  Else x inv may be an infinity
// (clamped) or a NaN (code 128).
__device__ __forceinline__ uint32_t four_codes(const float* x, float inv, bool finite) {
    uint32_t c[4];
    if (finite) {
#pragma unroll
        for (int d = 0; d < 4; ++d) c[d] = __float_as_uint(__fadd_rn(__fmul_rn(x[d], inv), 12583040.f));
    } else {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const float y = __fmul_rn(x[d], inv);
            c[d] = y == y ? (uint32_t)((int)fminf(fmaxf(rintf(y), -127.f), 127.f) + 128) : 128u;
        }
    }
    return ptx::prmt(ptx::prmt(c[0], c[1], 0x0040u), ptx::prmt(c[2], c[3], 0x0040u), 0x5410u);
}
// Codes of the page's first `at` tokens, rounded again to a scale that is 1 / ratio larger: 16
// bytes at a time, four in flight, by `count` threads of which this is number `id`.
__device__ __forceinline__ void round_again(const AppendArgs& g, uint8_t* codes, bool keys, int at, float ratio,
                                            int id, int count) {
    const int D = (int)g.cache.head_dim, P = 1 << g.page_shift;
    uint4* units = reinterpret_cast<uint4*>(codes);
    const int all = keys ? at * D / 16 : D * P / 16;
    for (int u0 = id; u0 < all; u0 += 4 * count) {
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (u0 + k * count < all) v[k] = units[u0 + k * count];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int u = u0 + k * count, slot = (16 * u) & (P - 1);  // values: of the first byte
            if (u >= all || (!keys && slot >= at)) continue;
            uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t now = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c = (int)((w[j] >> (8 * e)) & 0xFF);
                    const bool held = keys || slot + 4 * j + e < at;
                    const int r = (int)rintf(__fmul_rn((float)(c - 128), ratio)) + 128;
                    now |= (uint32_t)(held ? r : c) << (8 * e);
                }
                w[j] = now;
            }
            units[u] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// Prompts: blockIdx.x is a page slot.
template <int THREADS, int DT>
__global__ void __launch_bounds__(THREADS) kv_append_pages_kernel(const AppendArgs g) {
    __shared__ float s_amax[THREADS / 32];
    __shared__ uint4 s_codes[THREADS * 4];
    const q4lin_kv_cache_t& C = g.cache;
    const int D = (int)C.head_dim, P = 1 << g.page_shift, units = D / 8, h = blockIdx.y;
    const bool keys = blockIdx.z == 0;
    if (h == 0 && keys && offsets_bad(g)) atomicCAS(g.status, 0, kStatusIndex);
    const Share s = find_share<false>(g, blockIdx.x);
    if (s.n == 0) return;
    const int64_t page = page_of(g, s, keys);

    // Thread (u, q): channels of unit u, slots 8 q .. 8 q + 7 of the page.
    const int u = threadIdx.x % units, q = threadIdx.x / units;
    const void* src = keys ? g.a.k : g.a.v;
    const int64_t ts = keys ? g.a.k_token_stride : g.a.v_token_stride;
    const int64_t at0 = s.first * ts + h * (keys ? g.a.k_head_stride : g.a.v_head_stride);
    const bool vec = keys ? g.k_vec : g.v_vec;
    bool turned = false;
    int lo = 4 * u, hi = D / 2 + 4 * u;
    if (keys) rope_channels(g.a.rope, u, &turned, &lo, &hi);
    float x[kUnits][8];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int r = q * kUnits + i - s.at;  // new token
#pragma unroll
        for (int d = 0; d < 8; ++d) x[i][d] = 0.f;
        if (r >= 0 && r < s.n) {
            load_four(src, DT, at0 + r * ts + lo, vec, x[i]);
            load_four(src, DT, at0 + r * ts + hi, vec, x[i] + 4);
        }
    }
    if (page < 0) {
        if (threadIdx.x == 0) atomicCAS(g.status, 0, kStatusIndex);
        return;
    }
    const int64_t head = page * C.kv_heads + h;
    uint8_t* codes = (keys ? C.k_codes : C.v_codes) + head * ((int64_t)D << g.page_shift);
    float* scale = (keys ? C.k_scales : C.v_scales) + head;
    const float s0 = s.at > 0 ? *scale : 0.f;
    float amax = 0.f, zero = 0.f;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int r = q * kUnits + i - s.at;
        if (turned && r >= 0 && r < s.n) rope_unit(g.a.rope, s.p0 + r, u, x[i]);
        largest(x[i], amax, zero);
    }
    const bool finite = !__syncthreads_or(zero != 0.f);
    if (!finite) {
        if (threadIdx.x == 0) atomicCAS(g.status, 0, kStatusNonFinite);
        amax = 0.f;
#pragma unroll
        for (int i = 0; i < kUnits; ++i) amax = largest_finite(x[i], amax);
    }
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));  // not negative
    if ((threadIdx.x & 31) == 0) s_amax[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) amax = fmaxf(amax, s_amax[w]);
    const float now = new_scale(s0, amax), inv = now > 0.f ? __frcp_rn(now) : 0.f;
    // (Every thread has read s0; the barrier above orders that before the store.)
    if (threadIdx.x == 0) *scale = now;
    if (now > s0 && s0 > 0.f) {
        round_again(g, codes, keys, s.at, __fdiv_rn(s0, now), threadIdx.x, THREADS);
        __syncthreads();  // before new codes are stored into the same 16 bytes
    }

    uint32_t code[kUnits][2];
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
        code[i][0] = four_codes(x[i], inv, finite), code[i][1] = four_codes(x[i] + 4, inv, finite);
    const int slot0 = q * kUnits;
    const bool whole = slot0 >= s.at && slot0 + kUnits <= s.at + s.n;
    if (!keys && whole) {
        // 4 x 4 byte transposes: word i of channel d holds slots 4 i .. 4 i + 3.
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int i = 0; i < kUnits; i += 4) {
                const uint32_t a = code[i][w], b4 = code[i + 1][w], c = code[i + 2][w], d = code[i + 3][w];
                const uint32_t ab0 = ptx::prmt(a, b4, 0x5140u), ab1 = ptx::prmt(a, b4, 0x7362u);
                const uint32_t cd0 = ptx::prmt(c, d, 0x5140u), cd1 = ptx::prmt(c, d, 0x7362u);
                code[i][w] = ptx::prmt(ab0, cd0, 0x5410u), code[i + 1][w] = ptx::prmt(ab0, cd0, 0x7632u);
                code[i + 2][w] = ptx::prmt(ab1, cd1, 0x5410u), code[i + 3][w] = ptx::prmt(ab1, cd1, 0x7632u);
            }
    }
    if (s.n == P) {
        // A whole page leaves by 16 bytes a thread, one after the other, through shared memory
        // (stored from where they are, 4 or 8 bytes at a time, 13.2 and 19.2 us for the prompts at
        // the head of this file instead of 12.7 and 18.8).
        // There, 8 slots of a channel (of G such groups) trade places by its number.
        uint8_t* stage = reinterpret_cast<uint8_t*>(s_codes);
        const int G = P / kUnits;
        if (q < G) {
            if (keys) {
#pragma unroll
                for (int i = 0; i < kUnits; ++i) {
                    *reinterpret_cast<uint32_t*>(stage + (slot0 + i) * D + lo) = code[i][0];
                    *reinterpret_cast<uint32_t*>(stage + (slot0 + i) * D + hi) = code[i][1];
                }
            } else {
#pragma unroll
                for (int w = 0; w < 2; ++w)
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        const int channel = (w ? hi : lo) + d;
                        *reinterpret_cast<uint2*>(stage + channel * P + ((q ^ (channel >> 2)) & (G - 1)) * kUnits) =
                            make_uint2(code[d][w], code[4 + d][w]);
                    }
            }
        }
        __syncthreads();
        for (int n = threadIdx.x; n < P * D / 16; n += THREADS) {
            uint4 v = s_codes[n];
            if (!keys) {
                const int channel = (16 * n) >> g.page_shift, k = (channel >> 2) & (G - 1);
                v = s_codes[n ^ (k >> 1)];
                if (k & 1) v = make_uint4(v.z, v.w, v.x, v.y);
            }
            reinterpret_cast<uint4*>(codes)[n] = v;
        }
        return;
    }
    if (keys) {
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int slot = slot0 + i, r = slot - s.at;
            if (r < 0 || r >= s.n) continue;
            *reinterpret_cast<uint32_t*>(codes + slot * D + lo) = code[i][0];
            *reinterpret_cast<uint32_t*>(codes + slot * D + hi) = code[i][1];
        }
        return;
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        if (whole) {
#pragma unroll
            for (int d = 0; d < 4; ++d)
                *reinterpret_cast<uint2*>(codes + (((w ? hi : lo) + d) << g.page_shift) + slot0) =
                    make_uint2(code[d][w], code[4 + d][w]);
        } else {
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
                const int r = slot0 + i - s.at;
                if (r < 0 || r >= s.n) continue;
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    codes[(((w ? hi : lo) + d) << g.page_shift) + slot0 + i] =
                        (uint8_t)(code[i][w] >> (8 * d));
            }
        }
    }
}

// Few tokens a sequence: blockIdx.x is a token; a warp takes a head's keys or values.
constexpr int kTokenWarps = 4;
template <int DT>
__global__ void __launch_bounds__(32 * kTokenWarps) kv_append_tokens_kernel(const AppendArgs g) {
    const q4lin_kv_cache_t& C = g.cache;
    const int D = (int)C.head_dim, units = D / 8, per = 32 / units;  // tokens at a time
    const int lane = threadIdx.x & 31, item = blockIdx.y * kTokenWarps + (threadIdx.x >> 5);
    const int h = item >> 1;
    const bool keys = (item & 1) == 0;
    if (blockIdx.y == 0 && offsets_bad(g)) atomicCAS(g.status, 0, kStatusIndex);
    if (h >= C.kv_heads) return;
    const Share s = find_share<true>(g, blockIdx.x);
    if (s.n == 0) return;
    const int64_t page = page_of(g, s, keys);
    const int u = lane % units;
    const void* src = keys ? g.a.k : g.a.v;
    const int64_t ts = keys ? g.a.k_token_stride : g.a.v_token_stride;
    const int64_t at0 = s.first * ts + h * (keys ? g.a.k_head_stride : g.a.v_head_stride);
    const bool vec = keys ? g.k_vec : g.v_vec;
    bool turned = false;
    int lo = 8 * u, hi = 8 * u + 4;
    if (keys) rope_channels(g.a.rope, u, &turned, &lo, &hi);
    if (turned && s.p0 + s.n > g.a.rope.positions) turned = false;  // reported below
    float x[8];
    auto load = [&](int r0) {  // tokens r0 .. r0 + per - 1, rotated
        const int r = r0 + lane / units;
#pragma unroll
        for (int d = 0; d < 8; ++d) x[d] = 0.f;
        if (r < s.n) {
            float c[4], sn[4];
            if (turned) rope_load(g.a.rope, s.p0 + r, u, c, sn);
            load_four(src, DT, at0 + r * ts + lo, vec, x);
            load_four(src, DT, at0 + r * ts + hi, vec, x + 4);
            if (turned) rope_apply(g.a.rope, c, sn, x);
        }
    };
    load(0);
    if (page < 0) {
        if (lane == 0) atomicCAS(g.status, 0, kStatusIndex);
        return;
    }
    const int64_t head = page * C.kv_heads + h;
    uint8_t* codes = (keys ? C.k_codes : C.v_codes) + head * ((int64_t)D << g.page_shift);
    float* scale = (keys ? C.k_scales : C.v_scales) + head;
    const float s0 = s.at > 0 ? *scale : 0.f;
    float amax = 0.f, zero = 0.f;
    largest(x, amax, zero);
    for (int r0 = per; r0 < s.n; r0 += per) {
        load(r0);
        largest(x, amax, zero);
    }
    const bool finite = !__any_sync(0xffffffffu, zero != 0.f);
    if (!finite) {
        if (lane == 0) atomicCAS(g.status, 0, kStatusNonFinite);
        amax = 0.f;
        for (int r0 = 0; r0 < s.n; r0 += per) {
            if (s.n > per) load(r0);
            amax = largest_finite(x, amax);
        }
    }
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));  // not negative
    const float now = new_scale(s0, amax), inv = now > 0.f ? __frcp_rn(now) : 0.f;
    if (lane == 0) *scale = now;
    if (now > s0 && s0 > 0.f) {
        round_again(g, codes, keys, s.at, __fdiv_rn(s0, now), lane, 32);
        __syncwarp();  // before new codes are stored into the same 16 bytes
    }
    for (int r0 = 0; r0 < s.n; r0 += per) {
        if (s.n > per) load(r0);
        const int r = r0 + lane / units, slot = s.at + r;
        if (r >= s.n) continue;
        const uint32_t a = four_codes(x, inv, finite), b = four_codes(x + 4, inv, finite);
        if (keys) {
            *reinterpret_cast<uint32_t*>(codes + slot * D + lo) = a;
            *reinterpret_cast<uint32_t*>(codes + slot * D + hi) = b;
        } else {
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                codes[((lo + d) << g.page_shift) + slot] = (uint8_t)(a >> (8 * d));
                codes[((hi + d) << g.page_shift) + slot] = (uint8_t)(b >> (8 * d));
            }
        }
    }
}

bool vector_rows(const void* p, int dtype, int64_t token_stride, int64_t head_stride) {
    return reinterpret_cast<uintptr_t>(p) % (4 * dtype_size(dtype)) == 0 && token_stride % 4 == 0 &&
           head_stride % 4 == 0;
}

template <int DT>
cudaError_t launch(const AppendArgs& g, cudaStream_t stream) {
    // A warp per token and head (of which those that do not open a page's share leave at once)
    // or a CTA per page slot and head, whichever are fewer.
    const int64_t slots = g.a.tokens / g.cache.page_size + 2 * g.cache.batch;
    if (g.a.tokens <= slots) {
        const dim3 grid((unsigned)g.a.tokens, (unsigned)((2 * g.cache.kv_heads + kTokenWarps - 1) / kTokenWarps));
        kv_append_tokens_kernel<DT><<<grid, 32 * kTokenWarps, 0, stream>>>(g);
        return cudaGetLastError();
    }
    const dim3 grid((unsigned)slots, (unsigned)g.cache.kv_heads, 2);
    const int64_t threads = g.cache.head_dim / 8 * (g.cache.page_size / kUnits);
    if (threads <= 64)
        kv_append_pages_kernel<64, DT><<<grid, 64, 0, stream>>>(g);
    else if (threads <= 128)
        kv_append_pages_kernel<128, DT><<<grid, 128, 0, stream>>>(g);
    else
        kv_append_pages_kernel<256, DT><<<grid, 256, 0, stream>>>(g);
    return cudaGetLastError();
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
    switch (a.dtype) {
        case Q4LIN_DTYPE_F32: return launch<Q4LIN_DTYPE_F32>(g, c.stream);
        case Q4LIN_DTYPE_F16: return launch<Q4LIN_DTYPE_F16>(g, c.stream);
        default: return launch<Q4LIN_DTYPE_BF16>(g, c.stream);
    }
}

}  // namespace q4lin
