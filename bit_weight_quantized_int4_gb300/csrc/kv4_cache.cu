// kv4_cache.cu -- keys and values into a paged cache of 4-bit codes, and out of it again.
//
// A code c of a token's head stands for (c - 8) s with one scale s for the head's channels:
// s = amax / 7.5 spreads the 16 codes over [-amax, amax], so that both ends are half a step from
// their codes, as far as any other value may be.  A token's codes and scales depend on nothing
// but the token, so an append touches no older ones.
//
// A warp takes a token's heads, keys or values, `PASSES` x 32 / (D / 8) of them; a lane holds
// eight channels of a head (the two groups of four that the rotation pairs).
#include <algorithm>

#include "q4lin_internal.h"
#include "serving.cuh"

namespace q4lin {
namespace {
using namespace serving;

constexpr int kWarps = 4;

struct Place {
    int64_t page;      // -1: none
    int64_t position;  // in the sequence
    int slot;          // in the page
};

// Where token `token` of the call lies in the cache; without a place where it belongs to no
// sequence, or where an index is out of range (`*bad`).  The whole warp asks for the same token.
__device__ __forceinline__ Place place_of(const q4lin_kv4_cache_t& C, int page_shift, const int32_t* offsets,
                                          const int32_t* starts, int64_t tokens, int64_t token, bool* bad) {
    const int64_t b = find_sequence(C.batch, token, [&](int64_t i) { return (int64_t)__ldg(offsets + i); });
    const int64_t o0 = __ldg(offsets + b), o1 = __ldg(offsets + b + 1), start = __ldg(starts + b);
    Place p = {-1, start + token - o0, 0};
    *bad = false;
    if (token < o0 || token >= o1) return p;
    *bad = true;
    if (o0 < 0 || o1 > tokens || start < 0) return p;
    const int64_t column = p.position >> page_shift;
    if (column >= C.pages_per_sequence) return p;
    const int64_t page = __ldg(C.page_table + b * C.table_stride + column);
    if (page < 0 || page >= C.num_pages) return p;
    *bad = false;
    p.page = page, p.slot = (int)(p.position & ((1 << page_shift) - 1));
    return p;
}

// Whether one of the offsets that this thread of the first CTA looks at decreases or passes the
// tokens: the searches need not come across it.
__device__ __forceinline__ bool offsets_bad(const int32_t* offsets, int64_t batch, int64_t tokens) {
    bool bad = false;
    for (int64_t b = threadIdx.x; b < batch; b += blockDim.x) {
        const int o0 = __ldg(offsets + b), o1 = __ldg(offsets + b + 1);
        bad |= o0 < 0 || o1 < o0 || o1 > tokens;
    }
    return bad;
}

struct AppendArgs {
    q4lin_kv4_cache_t cache;
    q4lin_kv_append_t a;
    int page_shift, k_vec, v_vec;
    int64_t chunks;  // of a token's heads, keys and values
    int* status;
};

// Codes of four channels, the even ones in the low halves of two bytes.  rint(x inv) is at most 8
// for finite x; an infinity is clamped, a NaN becomes 0.
__device__ __forceinline__ uint32_t four_codes(const float* x, float inv) {
    uint32_t w = 0;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const int c = min(max(__float2int_rn(__fmul_rn(x[d], inv)), -8), 7) + 8;
        w |= (uint32_t)c << (4 * d);
    }
    return w;
}

template <int D, int DT, int PASSES>
__global__ void __launch_bounds__(32 * kWarps) kv4_append_kernel(const AppendArgs g) {
    constexpr int U = D / 8, R = 32 / U;  // lanes of a head, heads of a pass
    const q4lin_kv4_cache_t& C = g.cache;
    const int lane = threadIdx.x & 31, u = lane % U;
    if (blockIdx.x == 0 && offsets_bad(g.a.offsets, C.batch, g.a.tokens)) atomicCAS(g.status, 0, kStatusIndex);
    const int64_t items = g.a.tokens * g.chunks;
    for (int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); w < items; w += (int64_t)gridDim.x * kWarps) {
        const int64_t token = w / g.chunks;
        const int chunk = (int)(w - token * g.chunks), half = (int)(g.chunks / 2);
        const bool keys = chunk < half;
        const int h0 = (keys ? chunk : chunk - half) * (PASSES * R) + lane / U;
        bool turned = false;
        int lo = 8 * u, hi = 8 * u + 4;
        if (keys) rope_channels(g.a.rope, u, &turned, &lo, &hi);
        const void* src = keys ? g.a.k : g.a.v;
        const int64_t at = token * (keys ? g.a.k_token_stride : g.a.v_token_stride);
        const int64_t hs = keys ? g.a.k_head_stride : g.a.v_head_stride;
        const bool vec = keys ? g.k_vec : g.v_vec;
        float x[PASSES][8];
#pragma unroll
        for (int p = 0; p < PASSES; ++p)
            if (h0 + p * R < C.kv_heads) {
                load_four(src, DT, at + (h0 + p * R) * hs + lo, vec, x[p]);
                load_four(src, DT, at + (h0 + p * R) * hs + hi, vec, x[p] + 4);
            }
        bool bad;
        Place place = place_of(C, g.page_shift, g.a.offsets, g.a.starts, g.a.tokens, token, &bad);
        if (keys && g.a.rope.cos && place.page >= 0 && place.position >= g.a.rope.positions) place.page = -1, bad = true;
        if (bad && lane == 0) atomicCAS(g.status, 0, kStatusIndex);
        if (place.page < 0) continue;
        float c[4], s[4];
        if (turned) rope_load(g.a.rope, place.position, u, c, s);
        uint8_t* codes = keys ? C.k_codes : C.v_codes;
        float* scales = keys ? C.k_scales : C.v_scales;
        bool finite = true;
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int h = h0 + p * R;
            if (h - lane / U >= C.kv_heads) break;
            const bool in = h < C.kv_heads;
            float amax = 0.f;
            if (in) {
                if (turned) rope_apply(g.a.rope, c, s, x[p]);
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                    const float m = fabsf(x[p][d]);
                    const bool fine = m <= 3.4028235e38f;
                    amax = fine ? fmaxf(amax, m) : amax;
                    finite = finite && fine;
                }
            }
#pragma unroll
            for (int o = U / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            float scale = __fmul_rn(amax, (float)(1.0 / 7.5));
            scale = scale >= 1.17549435e-38f ? scale : 0.f;
            const float inv = scale > 0.f ? __frcp_rn(scale) : 0.f;
            if (!in) continue;
            const int64_t row = ((place.page * C.kv_heads + h) << g.page_shift) + place.slot;
            if (u == 0) scales[row] = scale;
            *reinterpret_cast<uint16_t*>(codes + row * (D / 2) + lo / 2) = (uint16_t)four_codes(x[p], inv);
            *reinterpret_cast<uint16_t*>(codes + row * (D / 2) + hi / 2) = (uint16_t)four_codes(x[p] + 4, inv);
        }
        if (!finite) atomicCAS(g.status, 0, kStatusNonFinite);
    }
}

struct ReadArgs {
    q4lin_kv4_cache_t cache;
    q4lin_kv_read_t a;
    int page_shift;
    int64_t chunks;
    int* status;
};

template <int D, int DT, int PASSES>
__global__ void __launch_bounds__(32 * kWarps) kv4_read_kernel(const ReadArgs g) {
    constexpr int U = D / 8, R = 32 / U;
    const q4lin_kv4_cache_t& C = g.cache;
    const int lane = threadIdx.x & 31, u = lane % U;
    if (blockIdx.x == 0 && offsets_bad(g.a.offsets, C.batch, g.a.tokens)) atomicCAS(g.status, 0, kStatusIndex);
    const int64_t items = g.a.tokens * g.chunks;
    for (int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); w < items; w += (int64_t)gridDim.x * kWarps) {
        const int64_t token = w / g.chunks;
        const int h0 = (int)(w - token * g.chunks) * (PASSES * R) + lane / U;
        bool bad;
        const Place place = place_of(C, g.page_shift, g.a.offsets, g.a.starts, g.a.tokens, token, &bad);
        if (bad && lane == 0) atomicCAS(g.status, 0, kStatusIndex);
        if (place.page < 0) continue;
        uint32_t word[2][PASSES];
        float scale[2][PASSES];
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int h = h0 + p * R;
            if (h >= C.kv_heads) break;
            const int64_t row = ((place.page * C.kv_heads + h) << g.page_shift) + place.slot;
            if (g.a.k) {
                word[0][p] = __ldg(reinterpret_cast<const uint32_t*>(C.k_codes + row * (D / 2)) + u);
                scale[0][p] = __ldg(C.k_scales + row);
            }
            if (g.a.v) {
                word[1][p] = __ldg(reinterpret_cast<const uint32_t*>(C.v_codes + row * (D / 2)) + u);
                scale[1][p] = __ldg(C.v_scales + row);
            }
        }
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int h = h0 + p * R;
            if (h >= C.kv_heads) break;
#pragma unroll
            for (int kind = 0; kind < 2; ++kind) {
                void* out = kind ? g.a.v : g.a.k;
                if (!out) continue;
                float x[8];
#pragma unroll
                for (int d = 0; d < 8; ++d)
                    x[d] = (float)((int)(word[kind][p] >> (4 * d) & 15u) - 8) * scale[kind][p];
                const int64_t at = (token * C.kv_heads + h) * D + 8 * u;
                store_four(out, DT, at, true, x);
                store_four(out, DT, at + 4, true, x + 4);
            }
        }
    }
}

unsigned blocks_of(int64_t items) { return (unsigned)std::min<int64_t>((items + kWarps - 1) / kWarps, 1 << 30); }

template <int D, int DT>
cudaError_t append(AppendArgs& g, cudaStream_t stream) {
    constexpr int kPasses = 1, kHeads = kPasses * 32 / (D / 8);
    g.chunks = 2 * ((g.cache.kv_heads + kHeads - 1) / kHeads);
    kv4_append_kernel<D, DT, kPasses><<<blocks_of(g.a.tokens * g.chunks), 32 * kWarps, 0, stream>>>(g);
    return cudaGetLastError();
}
template <int D, int DT>
cudaError_t read(ReadArgs& g, cudaStream_t stream) {
    constexpr int kPasses = 1, kHeads = kPasses * 32 / (D / 8);
    g.chunks = (g.cache.kv_heads + kHeads - 1) / kHeads;
    kv4_read_kernel<D, DT, kPasses><<<blocks_of(g.a.tokens * g.chunks), 32 * kWarps, 0, stream>>>(g);
    return cudaGetLastError();
}
// f(head_dim, dtype) with both as types.
template <typename F>
cudaError_t by_dim_and_type(int64_t dim, int dtype, F f) {
    auto typed = [&](auto d) {
        constexpr int D = decltype(d)::value;
        if (dtype == Q4LIN_DTYPE_F32) return f.template operator()<D, Q4LIN_DTYPE_F32>();
        if (dtype == Q4LIN_DTYPE_F16) return f.template operator()<D, Q4LIN_DTYPE_F16>();
        return f.template operator()<D, Q4LIN_DTYPE_BF16>();
    };
    if (dim == 64) return typed(std::integral_constant<int, 64>{});
    if (dim == 128) return typed(std::integral_constant<int, 128>{});
    return typed(std::integral_constant<int, 256>{});
}
struct Append {
    AppendArgs& g;
    cudaStream_t stream;
    template <int D, int DT>
    cudaError_t operator()() const { return append<D, DT>(g, stream); }
};
struct Read {
    ReadArgs& g;
    cudaStream_t stream;
    template <int D, int DT>
    cudaError_t operator()() const { return read<D, DT>(g, stream); }
};
int shift_of(int64_t page_size) { return page_size == 16 ? 4 : page_size == 32 ? 5 : 6; }

}  // namespace

cudaError_t kv4_append_launch(const q4lin_kv4_cache_t& cache, const q4lin_kv_append_t& a, const LaunchCtx& c) {
    AppendArgs g;
    g.cache = cache;
    g.a = a;
    g.page_shift = shift_of(cache.page_size);
    g.k_vec = fours_aligned(a.k, a.dtype, a.k_token_stride, a.k_head_stride);
    g.v_vec = fours_aligned(a.v, a.dtype, a.v_token_stride, a.v_head_stride);
    g.status = c.status_word;
    return by_dim_and_type(cache.head_dim, a.dtype, Append{g, c.stream});
}

cudaError_t kv4_read_launch(const q4lin_kv4_cache_t& cache, const q4lin_kv_read_t& a, const LaunchCtx& c) {
    ReadArgs g;
    g.cache = cache;
    g.a = a;
    g.page_shift = shift_of(cache.page_size);
    g.status = c.status_word;
    return by_dim_and_type(cache.head_dim, a.dtype, Read{g, c.stream});
}

}  // namespace q4lin
