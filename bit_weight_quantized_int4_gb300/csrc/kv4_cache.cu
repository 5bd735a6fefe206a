// kv4_cache.cu -- keys and values into a paged cache of 4-bit codes, and out of it again.
//
// A code c of a token's head stands for (c - 8) s with one scale s for the head's channels:
// s = amax / 7.5 spreads the 16 codes over [-amax, amax], so that both ends are half a step from
// their codes, as far as any other value may be.  A token's codes and scales depend on nothing
// but the token, so an append touches no older ones.
//
// A warp takes a few consecutive tokens, whose places its lanes look up together, and of each one to four
// heads' keys or values; a lane holds eight channels of a head (the two groups of four that the
// rotation pairs).  More tokens a warp are fewer lookups, more warps hide more latency.
//
// Bound: memory, 4 and 4 1/2 bytes an element with fp32 for both.  Measured: 7 prompts of up to 2047
// tokens (4510 in all, 8 heads of 128, fp32, rotated) appended and read back in 23 us, a floor of 6
// each: the lookups, the rotation and the codes of short launches; 65531 tokens read in bf16 in 56 us,
// 340 MB, 0.89 of a copy's bandwidth (four heads a warp 75 us, one token a warp 92).  64 single
// tokens 2.8 us for each: a launch.
#include <algorithm>

#include "q4lin_internal.h"
#include "serving.cuh"

namespace q4lin {
namespace {
using namespace ptx;
using namespace serving;

constexpr int kWarps = 4;

struct Place {
    int64_t row;       // of the token's first head, in tokens' rows of codes; -1: none
    int64_t position;  // in the sequence
};

// Where tokens t0 + lane (lanes below `count`) of the call lie in the cache; without a place where one
// belongs to no sequence, or where an index is out of range (*bad).  The whole warp searches for the
// first token's sequence, and each lane goes on from there.
__device__ __forceinline__ Place place_of(const q4lin_kv4_cache_t& C, int page_shift, const int32_t* offsets,
                                          const int32_t* starts, int64_t tokens, int64_t t0, int count, bool* bad) {
    const int lane = threadIdx.x & 31;
    int64_t b = find_sequence(C.batch, t0, [&](int64_t i) { return (int64_t)__ldg(offsets + i); });
    const int64_t token = t0 + lane;
    Place p = {-1, 0};
    *bad = false;
    if (lane >= count) return p;
    int64_t o1 = __ldg(offsets + b + 1);
    if (o1 <= token && b + 1 < C.batch) {
        int64_t lo = b + 1, hi = C.batch;  // the last sequence that begins at or before the token
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) / 2;
            if (__ldg(offsets + mid) <= token)
                lo = mid;
            else
                hi = mid;
        }
        b = lo, o1 = __ldg(offsets + b + 1);
    }
    const int64_t o0 = __ldg(offsets + b), start = __ldg(starts + b);
    if (token < o0 || token >= o1) return p;
    p.position = start + token - o0;
    *bad = true;
    if (o0 < 0 || o1 > tokens || start < 0) return p;
    const int64_t column = p.position >> page_shift;
    if (column >= C.pages_per_sequence) return p;
    const int64_t page = __ldg(C.page_table + b * C.table_stride + column);
    if (page < 0 || page >= C.num_pages) return p;
    *bad = false;
    p.row = ((page * C.kv_heads) << page_shift) + (p.position & ((1 << page_shift) - 1));
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
    int page_shift, tokens_each;
    int* status;
};

// rint(x inv) clamped to [-8, 7], plus 8, of four channels: the even ones in the low halves of two
// bytes.  An infinity is clamped, a NaN becomes 8.
__device__ __forceinline__ uint32_t four_codes(const float* x, float inv) {
    uint32_t w = 0;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const int c = min(max(__float2int_rn(__fmul_rn(x[d], inv)), -8), 7) + 8;
        w |= (uint32_t)c << (4 * d);
    }
    return w;
}
// The same of finite channels: |x inv| is at most 7.5 and a few roundings, so rint gives -8 to 8, and
// adding 1.5 2^23 + 8 rounds to whole numbers, half to even, with the code in the float's low bits (the
// rest of which is a multiple of 2^16, so four of them add up to four codes).
__device__ __forceinline__ uint32_t four_finite_codes(const float* x, float inv) {
    constexpr float kOffset = 12582920.f;
    uint32_t c[4];
#pragma unroll
    for (int d = 0; d < 4; ++d)  // (intrinsics: the product is rounded before the sum)
        c[d] = __float_as_uint(fminf(__fadd_rn(__fmul_rn(x[d], inv), kOffset), kOffset + 7.f));
    return (c[3] * 16u + c[2]) * 256u + (c[1] * 16u + c[0]);  // its low 16 bits
}
// The largest of three, or a NaN among them.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

template <int D, int DT, bool VEC>
__global__ void __launch_bounds__(32 * kWarps) kv4_append_kernel(const AppendArgs g) {
    constexpr int U = D / 8, R = 32 / U;  // lanes of a head, heads of a warp
    const q4lin_kv4_cache_t& C = g.cache;
    const int lane = threadIdx.x & 31, u = lane % U, sub = lane / U;
    follow_stream();
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && offsets_bad(g.a.offsets, C.batch, g.a.tokens))
        atomicCAS(g.status, 0, kStatusIndex);
    const int64_t t0 = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * g.tokens_each;
    if (t0 >= g.a.tokens) return;
    const int count = (int)min((int64_t)g.tokens_each, g.a.tokens - t0);
    const bool keys = blockIdx.z == 0;
    const int h = (int)blockIdx.y * R + sub, heads = (int)C.kv_heads;
    bool turned = false;
    int lo = 8 * u, hi = 8 * u + 4;
    if (keys) rope_channels(g.a.rope, u, &turned, &lo, &hi);
    const void* src = keys ? g.a.k : g.a.v;
    const int64_t ts = keys ? g.a.k_token_stride : g.a.v_token_stride;
    const int64_t hs = keys ? g.a.k_head_stride : g.a.v_head_stride;
    uint8_t* codes = keys ? C.k_codes : C.v_codes;
    float* scales = keys ? C.k_scales : C.v_scales;
    const int64_t at0 = t0 * ts + min(h, heads - 1) * hs;
    float next[8];
    auto fetch = [&](int i) {
        load_four(src, DT, at0 + i * ts + lo, VEC, next);
        load_four(src, DT, at0 + i * ts + hi, VEC, next + 4);
    };
    fetch(0);
    bool bad, finite = true;
    Place place = place_of(C, g.page_shift, g.a.offsets, g.a.starts, g.a.tokens, t0, count, &bad);
    if (keys && g.a.rope.cos && place.row >= 0 && place.position >= g.a.rope.positions) place.row = -1, bad = true;
    if (bad) atomicCAS(g.status, 0, kStatusIndex);
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
        const int64_t row0 = __shfl_sync(0xffffffffu, place.row, i), position = __shfl_sync(0xffffffffu, place.position, i);
        float x[8], c[4], s[4];
#pragma unroll
        for (int d = 0; d < 8; ++d) x[d] = next[d];
        if (i + 1 < count) fetch(i + 1);
        if (row0 < 0) continue;
        if (turned) {
            rope_load(g.a.rope, position, u, c, s);
            rope_apply(g.a.rope, c, s, x);
        }
        float amax = max3_nan(fabsf(x[0]), fabsf(x[1]), fabsf(x[2]));
        amax = max3_nan(amax, fabsf(x[3]), fabsf(x[4]));
        amax = max3_nan(amax, fabsf(x[5]), fabsf(x[6]));
        amax = max3_nan(amax, fabsf(x[7]), 0.f);
        const bool fine = __all_sync(0xffffffffu, amax <= 3.4028235e38f);
        if (!fine) {
            amax = 0.f;
#pragma unroll
            for (int d = 0; d < 8; ++d) amax = fabsf(x[d]) <= 3.4028235e38f ? fmaxf(amax, fabsf(x[d])) : amax;
            finite = false;
        }
#pragma unroll
        for (int o = U / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        float scale = __fmul_rn(amax, (float)(1.0 / 7.5));
        scale = scale >= 1.17549435e-38f ? scale : 0.f;
        const float inv = scale > 0.f ? __frcp_rn(scale) : 0.f;
        const uint32_t a = fine ? four_finite_codes(x, inv) : four_codes(x, inv);
        const uint32_t b = fine ? four_finite_codes(x + 4, inv) : four_codes(x + 4, inv);
        if (h >= heads) continue;
        const int64_t row = row0 + ((int64_t)h << g.page_shift);
        uint8_t* to = codes + row * (D / 2);
        if (u == 0) scales[row] = scale;
        if (hi == lo + 4) {
            *reinterpret_cast<uint32_t*>(to + lo / 2) = prmt(a, b, 0x5410u);
        } else {
            *reinterpret_cast<uint16_t*>(to + lo / 2) = (uint16_t)a;
            *reinterpret_cast<uint16_t*>(to + hi / 2) = (uint16_t)b;
        }
    }
    if (!finite && lane == 0) atomicCAS(g.status, 0, kStatusNonFinite);
}

struct ReadArgs {
    q4lin_kv4_cache_t cache;
    q4lin_kv_read_t a;
    int page_shift, tokens_each;
    int* status;
};

template <int D, int DT>
__global__ void __launch_bounds__(32 * kWarps) kv4_read_kernel(const ReadArgs g) {
    constexpr int U = D / 8, R = 32 / U;
    const q4lin_kv4_cache_t& C = g.cache;
    const int lane = threadIdx.x & 31, u = lane % U, sub = lane / U;
    follow_stream();
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && offsets_bad(g.a.offsets, C.batch, g.a.tokens))
        atomicCAS(g.status, 0, kStatusIndex);
    const int64_t t0 = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * g.tokens_each;
    if (t0 >= g.a.tokens) return;
    const int count = (int)min((int64_t)g.tokens_each, g.a.tokens - t0);
    const bool keys = blockIdx.z == 0 && g.a.k;
    const int h = (int)blockIdx.y * R + sub, heads = (int)C.kv_heads;
    const uint8_t* codes = keys ? C.k_codes : C.v_codes;
    const float* scales = keys ? C.k_scales : C.v_scales;
    void* out = keys ? g.a.k : g.a.v;
    bool bad;
    const Place place = place_of(C, g.page_shift, g.a.offsets, g.a.starts, g.a.tokens, t0, count, &bad);
    if (bad) atomicCAS(g.status, 0, kStatusIndex);
    constexpr int kTogether = 4;  // tokens whose loads overlap
#pragma unroll 1
    for (int i0 = 0; i0 < count; i0 += kTogether) {
        uint32_t word[kTogether];
        float scale[kTogether];
        bool in[kTogether];
#pragma unroll
        for (int k = 0; k < kTogether; ++k) {
            const int64_t row0 = __shfl_sync(0xffffffffu, place.row, i0 + k);  // (-1 past `count`)
            in[k] = row0 >= 0 && h < heads;
            const int64_t row = row0 + ((int64_t)h << g.page_shift);
            if (in[k]) word[k] = __ldg(reinterpret_cast<const uint32_t*>(codes + row * (D / 2)) + u), scale[k] = __ldg(scales + row);
        }
#pragma unroll
        for (int k = 0; k < kTogether; ++k) {
            if (!in[k]) continue;
            uint32_t pairs[4];  // channels n and n + 4
            nibbles_f16(word[k], pairs[0], pairs[1], pairs[2], pairs[3]);
            float x[8];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float2 v = fmul2(__half22float2(*reinterpret_cast<const __half2*>(&pairs[n])), make_float2(scale[k], scale[k]));
                x[n] = v.x, x[n + 4] = v.y;
            }
            const int64_t at = ((t0 + i0 + k) * heads + h) * D + 8 * u;
            if constexpr (DT == Q4LIN_DTYPE_F32) {
                store_four(out, DT, at, true, x);
                store_four(out, DT, at + 4, true, x + 4);
            } else {
                *reinterpret_cast<uint4*>(static_cast<unsigned short*>(out) + at) =
                    make_uint4(to_16x2(x[0], x[1], DT), to_16x2(x[2], x[3], DT), to_16x2(x[4], x[5], DT), to_16x2(x[6], x[7], DT));
            }
        }
    }
}

// Tokens of a warp, up to eight: as many as leave `warps` warps.  Measured, 8 heads of 128, one token a warp and as
// many as leave 64, 32, 16, 8 warps an SM: append of 700 tokens in fp32 4.8, 4.8, 4.8, 4.3, 4.2 us, of 4510 17.1, 13.0,
// 11.7, 11.6, 11.6, of 65536 in bf16 219, then 109; read of 700 in fp32 4.2, 4.2, 4.2, 4.6, 4.8, of 4510 16.4, 12.7,
// 13.1, 13.7, 13.5 (in bf16 14.4, 8.9, 6.9, 6.9, 6.9), of 65536 in bf16 175, then 57.
int tokens_each(int64_t tokens, int64_t warps_per_token, int64_t warps) {
    int each = 1;
    while (each < 8 && tokens * warps_per_token > 2 * each * warps) each *= 2;
    return each;
}

template <int D, int DT>
cudaError_t append(AppendArgs& g, bool vec, const LaunchCtx& c) {
    constexpr int kHeads = 32 / (D / 8);
    const unsigned chunks = (unsigned)((g.cache.kv_heads + kHeads - 1) / kHeads);
    g.tokens_each = tokens_each(g.a.tokens, 2 * chunks, 32 * c.sm_count);
    const int64_t groups = (g.a.tokens + g.tokens_each - 1) / g.tokens_each;
    const dim3 grid((unsigned)((groups + kWarps - 1) / kWarps), chunks, 2);
    if (vec) return launch_early(kv4_append_kernel<D, DT, true>, grid, 32 * kWarps, 0, c.stream, g);
    return launch_early(kv4_append_kernel<D, DT, false>, grid, 32 * kWarps, 0, c.stream, g);
}
template <int D, int DT>
cudaError_t read(ReadArgs& g, const LaunchCtx& c) {
    constexpr int kHeads = 32 / (D / 8);
    const unsigned chunks = (unsigned)((g.cache.kv_heads + kHeads - 1) / kHeads), kinds = g.a.k && g.a.v ? 2 : 1;
    g.tokens_each = tokens_each(g.a.tokens, kinds * chunks, 64 * c.sm_count);
    const int64_t groups = (g.a.tokens + g.tokens_each - 1) / g.tokens_each;
    const dim3 grid((unsigned)((groups + kWarps - 1) / kWarps), chunks, kinds);
    return launch_early(kv4_read_kernel<D, DT>, grid, 32 * kWarps, 0, c.stream, g);
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
    bool vec;
    const LaunchCtx& c;
    template <int D, int DT>
    cudaError_t operator()() const { return append<D, DT>(g, vec, c); }
};
struct Read {
    ReadArgs& g;
    const LaunchCtx& c;
    template <int D, int DT>
    cudaError_t operator()() const { return read<D, DT>(g, c); }
};
int shift_of(int64_t page_size) { return page_size == 16 ? 4 : page_size == 32 ? 5 : 6; }

}  // namespace

cudaError_t kv4_append_launch(const q4lin_kv4_cache_t& cache, const q4lin_kv_append_t& a, const LaunchCtx& c) {
    AppendArgs g;
    g.cache = cache;
    g.a = a;
    g.page_shift = shift_of(cache.page_size);
    g.status = c.status_word;
    const bool vec = fours_aligned(a.k, a.dtype, a.k_token_stride, a.k_head_stride) &&
                     fours_aligned(a.v, a.dtype, a.v_token_stride, a.v_head_stride);
    return by_dim_and_type(cache.head_dim, a.dtype, Append{g, vec, c});
}

cudaError_t kv4_read_launch(const q4lin_kv4_cache_t& cache, const q4lin_kv_read_t& a, const LaunchCtx& c) {
    ReadArgs g;
    g.cache = cache;
    g.a = a;
    g.page_shift = shift_of(cache.page_size);
    g.status = c.status_word;
    return by_dim_and_type(cache.head_dim, a.dtype, Read{g, c});
}

}  // namespace q4lin
