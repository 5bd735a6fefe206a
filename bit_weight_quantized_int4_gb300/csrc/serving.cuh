// serving.cuh -- device helpers shared by the operators around the linears (kv_append.cu,
// attention.cu, logprobs.cu): typed loads and stores, the position rotation, one-instruction
// exp2 and log2, untiled bulk copies, the warp-level fp16 MMA.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/q4lin.h"
#include "ptx.cuh"

namespace q4lin {
namespace serving {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Codes of the status word (q4lin_check_device_status).
constexpr int kStatusNonFinite = 3;
constexpr int kStatusIndex = 4;

__host__ __device__ constexpr int64_t dtype_size(int dtype) { return dtype == Q4LIN_DTYPE_F32 ? 4 : 2; }

__device__ __forceinline__ float load_one(const void* p, int dtype, int64_t i) {
    if (dtype == Q4LIN_DTYPE_F32) return __ldg(static_cast<const float*>(p) + i);
    const unsigned short b = __ldg(static_cast<const unsigned short*>(p) + i);
    if (dtype == Q4LIN_DTYPE_F16) return __half2float(__ushort_as_half(b));
    return __uint_as_float((uint32_t)b << 16);
}

__device__ __forceinline__ float2 unpack2(uint32_t w, int dtype) {
    if (dtype == Q4LIN_DTYPE_F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Four consecutive elements; `vec`: the address is aligned to the four of them.
__device__ __forceinline__ void load_four(const void* p, int dtype, int64_t i, bool vec, float* x) {
    if (!vec) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = load_one(p, dtype, i + e);
    } else if (dtype == Q4LIN_DTYPE_F32) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i));
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const unsigned short*>(p) + i));
        const float2 a = unpack2(v.x, dtype), b = unpack2(v.y, dtype);
        x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
    }
}

// Rounded to the type, nearest even.
__device__ __forceinline__ unsigned short to_16(float x, int dtype) {
    return dtype == Q4LIN_DTYPE_F16 ? __half_as_ushort(__float2half_rn(x))
                                    : __bfloat16_as_ushort(__float2bfloat16_rn(x));
}
__device__ __forceinline__ uint32_t to_16x2(float a, float b, int dtype) {
    return (uint32_t)to_16(a, dtype) | ((uint32_t)to_16(b, dtype) << 16);
}
__device__ __forceinline__ void store_one(void* p, int dtype, int64_t i, float x) {
    if (dtype == Q4LIN_DTYPE_F32)
        static_cast<float*>(p)[i] = x;
    else
        static_cast<unsigned short*>(p)[i] = to_16(x, dtype);
}

// Row `position` of the rotation for the eight channels of unit u (two groups of four, see
// rope_channels): the four cosines and sines.
__device__ __forceinline__ void rope_load(const q4lin_rope_t& r, int64_t position, int u, float (&c)[4],
                                          float (&s)[4]) {
    const int64_t at = position * (r.rotated / 2) + 4 * u;
    load_four(r.cos, Q4LIN_DTYPE_F32, at, (reinterpret_cast<uintptr_t>(r.cos) & 15) == 0, c);
    load_four(r.sin, Q4LIN_DTYPE_F32, at, (reinterpret_cast<uintptr_t>(r.sin) & 15) == 0, s);
}
// The rotation, each product and sum rounded once.
__device__ __forceinline__ void rope_apply(const q4lin_rope_t& r, const float (&c)[4], const float (&s)[4],
                                           float (&x)[8]) {
    if (r.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float a = x[2 * e], b = x[2 * e + 1];
            x[2 * e] = __fsub_rn(__fmul_rn(a, c[e]), __fmul_rn(b, s[e]));
            x[2 * e + 1] = __fadd_rn(__fmul_rn(b, c[e]), __fmul_rn(a, s[e]));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float a = x[e], b = x[4 + e];
            x[e] = __fsub_rn(__fmul_rn(a, c[e]), __fmul_rn(b, s[e]));
            x[4 + e] = __fadd_rn(__fmul_rn(b, c[e]), __fmul_rn(a, s[e]));
        }
    }
}
__device__ __forceinline__ void rope_unit(const q4lin_rope_t& r, int64_t position, int u, float (&x)[8]) {
    float c[4], s[4];
    rope_load(r, position, u, c, s);
    rope_apply(r, c, s, x);
}
// First channels of the two groups of four of unit u of a head: a rotated pair's two halves
// where the first half is rotated with the second, else eight consecutive channels.
__device__ __forceinline__ void rope_channels(const q4lin_rope_t& r, int u, bool* turned, int* lo, int* hi) {
    *turned = r.cos != nullptr && 8 * u < r.rotated;
    const bool halves = *turned && !r.interleaved;
    *lo = halves ? 4 * u : 8 * u;
    *hi = halves ? (int)(r.rotated / 2) + 4 * u : 8 * u + 4;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The last b in [0, batch) with key(b) <= at, by a 32-way search of one warp.
template <typename Key>
__device__ __forceinline__ int64_t find_sequence(int64_t batch, int64_t at, Key key) {
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, n = batch;
    while (true) {
        const int64_t step = (n + 31) / 32;
        const int64_t b = lo + lane * step;
        const bool below = lane * step < n && key(b) <= at;
        const unsigned m = __ballot_sync(0xffffffffu, below);
        const int last = m ? 31 - __clz(m) : 0;
        const int64_t left = n - last * step;
        lo += last * step;
        n = left < step ? left : step;
        if (step == 1) return lo;
    }
}

// `bytes` (a multiple of 16) from global to this CTA's shared memory, both 16-byte aligned,
// completing on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
        : "memory");
}
// Orders this thread's ordinary shared-memory accesses before later bulk copies there.
__device__ __forceinline__ void fence_async_shared() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// d += a b: a 16 x 16 and b 16 x 8 of fp16, d 16 x 8 of fp32.  Lane (g, t) = (lane / 4,
// lane % 4) holds of a the pairs (row g, k 2t), (g + 8, 2t), (g, 2t + 8), (g + 8, 2t + 8), of
// b (k 2t, column g), (2t + 8, g), and of d (row g, columns 2t, 2t + 1), (g + 8, ...).
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// The four codes of a word as exact fp16 pairs of code - 128: the byte permute builds
// 1024 + code (0x64cc), from which 1152 is subtracted.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t* lo, uint32_t* hi) {
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));
    const uint32_t a = ptx::prmt(w, 0x64646464u, 0x4140u), b = ptx::prmt(w, 0x64646464u, 0x4342u);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), bias);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
    *lo = *reinterpret_cast<const uint32_t*>(&x);
    *hi = *reinterpret_cast<const uint32_t*>(&y);
}
// Two values as fp16 pairs: the rounded values, and what the rounding left (22 bits in all).
__device__ __forceinline__ void split_f16(float a, float b, uint32_t* hi, uint32_t* lo) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 r = __half22float2(h);
    const __half2 l = __floats2half2_rn(a - r.x, b - r.y);
    *hi = *reinterpret_cast<const uint32_t*>(&h);
    *lo = *reinterpret_cast<const uint32_t*>(&l);
}

}  // namespace serving
}  // namespace q4lin
