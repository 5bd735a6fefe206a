// norm_rope.cu -- queries and keys normalised per head and rotated in one pass, and the gradient
// of that.
//
// A warp takes heads of one token, `PASSES` x 32 / (D / 8) of them at a time; a lane holds eight
// channels of a head (the two groups of four that the rotation pairs), and the token's angles and
// the weights of its channels for all of the warp's heads.
//
// Forward, y = R(x r w) with r = 1 / sqrt(mean x^2 + eps); backward, with g = R^T dy and u = x r:
// dw = sum g u, dx = r (g w - u mean(g w u)).  R turns pairs by an angle, so R^T turns them back.
#include <algorithm>

#include "q4lin_internal.h"
#include "serving.cuh"

namespace q4lin {
namespace {
using namespace ptx;
using namespace serving;

constexpr int kWarps = 4;

struct NormArgs {
    q4lin_norm_rope_t a;
    const void *dq, *dk;  // backward: the gradients that come in
    int64_t dq_token, dq_head, dk_token, dk_head;
    float* parts;  // backward: [kind][CTA][D] sums of the weights' gradients
    int q_vec, k_vec, q_out_vec, k_out_vec, dq_vec, dk_vec;
    int64_t q_chunks, chunks;  // of a token's heads
    int* status;
};

// What queries (keys) have in memory.
struct Side {
    const void* x;
    void* y;
    const void* d;
    const float* w;
    int64_t xt, xh, yt, yh, dt, dh, heads;
    bool x_vec, y_vec, d_vec;
};
__device__ __forceinline__ Side side_of(const NormArgs& g, bool keys) {
    Side s;
    s.x = keys ? g.a.k : g.a.q, s.y = keys ? g.a.k_out : g.a.q_out, s.d = keys ? g.dk : g.dq;
    s.w = keys ? g.a.k_weight : g.a.q_weight;
    s.xt = keys ? g.a.k_token_stride : g.a.q_token_stride, s.xh = keys ? g.a.k_head_stride : g.a.q_head_stride;
    s.yt = keys ? g.a.k_out_token_stride : g.a.q_out_token_stride;
    s.yh = keys ? g.a.k_out_head_stride : g.a.q_out_head_stride;
    s.dt = keys ? g.dk_token : g.dq_token, s.dh = keys ? g.dk_head : g.dq_head;
    s.heads = keys ? g.a.kv_heads : g.a.heads;
    s.x_vec = keys ? g.k_vec : g.q_vec, s.y_vec = keys ? g.k_out_vec : g.q_out_vec;
    s.d_vec = keys ? g.dk_vec : g.dq_vec;
    return s;
}

// Sum over the U lanes of a head.
template <int U>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
    for (int o = U / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// x becomes u = x r; the result is r.  Where the squares pass fp32's range, x is scaled by 2^-70
// first (whole warp: the sums need every lane).
template <int D>
__device__ __forceinline__ float normalise(float (&x)[8], float eps) {
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
    sum = head_sum<D / 8>(sum);
    float r = __frsqrt_rn(fmaf(sum, 1.f / D, eps)), back = 1.f;
    if (__any_sync(0xffffffffu, sum > 3e38f)) {
        constexpr float kDown = 8.470329472543003e-22f;  // 2^-70
        const bool far = sum > 3e38f;
        float again = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float y = x[e] * kDown;
            again = fmaf(y, y, again);
            if (far) x[e] = y;
        }
        again = head_sum<D / 8>(again);
        if (far) r = __frsqrt_rn(fmaf(again, 1.f / D, eps * kDown * kDown)), back = kDown;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= r;
    return r * back;
}
__device__ __forceinline__ void load_weight(const float* w, int lo, int hi, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = w ? __ldg(w + (e < 4 ? lo + e : hi + e - 4)) : 1.f;
}

// Four consecutive elements by ordinary loads: outputs may lie where the inputs are.
__device__ __forceinline__ void read_four(const void* p, int dtype, int64_t i, bool vec, float* x) {
    if (dtype == Q4LIN_DTYPE_F32) {
        const float* f = static_cast<const float*>(p) + i;
        if (vec) {
            const float4 v = *reinterpret_cast<const float4*>(f);
            x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = f[e];
        }
        return;
    }
    const unsigned short* b = static_cast<const unsigned short*>(p) + i;
    uint2 v;
    if (vec)
        v = *reinterpret_cast<const uint2*>(b);
    else
        v = make_uint2(b[0] | (uint32_t)b[1] << 16, b[2] | (uint32_t)b[3] << 16);
    const float2 lo = unpack2(v.x, dtype), hi = unpack2(v.y, dtype);
    x[0] = lo.x, x[1] = lo.y, x[2] = hi.x, x[3] = hi.y;
}

// The token's position; false where it is outside the table (reported).
__device__ __forceinline__ bool position_of(const NormArgs& g, int64_t token, int64_t* position) {
    if (!g.a.rope.cos) return true;
    *position = __ldg(g.a.positions + token);
    if (*position >= 0 && *position < g.a.rope.positions) return true;
    if ((threadIdx.x & 31) == 0) atomicCAS(g.status, 0, kStatusIndex);
    return false;
}

template <int D, int DT, int PASSES>
__global__ void __launch_bounds__(32 * kWarps) norm_rope_kernel(const NormArgs g) {
    constexpr int U = D / 8, R = 32 / U;
    const int lane = threadIdx.x & 31, u = lane % U;
    bool turned;
    int lo, hi;
    rope_channels(g.a.rope, u, &turned, &lo, &hi);
    const int64_t items = g.a.tokens * g.chunks;
    for (int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); i < items; i += (int64_t)gridDim.x * kWarps) {
        const int64_t token = i / g.chunks, chunk = i - token * g.chunks;
        const bool keys = chunk >= g.q_chunks;
        const Side s = side_of(g, keys);
        const int64_t h0 = (keys ? chunk - g.q_chunks : chunk) * (PASSES * R) + lane / U;
        float x[PASSES][8], c[4], sn[4], w[8];
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[p][e] = 0.f;
            const int64_t h = h0 + p * R, at = token * s.xt + h * s.xh;
            if (h < s.heads) {
                read_four(s.x, DT, at + lo, s.x_vec, x[p]);
                read_four(s.x, DT, at + hi, s.x_vec, x[p] + 4);
            }
        }
        load_weight(s.w, lo, hi, w);
        int64_t position = 0;
        if (!position_of(g, token, &position)) continue;
        if (turned) rope_load(g.a.rope, position, u, c, sn);
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int64_t h = h0 + p * R, at = token * s.yt + h * s.yh;
            normalise<D>(x[p], g.a.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[p][e] *= w[e];
            if (turned) rope_apply(g.a.rope, c, sn, x[p]);
            if (h < s.heads) {
                store_four(s.y, DT, at + lo, s.y_vec, x[p]);
                store_four(s.y, DT, at + hi, s.y_vec, x[p] + 4);
            }
        }
    }
}

// CTAs of a kind (queries, keys) walk over its items with the weights' sums in registers.
template <int D, int DT, int PASSES>
__global__ void __launch_bounds__(32 * kWarps) norm_rope_backward_kernel(const NormArgs g) {
    constexpr int U = D / 8, R = 32 / U;
    __shared__ float sums[kWarps * R][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, u = lane % U;
    griddep_launch_dependents();  // (the kernel that joins the sums waits for this one's end)
    bool turned;
    int lo, hi;
    rope_channels(g.a.rope, u, &turned, &lo, &hi);
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {
        const Side s = side_of(g, kind == 1);
        const int64_t chunks = kind ? g.chunks - g.q_chunks : g.q_chunks, items = g.a.tokens * chunks;
        float w[8], dw[8];
        load_weight(s.w, lo, hi, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[e] = 0.f;
        for (int64_t i = (int64_t)blockIdx.x * kWarps + warp; i < items; i += (int64_t)gridDim.x * kWarps) {
            const int64_t token = i / chunks, h0 = (i - token * chunks) * (PASSES * R) + lane / U;
            float x[PASSES][8], d[PASSES][8], c[4], sn[4];
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[p][e] = d[p][e] = 0.f;
                const int64_t h = h0 + p * R, at = token * s.xt + h * s.xh, dat = token * s.dt + h * s.dh;
                if (h < s.heads) {
                    read_four(s.x, DT, at + lo, s.x_vec, x[p]);
                    read_four(s.x, DT, at + hi, s.x_vec, x[p] + 4);
                    read_four(s.d, DT, dat + lo, s.d_vec, d[p]);
                    read_four(s.d, DT, dat + hi, s.d_vec, d[p] + 4);
                }
            }
            int64_t position = 0;
            if (!position_of(g, token, &position)) continue;
            if (turned) {
                rope_load(g.a.rope, position, u, c, sn);
#pragma unroll
                for (int e = 0; e < 4; ++e) sn[e] = -sn[e];  // back
            }
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                const int64_t h = h0 + p * R, at = token * s.yt + h * s.yh;
                const float r = normalise<D>(x[p], g.a.eps);
                if (turned) rope_apply(g.a.rope, c, sn, d[p]);
                float dot = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (h < s.heads) dw[e] = fmaf(d[p][e], x[p][e], dw[e]);
                    d[p][e] *= w[e];
                    dot = fmaf(d[p][e], x[p][e], dot);
                }
                dot = head_sum<U>(dot) * (1.f / D);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[p][e] = r * fmaf(-x[p][e], dot, d[p][e]);
                if (h < s.heads) {
                    store_four(s.y, DT, at + lo, s.y_vec, x[p]);
                    store_four(s.y, DT, at + hi, s.y_vec, x[p] + 4);
                }
            }
        }
        // The CTA's sums, the warps' and their rows' in order.
        if (kind) __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[warp * R + lane / U][e < 4 ? lo + e : hi + e - 4] = dw[e];
        __syncthreads();
        for (int d = threadIdx.x; d < D; d += 32 * kWarps) {
            float v = 0.f;
            for (int j = 0; j < kWarps * R; ++j) v += sums[j][d];
            g.parts[((int64_t)kind * gridDim.x + blockIdx.x) * D + d] = v;
        }
    }
}

// One CTA for 32 channels of a kind: the CTAs' sums, 8 stretches of them at a time.
__global__ void __launch_bounds__(256) norm_rope_join_kernel(const float* parts, int ctas, int D, float* dqw, float* dkw) {
    __shared__ float sums[8][32];
    const int kind = blockIdx.y, column = threadIdx.x & 31, stretch = threadIdx.x >> 5, d = blockIdx.x * 32 + column;
    float* to = kind ? dkw : dqw;
    griddep_wait();
    if (!to) return;
    float v = 0.f;
    for (int i = stretch; i < ctas; i += 8) v += __ldcg(parts + ((int64_t)kind * ctas + i) * D + d);
    sums[stretch][column] = v;
    __syncthreads();
    if (stretch) return;
#pragma unroll
    for (int j = 1; j < 8; ++j) v += sums[j][column];
    to[d] = v;
}

template <int D, int DT>
cudaError_t forward(NormArgs& g, const LaunchCtx& c) {
    constexpr int kPasses = 1, kHeads = kPasses * 32 / (D / 8);
    g.q_chunks = (g.a.heads + kHeads - 1) / kHeads;
    g.chunks = g.q_chunks + (g.a.kv_heads + kHeads - 1) / kHeads;
    const int64_t blocks = (g.a.tokens * g.chunks + kWarps - 1) / kWarps;
    norm_rope_kernel<D, DT, kPasses><<<(unsigned)std::min<int64_t>(blocks, 1 << 30), 32 * kWarps, 0, c.stream>>>(g);
    return cudaGetLastError();
}
template <int D, int DT>
cudaError_t backward(NormArgs& g, float* dqw, float* dkw, const LaunchCtx& c) {
    constexpr int kPasses = 1, kHeads = kPasses * 32 / (D / 8);
    g.q_chunks = (g.a.heads + kHeads - 1) / kHeads;
    g.chunks = g.q_chunks + (g.a.kv_heads + kHeads - 1) / kHeads;
    const int64_t blocks = (g.a.tokens * std::max(g.q_chunks, g.chunks - g.q_chunks) + kWarps - 1) / kWarps;
    const unsigned grid = (unsigned)std::min<int64_t>(blocks, 8 * c.sm_count);
    if ((int64_t)2 * grid * D > c.ws_floats) return cudaErrorInvalidValue;
    g.parts = c.ws;
    norm_rope_backward_kernel<D, DT, kPasses><<<grid, 32 * kWarps, 0, c.stream>>>(g);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (!dqw && !dkw)) return e;
    // Its launch overlaps the first kernel; it waits for that one's end on the device.
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(D / 32, 2);
    cfg.blockDim = dim3(256);
    cfg.stream = c.stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_rope_join_kernel, (const float*)g.parts, (int)grid, D, dqw, dkw);
}

NormArgs args_of(const q4lin_norm_rope_t& a, const LaunchCtx& c) {
    NormArgs g = {};
    g.a = a;
    g.q_vec = fours_aligned(a.q, a.dtype, a.q_token_stride, a.q_head_stride);
    g.k_vec = fours_aligned(a.k, a.dtype, a.k_token_stride, a.k_head_stride);
    g.q_out_vec = fours_aligned(a.q_out, a.dtype, a.q_out_token_stride, a.q_out_head_stride);
    g.k_out_vec = fours_aligned(a.k_out, a.dtype, a.k_out_token_stride, a.k_out_head_stride);
    g.status = c.status_word;
    return g;
}
template <int D>
cudaError_t forward_typed(NormArgs& g, const LaunchCtx& c) {
    if (g.a.dtype == Q4LIN_DTYPE_F32) return forward<D, Q4LIN_DTYPE_F32>(g, c);
    if (g.a.dtype == Q4LIN_DTYPE_F16) return forward<D, Q4LIN_DTYPE_F16>(g, c);
    return forward<D, Q4LIN_DTYPE_BF16>(g, c);
}
template <int D>
cudaError_t backward_typed(NormArgs& g, float* dqw, float* dkw, const LaunchCtx& c) {
    if (g.a.dtype == Q4LIN_DTYPE_F32) return backward<D, Q4LIN_DTYPE_F32>(g, dqw, dkw, c);
    if (g.a.dtype == Q4LIN_DTYPE_F16) return backward<D, Q4LIN_DTYPE_F16>(g, dqw, dkw, c);
    return backward<D, Q4LIN_DTYPE_BF16>(g, dqw, dkw, c);
}

}  // namespace

cudaError_t norm_rope_launch(const q4lin_norm_rope_t& a, const LaunchCtx& c) {
    NormArgs g = args_of(a, c);
    if (a.head_dim == 64) return forward_typed<64>(g, c);
    if (a.head_dim == 128) return forward_typed<128>(g, c);
    return forward_typed<256>(g, c);
}

cudaError_t norm_rope_backward_launch(const q4lin_norm_rope_backward_t& b, const LaunchCtx& c) {
    NormArgs g = args_of(b.forward, c);
    g.dq = b.d_q_out, g.dk = b.d_k_out;
    g.dq_token = b.d_q_out_token_stride, g.dq_head = b.d_q_out_head_stride;
    g.dk_token = b.d_k_out_token_stride, g.dk_head = b.d_k_out_head_stride;
    g.dq_vec = fours_aligned(g.dq, g.a.dtype, g.dq_token, g.dq_head);
    g.dk_vec = fours_aligned(g.dk, g.a.dtype, g.dk_token, g.dk_head);
    if (g.a.head_dim == 64) return backward_typed<64>(g, b.d_q_weight, b.d_k_weight, c);
    if (g.a.head_dim == 128) return backward_typed<128>(g, b.d_q_weight, b.d_k_weight, c);
    return backward_typed<256>(g, b.d_q_weight, b.d_k_weight, c);
}

}  // namespace q4lin
