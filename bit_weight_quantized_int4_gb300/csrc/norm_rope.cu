// norm_rope.cu -- queries and keys normalised per head and rotated in one pass, and the gradient
// of that.
//
// A pass of a warp takes 32 / (D / 8) heads of one token; a lane holds eight channels of a head (the two
// groups of four that the rotation pairs), and keeps the token's angles and the weights of its channels.
// Forward, a warp takes a token's heads (a part of them where tokens are few); backward, where a warp's
// sums over its rows cost a join, as many CTAs as fit share all passes out evenly.
//
// Bound: memory, for the gradient with bf16 the instructions beside it (half of a warp scheduler's slots).
// Measured: 8192 tokens of 40 heads of 128 in bf16 normalised and rotated in 31 us, 0.81 of a copy's
// bandwidth; their gradient in 52.7 us, 0.72; of 4096 tokens in fp32 30.8 and 43.5 us, 0.81 and 0.86; one
// token 2.6 and 5.6 us, one launch and two.
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

// Passes in flight of a warp.  Forward, in registers (8192 tokens of 40 heads of 128 in bf16): 2 / 3 / 4
// passes 33.3, 32.8, 31.8 us.  Backward, slots of the ring for two bytes an element, the CTA's warps and the
// CTAs of an SM (the same, and 4096 tokens in fp32): 6, 8 and 2 51.8 and 43.7 us; 6, 8 and 3, whose registers
// do not hold a row's work, 65 and 49; 6, 6 and 3 52.7 and 44.5; 8, 4 and 5 52.9 and 44.4; 12, 4 and 4 56 and 44.6.
// With rows in registers, as forward, 55 and 76 us.
constexpr int kAhead = 4, kBackSlots = 6, kBackCtas = 2;
constexpr int kWarps = 4, kBackWarps = 8;

// Bytes from a head to the one that a warp takes next.
struct Steps {
    int64_t x, d, y;
};
struct NormArgs {
    q4lin_norm_rope_t a;
    const void *dq, *dk;  // backward: the gradients that come in
    int64_t dq_token, dq_head, dk_token, dk_head;
    Steps steps[2];  // backward: of queries, of keys
    float* parts;    // backward: [kind][CTA][D] sums of the weights' gradients
    bool vec;            // groups of four elements of all arrays are aligned
    int64_t part_heads;  // of a token's heads, queries' and keys', in a part
    int* status;
};

// What queries (keys) have in memory.
struct Side {
    const void* x;
    void* y;
    const void* d;
    const float* w;
    int64_t xt, xh, yt, yh, dt, dh, heads;
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
    return s;
}

// A lane's eight channels: two groups of four, as pairs.
struct Eight {
    float2 v[4];
};
// Sum over the U lanes of a head.
template <int U>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
    for (int o = U / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int U>
__device__ __forceinline__ float dot(const Eight& a, const Eight& b) {
    float2 sum = fmul2(a.v[0], b.v[0]);
#pragma unroll
    for (int e = 1; e < 4; ++e) sum = ffma2(a.v[e], b.v[e], sum);
    return head_sum<U>(sum.x + sum.y);
}
__device__ __forceinline__ void scale_by(Eight& x, float f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x.v[e] = fmul2(x.v[e], make_float2(f, f));
}
// Sums of x x and of x y.
template <int U>
__device__ __forceinline__ float2 two_sums(const Eight& x, const Eight& y) {
    float2 a = fmul2(x.v[0], x.v[0]), b = fmul2(x.v[0], y.v[0]);
#pragma unroll
    for (int e = 1; e < 4; ++e) a = ffma2(x.v[e], x.v[e], a), b = ffma2(x.v[e], y.v[e], b);
    float2 v = make_float2(a.x + a.y, b.x + b.y);
#pragma unroll
    for (int o = U / 2; o; o >>= 1)
        v = fadd2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
    return v;
}
// Whether the squares of a row, which add up to `sum`, pass fp32's range, or are lost below it where eps
// does not hide that.
__device__ __forceinline__ bool is_far(float sum, float eps) { return sum > 3e38f || (eps < 1e-30f && sum < 1e-30f); }
// Such a row's x scaled by a power of two (*back), and r = 1 / sqrt(mean x^2 + eps) of that.  By a whole warp:
// the sum needs every lane.
template <int D>
__device__ __forceinline__ void scale_far(Eight& x, bool far, float sum, float eps, float* r, float* back) {
    const float by = sum > 3e38f ? 8.470329472543003e-22f : 1.2676506002282294e30f;  // 2^-70, 2^100
    if (far) scale_by(x, by);
    const float again = dot<D / 8>(x, x);
    if (far) *r = rsqrtf(fmaf(again, 1.f / D, eps * by * by)), *back = by;
}
// Whether one of a lane's elements is not 0.
__device__ __forceinline__ bool any_of(const Eight& x) {
    uint32_t bits = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) bits |= __float_as_uint(x.v[e].x) | __float_as_uint(x.v[e].y);
    return bits << 1 != 0;
}
// x becomes x r.
template <int D>
__device__ __forceinline__ void normalise(Eight& x, float eps) {
    const float sum = dot<D / 8>(x, x);
    float r = rsqrtf(fmaf(sum, 1.f / D, eps)), back;
    const bool far = is_far(sum, eps);
    if (__any_sync(0xffffffffu, far)) scale_far<D>(x, far, sum, eps, &r, &back);
    scale_by(x, r);
}
template <bool VEC>
__device__ __forceinline__ Eight load_weight(const float* w, int lo, int hi) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 1.f;
    if (w) {
        load_four(w, Q4LIN_DTYPE_F32, lo, VEC, v);
        load_four(w, Q4LIN_DTYPE_F32, hi, VEC, v + 4);
    }
    return {make_float2(v[0], v[1]), make_float2(v[2], v[3]), make_float2(v[4], v[5]), make_float2(v[6], v[7])};
}

// A lane's eight elements as they lie in memory, by ordinary loads: outputs may lie where the inputs
// are.  VEC: groups of four are aligned.
template <int DT, bool VEC>
struct Raw {
    uint2 w[DT == Q4LIN_DTYPE_F32 ? 4 : 2];

    // Groups at p + lo and p + hi (bytes); zeros where the lane has no row.
    __device__ __forceinline__ void load(const char* p, int lo, int hi, bool in) {
        constexpr int kGroup = DT == Q4LIN_DTYPE_F32 ? 2 : 1;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const char* from = p + (g ? hi : lo);
#pragma unroll
            for (int e = 0; e < kGroup; ++e) w[g * kGroup + e] = make_uint2(0u, 0u);
            if (!in) continue;
            if constexpr (VEC && DT == Q4LIN_DTYPE_F32) {
                const uint4 v = *reinterpret_cast<const uint4*>(from);
                w[2 * g] = make_uint2(v.x, v.y), w[2 * g + 1] = make_uint2(v.z, v.w);
            } else if constexpr (VEC) {
                w[g] = *reinterpret_cast<const uint2*>(from);
            } else if constexpr (DT == Q4LIN_DTYPE_F32) {
                const uint32_t* f = reinterpret_cast<const uint32_t*>(from);
                w[2 * g] = make_uint2(f[0], f[1]), w[2 * g + 1] = make_uint2(f[2], f[3]);
            } else {
                const unsigned short* b = reinterpret_cast<const unsigned short*>(from);
                w[g] = make_uint2(b[0] | (uint32_t)b[1] << 16, b[2] | (uint32_t)b[3] << 16);
            }
        }
    }
    __device__ __forceinline__ Eight unpack() const {
        Eight x;
        if constexpr (DT == Q4LIN_DTYPE_F32) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x.v[e] = make_float2(__uint_as_float(w[e].x), __uint_as_float(w[e].y));
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) x.v[2 * e] = unpack2(w[e].x, DT), x.v[2 * e + 1] = unpack2(w[e].y, DT);
        }
        return x;
    }
};

// The token's position, and whether it is in the table (else reported, and one that is).
__device__ __forceinline__ int64_t position_of(const NormArgs& g, int64_t token, bool* good) {
    *good = true;
    if (!g.a.rope.cos) return 0;
    const int64_t position = __ldg(g.a.positions + token);
    *good = position >= 0 && position < g.a.rope.positions;
    if (!*good && (threadIdx.x & 31) == 0) atomicCAS(g.status, 0, kStatusIndex);
    return *good ? position : 0;
}

// The rotation by the four angles of a lane, of pairs (channel, channel half the rotated ones further)
// or of neighbours.
struct Angles {
    float2 c[2], s[2];
};
__device__ __forceinline__ void turn(const q4lin_rope_t& r, const Angles& a, Eight& x) {
    if (r.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float c = e % 2 ? a.c[e / 2].y : a.c[e / 2].x, s = e % 2 ? a.s[e / 2].y : a.s[e / 2].x;
            const float2 v = x.v[e];
            x.v[e] = make_float2(fmaf(v.x, c, -(v.y * s)), fmaf(v.y, c, v.x * s));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float2 p = x.v[e], q = x.v[2 + e], minus = make_float2(-a.s[e].x, -a.s[e].y);
            x.v[e] = ffma2(p, a.c[e], fmul2(q, minus)), x.v[2 + e] = ffma2(q, a.c[e], fmul2(p, a.s[e]));
        }
    }
}
__device__ __forceinline__ Angles angles_of(const q4lin_rope_t& r, int64_t position, int u, float sign) {
    float c[4], s[4];
    rope_load(r, position, u, c, s);
    return {{make_float2(c[0], c[1]), make_float2(c[2], c[3])},
            {make_float2(sign * s[0], sign * s[1]), make_float2(sign * s[2], sign * s[3])}};
}
template <int DT, bool VEC>
__device__ __forceinline__ void store_row(char* p, int lo, int hi, const Eight& x) {
    const float y[8] = {x.v[0].x, x.v[0].y, x.v[1].x, x.v[1].y, x.v[2].x, x.v[2].y, x.v[3].x, x.v[3].y};
    store_four(p + lo, DT, 0, VEC, y);
    store_four(p + hi, DT, 0, VEC, y + 4);
}

// A part's heads: queries [q0, q1) and keys [k0, k1).
struct Heads {
    int64_t q0, q1, k0, k1;
};
__device__ __forceinline__ Heads heads_of(const NormArgs& g, int part) {
    const int64_t all = g.a.heads + g.a.kv_heads, h0 = part * g.part_heads, h1 = min(h0 + g.part_heads, all);
    const int64_t n = g.a.heads;
    return {min(h0, n), min(h1, n), max(h0, n) - n, max(h1, n) - n};
}

template <int D, int DT, int AHEAD, bool VEC>
__global__ void __launch_bounds__(32 * kWarps) norm_rope_kernel(const NormArgs g) {
    constexpr int U = D / 8, R = 32 / U, kSize = (int)dtype_size(DT);
    const int lane = threadIdx.x & 31, u = lane % U, sub = lane / U;
    const int64_t token = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    follow_stream();
    if (token >= g.a.tokens) return;
    bool turned, good = true, first = true;
    int lo, hi;
    rope_channels(g.a.rope, u, &turned, &lo, &hi);
    const int lo_at = lo * kSize, hi_at = hi * kSize;
    const Heads heads = heads_of(g, blockIdx.y);
    Angles angles;
    auto rows = [&](auto keys) {
        const Side s = side_of(g, decltype(keys)::value);
        const int begin = (int)(decltype(keys)::value ? heads.k0 : heads.q0);
        const int end = (int)(decltype(keys)::value ? heads.k1 : heads.q1);
        if (begin >= end) return;
        Raw<DT, VEC> raw[AHEAD];
        const char* x_at = static_cast<const char*>(s.x) + (token * s.xt + (begin + sub) * s.xh) * kSize;
        char* y_at = static_cast<char*>(s.y) + (token * s.yt + (begin + sub) * s.yh) * kSize;
        const int64_t x_step = R * s.xh * kSize, y_step = R * s.yh * kSize;
        auto fetch = [&](Raw<DT, VEC>& r, int h) {
            r.load(x_at, lo_at, hi_at, h < end);
            x_at += x_step;
        };
#pragma unroll
        for (int p = 0; p < AHEAD; ++p) fetch(raw[p], begin + sub + p * R);
        const Eight w = load_weight<VEC>(s.w, lo, hi);
        if (first) {  // (behind the first rows' loads)
            const int64_t position = position_of(g, token, &good);
            if (turned) angles = angles_of(g.a.rope, position, u, 1.f);
            first = false;
        }
#pragma unroll 1
        for (int h0 = begin; h0 < end; h0 += AHEAD * R) {
#pragma unroll
            for (int p = 0; p < AHEAD; ++p) {
                const int hp = h0 + p * R, h = hp + sub;
                if (hp >= end) break;
                Eight x = raw[p].unpack();
                fetch(raw[p], h + AHEAD * R);
                normalise<D>(x, g.a.eps);
#pragma unroll
                for (int e = 0; e < 4; ++e) x.v[e] = fmul2(x.v[e], w.v[e]);
                if (turned) turn(g.a.rope, angles, x);
                if (h < end && good) store_row<DT, VEC>(y_at, lo_at, hi_at, x);
                y_at += y_step;
            }
        }
    };
    rows(std::false_type{});
    rows(std::true_type{});
}

// Rows of x and dy on their way to a lane: copies to a ring in shared memory that only the lane reads
// (VEC), so that many rows of a warp are in flight without a register for any.  Else the next row's
// elements in registers: there is no copy of two bytes.
template <int DT, bool VEC>
struct Rows {
    static constexpr int kSlots = VEC ? kBackSlots / (DT == Q4LIN_DTYPE_F32 ? 2 : 1) : 1, kGroup = DT == Q4LIN_DTYPE_F32 ? 16 : 8;
    static constexpr int kBytes = VEC ? kSlots * 4 * kGroup * 32 * kBackWarps : 0;
    uint32_t ring;  // the lane's first group of slot 0; groups lie 32 lanes apart
    Raw<DT, VEC> x, d;

    __device__ __forceinline__ void init(void* shared) {
        if constexpr (VEC) {
            const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
            ring = smem_u32(shared) + (warp * kSlots * 4 * 32 + lane) * kGroup;
        }
    }
    // Into slot `to` (rows that there are not leave what was there, which nobody uses).
    __device__ __forceinline__ void fetch(int to, const char* px, const char* pd, int lo, int hi, bool in) {
        if constexpr (VEC) {
            const uint32_t at = ring + to * (4 * 32 * kGroup);
            if (in) {
                cp_async_ca<kGroup>(at, px + lo);
                cp_async_ca<kGroup>(at + 32 * kGroup, px + hi);
                cp_async_ca<kGroup>(at + 64 * kGroup, pd + lo);
                cp_async_ca<kGroup>(at + 96 * kGroup, pd + hi);
            }
            cp_async_commit();
        } else {
            x.load(px, lo, hi, in), d.load(pd, lo, hi, in);
        }
    }
    __device__ __forceinline__ void read(int from, Eight& ex, Eight& ed) {
        if constexpr (VEC) {
            cp_async_wait_group<kSlots - 2>();
            const uint32_t at = ring + from * (4 * 32 * kGroup);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                lds_group(x, g, at + g * 32 * kGroup);
                lds_group(d, g, at + (2 + g) * 32 * kGroup);
            }
        }
        ex = x.unpack(), ed = d.unpack();
    }
    static __device__ __forceinline__ void lds_group(Raw<DT, VEC>& r, int g, uint32_t at) {
        if constexpr (DT == Q4LIN_DTYPE_F32)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(r.w[2 * g].x), "=r"(r.w[2 * g].y), "=r"(r.w[2 * g + 1].x), "=r"(r.w[2 * g + 1].y)
                         : "r"(at)
                         : "memory");
        else
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.w[g].x), "=r"(r.w[g].y) : "r"(at) : "memory");
    }
};

// A warp takes a stretch of the (token, R heads) of queries, then of keys, all warps equally many, with
// the weights' sums in registers.
template <int D, int DT, bool VEC>
__global__ void __launch_bounds__(32 * kBackWarps, kBackCtas) norm_rope_backward_kernel(const NormArgs g) {
    constexpr int U = D / 8, R = 32 / U, kSize = (int)dtype_size(DT);
    using Ring = Rows<DT, VEC>;
    constexpr int kSums = kBackWarps * R * D * 4;
    __shared__ __align__(16) char shared[Ring::kBytes > kSums ? Ring::kBytes : kSums];
    float(*sums)[D] = reinterpret_cast<float(*)[D]>(shared);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, u = lane % U, sub = lane / U;
    follow_stream();  // (so does the kernel that joins the sums)
    bool turned;
    int lo, hi;
    rope_channels(g.a.rope, u, &turned, &lo, &hi);
    const int lo_at = lo * kSize, hi_at = hi * kSize;
    Ring ring;
    ring.init(shared);
    auto rows = [&](auto keys) {
        constexpr bool kKeys = decltype(keys)::value;
        const Side s = side_of(g, kKeys);
        const int heads = (int)s.heads, each = (heads + R - 1) / R;  // passes of a token
        const int64_t all = g.a.tokens * each, warps = (int64_t)gridDim.x * kBackWarps;
        const int64_t w0 = (int64_t)blockIdx.x * kBackWarps + warp;
        const int64_t share = all / warps, more = all % warps;
        int left = (int)(share + (w0 < more));
        const Eight w = load_weight<VEC>(s.w, lo, hi);
        Eight dw;
#pragma unroll
        for (int e = 0; e < 4; ++e) dw.v[e] = make_float2(0.f, 0.f);
        if (left > 0) {
            const int64_t first = w0 * share + min(w0, more);
            int64_t token = first / each, next_token = token;  // of the row worked on, of the one fetched next
            int h = (int)(first - token * each) * R + sub, next_h = h, to_fetch = left;
            const Steps& step = g.steps[kKeys];  // from R heads to the next
            const char *x_at, *d_at;
            char* y_at;
            auto place = [&](const void* p, int64_t t, int64_t at, int64_t hs, int head) {
                return static_cast<const char*>(p) + (t * at + head * hs) * kSize;
            };
            x_at = place(s.x, token, s.xt, s.xh, h), d_at = place(s.d, token, s.dt, s.dh, h);
            y_at = const_cast<char*>(place(s.y, token, s.yt, s.yh, h));
            auto fetch = [&](int to) {
                ring.fetch(to, x_at, d_at, lo_at, hi_at, to_fetch > 0 && next_h < heads);
                --to_fetch, next_h += R, x_at += step.x, d_at += step.d;
                if (next_h >= each * R) {
                    next_h = sub, ++next_token;
                    x_at = place(s.x, next_token, s.xt, s.xh, sub), d_at = place(s.d, next_token, s.dt, s.dh, sub);
                }
            };
            constexpr int kFirst = VEC ? Ring::kSlots - 1 : 1;
#pragma unroll
            for (int p = 0; p < kFirst; ++p) fetch(p);
            int slot = 0, into = kFirst;
            bool good = true, next_good = true;
            int next = (int)position_of(g, token, &next_good);
            Angles angles;
            bool begins = true;
#pragma unroll 1
            for (; left > 0; --left) {
                if (begins) {
                    if (turned) angles = angles_of(g.a.rope, next, u, -1.f);  // back
                    good = next_good, begins = false;
                    ++token;
                    if (token < g.a.tokens) next = (int)position_of(g, token, &next_good);
                }
                const bool in = h < heads && good;
                Eight x, d;
                ring.read(slot, x, d);
                // (The slot written to is the one read last time, whose row has been stored since.)
                fetch(into);
                if constexpr (VEC) {
                    into = slot, slot = slot + 1 == Ring::kSlots ? 0 : slot + 1;
                }
                if (turned) turn(g.a.rope, angles, d);
                Eight gw;
#pragma unroll
                for (int e = 0; e < 4; ++e) gw.v[e] = fmul2(d.v[e], w.v[e]);
                // Both sums at once; with u = x r, the second is that of g w u over r.  Where x is to be scaled, or
                // the sum leaves fp32's range, or terms may be lost below it, it is taken anew with u.
                const float2 both = two_sums<U>(x, gw);
                float r = rsqrtf(fmaf(both.x, 1.f / D, g.a.eps)), back = 1.f, mean = both.y * (1.f / D) * r;
                const bool far = is_far(both.x, g.a.eps);
                const bool lost = in && (far || !(fabsf(both.y) <= 3e38f) || fabsf(both.y) < 1e-30f);
                // (Padding's gradients are zeros, and so is their sum.)
                if (__any_sync(0xffffffffu, lost) && __any_sync(0xffffffffu, lost && (far || any_of(gw)))) {
                    scale_far<D>(x, far, both.x, g.a.eps, &r, &back);
                    Eight u = x;
                    scale_by(u, r);
                    const float again = dot<U>(u, gw);
                    if (lost) mean = again * (1.f / D);
                }
                scale_by(x, r);
                mean = -mean;
                if (in) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) dw.v[e] = ffma2(d.v[e], x.v[e], dw.v[e]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) x.v[e] = ffma2(x.v[e], make_float2(mean, mean), gw.v[e]);
                scale_by(x, r);
                if (back != 1.f) scale_by(x, back);  // (their product may have no room where a zero has)
                if (in) store_row<DT, VEC>(y_at, lo_at, hi_at, x);
                h += R, y_at += step.y;
                if (h >= each * R) {
                    h = sub, begins = true;
                    y_at = const_cast<char*>(place(s.y, token, s.yt, s.yh, sub));
                }
            }
        }
        // The CTA's sums, the warps' and their rows' in order (where the rings were).
        if constexpr (VEC) cp_async_wait_all();
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e)
            *reinterpret_cast<float2*>(&sums[warp * R + sub][(e < 2 ? lo : hi) + e % 2 * 2]) = dw.v[e];
        __syncthreads();
        for (int d = threadIdx.x; d < D; d += 32 * kBackWarps) {
            float v = 0.f;
#pragma unroll
            for (int j = 0; j < kBackWarps * R; ++j) v += sums[j][d];
            g.parts[(kKeys * (int64_t)gridDim.x + blockIdx.x) * D + d] = v;
        }
        if (!kKeys) __syncthreads();
    };
    rows(std::false_type{});
    rows(std::true_type{});
}

// One CTA for 32 channels of a kind: the CTAs' sums, every 32nd of them by a warp.
__global__ void __launch_bounds__(1024) norm_rope_join_kernel(const float* parts, int ctas, int D, float* dqw, float* dkw) {
    __shared__ float sums[32][33];
    const int kind = blockIdx.y, column = threadIdx.x & 31, stretch = threadIdx.x >> 5, d = blockIdx.x * 32 + column;
    float* to = kind ? dkw : dqw;
    follow_stream();
    if (!to) return;
    float v = 0.f;
#pragma unroll 8
    for (int i = stretch; i < ctas; i += 32) v += __ldcg(parts + ((int64_t)kind * ctas + i) * D + d);
    sums[stretch][column] = v;
    __syncthreads();
    v = sums[column][stretch];  // of channel `stretch`
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (column == 0) to[blockIdx.x * 32 + stretch] = v;
}

// Parts of a token's heads, whole rows of lanes each, so that there are `warps` warps where the
// heads allow.  Measured, 40 heads of 128 in bf16, 4, 16, 32, 64, 128 warps an SM: 200 tokens 4.2, 3.5, 3.5, 3.5, 3.5 us,
// 2048 13.0, 10.6, 11.8, 12.4, 13.7, 8192 30.7, 30.8, 30.8, 32.2, 33.7; 701 of 32 heads 6.9, 4.9, 4.8, 4.9, 6.2, of 40
// heads of 256 in fp32 26.4, 13.2, 13.0, 13.3, 14.4.
unsigned parts_of(NormArgs& g, int64_t row_heads, int64_t warps) {
    const int64_t rows = (g.a.heads + g.a.kv_heads + row_heads - 1) / row_heads;
    const int64_t parts = std::max<int64_t>(1, std::min(std::min(rows, (warps + g.a.tokens - 1) / g.a.tokens), (int64_t)65535));
    const int64_t each = (rows + parts - 1) / parts;
    g.part_heads = each * row_heads;
    return (unsigned)((rows + each - 1) / each);
}

template <int D, int DT>
cudaError_t forward(NormArgs& g, const LaunchCtx& c) {
    const unsigned parts = parts_of(g, 32 / (D / 8), 64 * c.sm_count);
    const dim3 grid((unsigned)((g.a.tokens + kWarps - 1) / kWarps), parts);
    if (g.vec) return launch_early(norm_rope_kernel<D, DT, kAhead, true>, grid, 32 * kWarps, 0, c.stream, g);
    return launch_early(norm_rope_kernel<D, DT, 1, false>, grid, 32 * kWarps, 0, c.stream, g);
}
template <int D, int DT>
cudaError_t backward(NormArgs& g, float* dqw, float* dkw, const LaunchCtx& c) {
    constexpr int kHeads = 32 / (D / 8), kStep = kHeads * (int)dtype_size(DT);
    g.steps[0] = {kStep * g.a.q_head_stride, kStep * g.dq_head, kStep * g.a.q_out_head_stride};
    g.steps[1] = {kStep * g.a.k_head_stride, kStep * g.dk_head, kStep * g.a.k_out_head_stride};
    const int64_t passes = g.a.tokens * ((std::max(g.a.heads, g.a.kv_heads) + kHeads - 1) / kHeads);
    const int64_t ctas = std::max<int64_t>(1, std::min<int64_t>((passes + kBackWarps - 1) / kBackWarps, kBackCtas * c.sm_count));
    if (2 * ctas * D > c.ws_floats) return cudaErrorInvalidValue;
    g.parts = c.ws;
    const auto kernel = g.vec ? norm_rope_backward_kernel<D, DT, true> : norm_rope_backward_kernel<D, DT, false>;
    const cudaError_t e = launch_early(kernel, dim3((unsigned)ctas), 32 * kBackWarps, 0, c.stream, g);
    if (e != cudaSuccess || (!dqw && !dkw)) return e;
    return launch_early(norm_rope_join_kernel, dim3(D / 32, 2), 1024, 0, c.stream, (const float*)g.parts, (int)ctas, D, dqw, dkw);
}

NormArgs args_of(const q4lin_norm_rope_t& a, const LaunchCtx& c) {
    NormArgs g = {};
    g.a = a;
    auto aligned_rows = [&](const void* p, int64_t t, int64_t h, int64_t heads) {
        return heads == 0 || fours_aligned(p, a.dtype, t, h);
    };
    g.vec = aligned_rows(a.q, a.q_token_stride, a.q_head_stride, a.heads) &&
            aligned_rows(a.k, a.k_token_stride, a.k_head_stride, a.kv_heads) &&
            aligned_rows(a.q_out, a.q_out_token_stride, a.q_out_head_stride, a.heads) &&
            aligned_rows(a.k_out, a.k_out_token_stride, a.k_out_head_stride, a.kv_heads) &&
            reinterpret_cast<uintptr_t>(a.q_weight) % 16 == 0 && reinterpret_cast<uintptr_t>(a.k_weight) % 16 == 0;
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
    g.vec = g.vec && (g.a.heads == 0 || fours_aligned(g.dq, g.a.dtype, g.dq_token, g.dq_head)) &&
            (g.a.kv_heads == 0 || fours_aligned(g.dk, g.a.dtype, g.dk_token, g.dk_head));
    if (g.a.head_dim == 64) return backward_typed<64>(g, b.d_q_weight, b.d_k_weight, c);
    if (g.a.head_dim == 128) return backward_typed<128>(g, b.d_q_weight, b.d_k_weight, c);
    return backward_typed<256>(g, b.d_q_weight, b.d_k_weight, c);
}

}  // namespace q4lin
