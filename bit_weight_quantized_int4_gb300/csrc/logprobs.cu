// logprobs.cu -- per row of logits: log-sum-exp, a given token's log probability, entropy and
// the largest entries; and the gradient of the log probability and the entropy.
//
// Bound: the logits, read once (and the gradient written once); few rows are cut over
// several CTAs, whose results the last one to arrive joins through the handle's workspace.
//
// One pass keeps, per thread, m = the largest entry so far, l = sum e^(x - m) and
// t = sum e^(x - m) (x - m): lse = m + ln l, entropy = ln l - t / l.  The top entries cost
// little on the way: each thread notes the maxima of eight stretches of its entries; of 32
// groups of stretches, the k-th largest of the groups' maxima bounds the k-th largest entry
// from below, and only stretches whose maximum reaches that bound (about 32 ln(32 / (32 - k))
// of 2048 in a row in no order) are looked at again, from L2.
//
// Measured (fp32, 128257 entries): 1000 rows, 513 MB, with 20 top entries 95 us: 5.4 TB/s, 0.80 of
// a copy's bandwidth (8 % of the row is read from memory a second time, and 1000 CTAs are 1.6
// rounds); one row 8.2 us, the join of its 32 CTAs and the chain of the top entries.  The gradient
// of 1000 rows, 1026 MB, 158 us: 6.5 TB/s, 0.96; of 8 rows of 128256 bf16 entries 3.0 us.
#include <algorithm>

#include "q4lin_internal.h"
#include "serving.cuh"

namespace q4lin {
namespace {
using namespace serving;

constexpr int kThreads = 256;
constexpr int kCtas = 4;  // per SM
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTop = 32;
constexpr int kStretches = 8;
constexpr int kMaxSplits = 32;
// Stands in for differences x - m below it (a mask's lowest value, -infinity): its exponential
// is 0 in fp32 as theirs is, and its products with sums stay finite.
constexpr float kNegative = -1.0e4f;

struct LpArgs {
    q4lin_logprobs_t a;
    int splits;        // CTAs per row
    int64_t chunk;     // entries per CTA, a multiple of 8
    float* ws;         // [rows][splits] of LpPart
    int* tickets;      // [rows]
    int* status;
};
// A CTA's share of a row.
struct LpPart {
    float m, l, t;
    int pad;
    unsigned long long top[kMaxTop];
};

// Order of the entries: larger is larger or, of equal ones, has the lower index.  A NaN is
// above everything.
__device__ __forceinline__ unsigned long long order_key(float x, uint32_t index) {
    const uint32_t b = __float_as_uint(x);
    uint32_t k = b & 0x80000000u ? ~b : b | 0x80000000u;
    if (x != x) k = 0xFFFFFFFFu;
    if (x == 0.f) k = 0x80000000u;  // -0 and +0 are equal
    return ((unsigned long long)k << 32) | (uint32_t)~index;
}
__device__ __forceinline__ float key_value(unsigned long long key) {
    const uint32_t k = (uint32_t)(key >> 32);
    if (k == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ uint32_t key_index(unsigned long long key) { return ~(uint32_t)key; }

// (m, l, t) joined with (m2, l2, t2).  With nothing seen, m is -infinity and l, t are 0.
__device__ __forceinline__ void join(float& m, float& l, float& t, float m2, float l2, float t2) {
    const float top = fmaxf(m, m2);
    if (top == -INFINITY) return;
    // (An infinite maximum leaves l = 0: lse is infinite, everything else becomes NaN.)
    const float d = fmaxf(m - top, kNegative), d2 = fmaxf(m2 - top, kNegative);
    const float a = ex2(d * kLog2e), a2 = ex2(d2 * kLog2e);
    t = a * fmaf(l, d, t) + a2 * fmaf(l2, d2, t2);
    l = l * a + l2 * a2;
    m = top;
}

// Eight entries of 16-bit logits or four of fp32 at a time where the row's address allows.
template <int DT>
struct Vec {
    static constexpr int N = DT == Q4LIN_DTYPE_F32 ? 4 : 8;
    static __device__ __forceinline__ void load(const void* p, int64_t i, float* x) {
        widen(__ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * dtype_size(DT))), x);
    }
    // Where the same kernel writes to the place afterwards.
    static __device__ __forceinline__ void load_before_store(const void* p, int64_t i, float* x) {
        widen(*reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * dtype_size(DT)), x);
    }
    static __device__ __forceinline__ void widen(const uint4& v, float* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (DT == Q4LIN_DTYPE_F32) {
                x[j] = __uint_as_float(w[j]);
            } else {
                const float2 f = unpack2(w[j], DT);
                x[2 * (j % 4)] = f.x, x[2 * (j % 4) + 1] = f.y;
            }
        }
    }
};

// A CTA's entries [begin, end) of a row: `head` single ones up to a 16-byte boundary, then
// vectors, then single ones.  Thread i takes single entry i, and vectors i, i + kThreads, ...
template <int DT>
struct Span {
    const void* row;
    int64_t begin, end, vec0, vecs;
    __device__ Span(const void* p, int64_t b, int64_t e) : row(p), begin(b), end(e) {
        constexpr int size = (int)dtype_size(DT), N = Vec<DT>::N;
        const uintptr_t at = reinterpret_cast<uintptr_t>(p) + b * size;
        const int64_t head = ((16 - (at & 15)) & 15) / size;
        vec0 = min(b + head, e);
        vecs = (e - vec0) / N;
    }
    __device__ int64_t tail() const { return vec0 + vecs * Vec<DT>::N; }
    // Single entries: those before the vectors, then those after.
    __device__ int singles() const { return (int)((vec0 - begin) + (end - tail())); }
    __device__ int64_t single(int i) const {
        const int head = (int)(vec0 - begin);
        return i < head ? begin + i : tail() + (i - head);
    }
};

template <int DT>
__global__ void __launch_bounds__(kThreads, kCtas) logprobs_kernel(const LpArgs g) {
    constexpr int N = Vec<DT>::N, kAhead = DT == Q4LIN_DTYPE_F32 ? 4 : 2;  // 16 entries a round
    constexpr int kCandidates = 2048;
    __shared__ unsigned long long s_cand[kCandidates], s_key[kMaxSplits], s_thr, s_top[kMaxTop];
    __shared__ float s_bound, s_m[kWarps], s_l[kWarps], s_t[kWarps], s_mx[kStretches][kThreads];
    __shared__ unsigned short s_owner[kStretches * kThreads];
    __shared__ int s_owners, s_above, s_ties, s_last;
    const int64_t row = blockIdx.x / g.splits;
    const int split = (int)(blockIdx.x % g.splits);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, K = (int)g.a.top;
    const char* base = static_cast<const char*>(g.a.logits) + row * g.a.row_stride * dtype_size(DT);
    const Span<DT> span(base, split * g.chunk, min(g.a.vocabulary, (split + 1) * g.chunk));

    // ---- one pass: m, l and t
    float m = -INFINITY, l = 0.f, t = 0.f;
    bool nan = false;
    auto rescale = [&](float top) {
        if (m != -INFINITY) {
            const float d = fmaxf(m - top, kNegative), a = ex2(d * kLog2e);
            t = a * fmaf(l, d, t);
            l *= a;
        }
        m = top;
    };
    auto add = [&](float x) {
        const float d = fmaxf(x - m, kNegative), e = ex2(d * kLog2e);  // a NaN adds nothing here
        l += e;
        t = fmaf(e, d, t);
    };
    // A round's vectors are asked for while the round before is added.
    float ahead[kAhead][N];
    auto load = [&](int64_t v) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t at = v + i * kThreads;
            if (at < span.vecs) {
                Vec<DT>::load(base, span.vec0 + at * N, ahead[i]);
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e) ahead[i][e] = -INFINITY;
            }
        }
    };
    // A stretch: `per` rounds of a thread.
    const int rounds = (int)((span.vecs + kThreads * kAhead - 1) / (kThreads * kAhead));
    const int per = max(1, (rounds + kStretches - 1) / kStretches);
    float stretch = -INFINITY, *note = &s_mx[0][tid];
    int left = per;
#pragma unroll
    for (int i = 0; i < kStretches; ++i) s_mx[i][tid] = -INFINITY;
    load(tid);
    for (int64_t v = tid; v < span.vecs; v += kThreads * kAhead) {
        float x[kAhead][N];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int e = 0; e < N; ++e) x[i][e] = ahead[i][e];
        load(v + kThreads * kAhead);
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int e = 0; e < N; ++e) {
                top = fmaxf(top, x[i][e]);
                nan |= x[i][e] != x[i][e];
            }
        if (top > m) rescale(top);
        if (m != -INFINITY) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
#pragma unroll
                for (int e = 0; e < N; ++e) add(x[i][e]);
        }
        stretch = fmaxf(stretch, top);
        if (--left == 0) *note = stretch, note += kThreads, left = per, stretch = -INFINITY;
    }
    if (left < per) *note = stretch;
    if (tid < span.singles()) {
        const float x = load_one(base, DT, span.single(tid));
        nan |= x != x;
        if (x > m) rescale(x);
        if (m != -INFINITY) add(x);
        s_mx[0][tid] = fmaxf(s_mx[0][tid], x);  // single entries count with the first stretch
    }
    const bool any_nan = __syncthreads_or(nan);

    // ---- the CTA's m, l, t
    float rm = m, rl = l, rt = t;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, rm, o), l2 = __shfl_xor_sync(0xffffffffu, rl, o),
                    t2 = __shfl_xor_sync(0xffffffffu, rt, o);
        join(rm, rl, rt, m2, l2, t2);
    }
    if (lane == 0) s_m[warp] = rm, s_l[warp] = rl, s_t[warp] = rt;
    if (tid == 0) s_owners = s_above = s_ties = 0;
    __syncthreads();
    rm = s_m[0], rl = s_l[0], rt = s_t[0];
    for (int w = 1; w < kWarps; ++w) join(rm, rl, rt, s_m[w], s_l[w], s_t[w]);
    if (any_nan) rm = fmaxf(rm, 0.f), rl = rt = __uint_as_float(0x7FC00000u);

    // ---- the CTA's `mine` largest entries (it may hold fewer than K)
    const int mine = (int)min((int64_t)K, span.end - span.begin);
    if (K > 0) {
        // The bound: group = lane, over the warps and stretches.
        if (warp == 0) {
            float group = -INFINITY;
#pragma unroll
            for (int i = 0; i < kStretches; ++i)
#pragma unroll
                for (int w = 0; w < kWarps; ++w) group = fmaxf(group, s_mx[i][w * 32 + lane]);
            int rank = 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float other = __shfl_sync(0xffffffffu, group, i);
                rank += other > group || (other == group && i < lane);
            }
            if (rank == mine - 1) s_bound = group;
        }
        __syncthreads();
        const float bound = s_bound;
#pragma unroll
        for (int i = 0; i < kStretches; ++i)
            if (s_mx[i][tid] >= bound) s_owner[atomicAdd(&s_owners, 1)] = (unsigned short)(i * kThreads + tid);
        __syncthreads();
        const int owners = s_owners;
        const int depth = per * kAhead + 1;  // vectors of a stretch, and a single entry
        // Every entry x (at index `at`) of the owners, in no order.
        auto owned = [&](auto&& f) {
#pragma unroll 2
            for (int i = tid; i < owners * depth; i += kThreads) {
                const int r = i / owners, o = s_owner[i - r * owners], th = o % kThreads, st = o / kThreads;
                const int64_t v = th + ((int64_t)st * per * kAhead + r) * kThreads;
                if (r == depth - 1) {
                    if (st == 0 && th < span.singles()) f(load_one(base, DT, span.single(th)), span.single(th));
                } else if (v < span.vecs) {
                    const int64_t at = span.vec0 + v * N;
                    float x[N];
                    Vec<DT>::load(base, at, x);
#pragma unroll
                    for (int e = 0; e < N; ++e) f(x[e], at + e);
                }
            }
        };
        // Entries above the bound fill the list from its front, those equal to it from its end.
        if (!any_nan)
            owned([&](float x, int64_t at) {
                if (x < bound) return;
                const int i = atomicAdd(x > bound ? &s_above : &s_ties, 1);
                if (i < kCandidates) s_cand[x > bound ? i : kCandidates - 1 - i] = order_key(x, (uint32_t)at);
            });
        __syncthreads();
        int above = s_above, ties = s_ties;
        const bool listed = !any_nan && above + ties <= kCandidates;
        if (!any_nan && !listed && above <= kCandidates - kThreads - kMaxTop) {
            // Many equal entries (a mask's lowest value, a flat row): those above the bound
            // again, and then of the equal ones the first few, in the order of their indices.
            __syncthreads();
            if (tid == 0) s_above = s_ties = 0;
            __syncthreads();
            owned([&](float x, int64_t at) {
                if (x > bound) s_cand[atomicAdd(&s_above, 1)] = order_key(x, (uint32_t)at);
            });
            ties = 0;
            for (int64_t at = span.begin; at < span.end && ties < mine; at += kThreads) {
                if (at + tid < span.end && load_one(base, DT, at + tid) == bound)
                    s_cand[kCandidates - 1 - atomicAdd(&s_ties, 1)] =
                        order_key(bound, (uint32_t)(at + tid));
                __syncthreads();
                ties = s_ties;
                __syncthreads();
            }
            above = s_above;
        } else if (!listed) {
            // A NaN, or too many entries above the bound (sorted rows): the largest entry below
            // the last one found, as often as needed.
            unsigned long long below = ~0ull;
            for (int k = 0; k < mine; ++k) {
                unsigned long long top = 0;
                for (int64_t at = span.begin + tid; at < span.end; at += kThreads) {
                    const unsigned long long key = order_key(load_one(base, DT, at), (uint32_t)at);
                    // (A NaN at index 0 has the largest key there is.)
                    if ((k == 0 || key < below) && key > top) top = key;
                }
                __syncthreads();
                s_cand[tid] = top;
                __syncthreads();
                for (int w = kThreads / 2; w; w >>= 1) {
                    if (tid < w && s_cand[tid + w] > s_cand[tid]) s_cand[tid] = s_cand[tid + w];
                    __syncthreads();
                }
                below = s_cand[0];
                if (tid == 0) s_top[k] = below;
            }
            above = ties = 0;
        }
        for (int i = tid; i < above + ties; i += kThreads) {
            const auto at = [&](int j) { return s_cand[j < above ? j : kCandidates - 1 - (j - above)]; };
            const unsigned long long key = at(i);
            int place = 0;
            for (int j = 0; j < above + ties; ++j) place += at(j) > key;
            if (place < mine) s_top[place] = key;
        }
        __syncthreads();
    }

    // ---- rows over several CTAs: the last one joins
    if (g.splits > 1) {
        LpPart* parts = reinterpret_cast<LpPart*>(g.ws) + row * g.splits;
        if (tid < K) parts[split].top[tid] = tid < mine ? s_top[tid] : 0;
        if (tid == 0) parts[split].m = rm, parts[split].l = rl, parts[split].t = rt;
        __syncthreads();
        if (tid == 0) {
            __threadfence();
            s_last = atomicAdd(g.tickets + row, 1) == g.splits - 1;
            __threadfence();
            if (s_last) g.tickets[row] = 0;
        }
        __syncthreads();
        if (!s_last) return;
        // By every warp alike: a lane per part, then the lanes are joined.
        static_assert(kMaxSplits <= 32, "a lane each");
        rm = -INFINITY, rl = rt = 0.f;
        if (lane < g.splits) {
            const LpPart* p = parts + lane;
            rm = __ldcg(&p->m), rl = __ldcg(&p->l), rt = __ldcg(&p->t);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, rm, o), l2 = __shfl_xor_sync(0xffffffffu, rl, o),
                        t2 = __shfl_xor_sync(0xffffffffu, rt, o);
            join(rm, rl, rt, m2, l2, t2);
        }
        if (K > 0) {
            // The K-th largest of the CTAs' maxima bounds from below, as above; lists of at
            // most kMaxSplits * kMaxTop keys fit the candidates.
            if (tid == 0) s_above = 0, s_thr = 0;
            if (tid < g.splits) s_key[tid] = __ldcg(&parts[tid].top[0]);
            __syncthreads();
            if (tid < g.splits && K <= g.splits) {
                int rank = 0;
                for (int i = 0; i < g.splits; ++i) rank += s_key[i] > s_key[tid];
                if (rank == K - 1) s_thr = s_key[tid];
            }
            __syncthreads();
            const unsigned long long thr = s_thr;
            for (int i = tid; i < g.splits * K; i += kThreads) {
                const unsigned long long key = __ldcg(&parts[i / K].top[i % K]);
                if (key != 0 && key >= thr) s_cand[atomicAdd(&s_above, 1)] = key;
            }
            __syncthreads();
            const int count = s_above;
            for (int i = tid; i < count; i += kThreads) {
                const unsigned long long key = s_cand[i];
                int rank = 0;
                for (int j = 0; j < count; ++j) rank += s_cand[j] > key;
                if (rank < K) s_top[rank] = key;
            }
            __syncthreads();
        }
    }

    // ---- results
    const float ll = logf(rl);
    // (An infinite maximum has left l = 0, or NaN where the row holds one of those too.)
    const float lse = rm == -INFINITY ? -INFINITY : rm == INFINITY && rl == 0.f ? INFINITY : rm + ll;
    if (tid == 0) {
        if (g.a.lse) g.a.lse[row] = lse;
        if (g.a.entropy) g.a.entropy[row] = rm == -INFINITY ? 0.f : ll - rt / rl;
        if (g.a.logprob) {
            const int token = g.a.tokens ? __ldg(g.a.tokens + row) : -1;
            float lp = 0.f;
            if (token >= 0 && token < g.a.vocabulary) {
                const float x = load_one(base, DT, token);
                lp = x == -INFINITY && !(lse != lse) ? -INFINITY : (x - rm) - ll;
            } else if (token != -1) {
                atomicCAS(g.status, 0, kStatusIndex);
            }
            g.a.logprob[row] = lp;
        }
    }
    if (tid < K) {
        const unsigned long long key = s_top[tid];
        const float x = key_value(key);
        g.a.top_tokens[row * K + tid] = (int32_t)key_index(key);
        g.a.top_logprobs[row * K + tid] = x == -INFINITY && !(lse != lse) ? -INFINITY : (x - rm) - ll;
    }
}

struct LbArgs {
    q4lin_logprobs_backward_t a;
    int splits;
    int64_t chunk;
    int* status;
};

template <int DT>
__global__ void __launch_bounds__(kThreads, kCtas) logprobs_backward_kernel(const LbArgs g) {
    constexpr int N = Vec<DT>::N, kAhead = DT == Q4LIN_DTYPE_F32 ? 4 : 2;
    constexpr int size = (int)dtype_size(DT);
    const int64_t row = blockIdx.x / g.splits;
    const int split = (int)(blockIdx.x % g.splits), tid = threadIdx.x;
    const char* x_row = static_cast<const char*>(g.a.logits) + row * g.a.row_stride * size;
    char* d_row = static_cast<char*>(g.a.d_logits) + row * g.a.d_row_stride * size;
    const int64_t begin = split * g.chunk, end = min(g.a.vocabulary, begin + g.chunk);
    const float lse = __ldg(g.a.lse + row);
    int token = -1;
    float d_lp = 0.f, d_h = 0.f, h = 0.f;
    if (g.a.d_logprob) {
        token = __ldg(g.a.tokens + row);
        if (token < -1 || token >= g.a.vocabulary) {
            if (split == 0 && tid == 0) atomicCAS(g.status, 0, kStatusIndex);
            token = -1;
        }
        if (token >= 0) d_lp = __ldg(g.a.d_logprob + row);
    }
    if (g.a.d_entropy) d_h = __ldg(g.a.d_entropy + row), h = __ldg(g.a.entropy + row);
    const bool empty = lse == -INFINITY;
    // -p (d_lp + d_h (y + h)) with y = x - lse = ln p; p = 0 gives 0.
    const float c = fmaf(d_h, h, d_lp);
    auto value = [&](float x, int64_t at) {
        const float y = x - lse;
        const float p = ex2(y * kLog2e);
        float d = -p * fmaf(d_h, fmaxf(y, kNegative), c);
        if (empty || x == -INFINITY) d = 0.f;
        if (at == token && !empty) d += d_lp;
        return d;
    };
    // (The logits' place may be the gradient's: no read-only loads.)
    auto load_entry = [&](int64_t at) {
        if (DT == Q4LIN_DTYPE_F32) return reinterpret_cast<const float*>(x_row)[at];
        return unpack2(reinterpret_cast<const unsigned short*>(x_row)[at], DT).x;
    };
    const Span<DT> span(x_row, begin, end);
    // Vectors where input and output are aligned alike, else single entries.
    const bool alike = ((reinterpret_cast<uintptr_t>(x_row) ^ reinterpret_cast<uintptr_t>(d_row)) & 15) == 0;
    if (!alike) {
        for (int64_t at = begin + tid; at < end; at += kThreads)
            store_one(d_row, DT, at, value(load_entry(at), at));
        return;
    }
    if (tid < span.singles()) {
        const int64_t at = span.single(tid);
        store_one(d_row, DT, at, value(load_entry(at), at));
    }
    for (int64_t v = tid; v < span.vecs; v += kThreads * kAhead) {
        float x[kAhead][N];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (v + i * kThreads < span.vecs) Vec<DT>::load_before_store(x_row, span.vec0 + (v + i * kThreads) * N, x[i]);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (v + i * kThreads >= span.vecs) continue;
            const int64_t at = span.vec0 + (v + i * kThreads) * N;
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < N; ++e) x[i][e] = value(x[i][e], at + e);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = DT == Q4LIN_DTYPE_F32 ? __float_as_uint(x[i][j])
                                             : to_16x2(x[i][2 * j % N], x[i][(2 * j + 1) % N], DT);
            __stcs(reinterpret_cast<uint4*>(d_row + at * size), make_uint4(w[0], w[1], w[2], w[3]));
        }
    }
}

// CTAs per row so that about `want` of them run, each with at least `least` entries.
int splits_for(int64_t rows, int64_t vocabulary, int64_t want, int64_t least, int64_t most) {
    const int64_t s = std::min((want + rows - 1) / rows, (vocabulary + least - 1) / least);
    return (int)std::max<int64_t>(1, std::min(s, most));
}

}  // namespace

cudaError_t logprobs_launch(const q4lin_logprobs_t& a, const LaunchCtx& c) {
    LpArgs g;
    g.a = a;
    g.ws = c.ws;
    g.tickets = c.tickets;
    g.status = c.status_word;
    // CTAs per row.  A cut costs a join of 2 to 3 us and the time after the entries once more; it
    // pays on long rows while they are too few for the SMs (128256 fp32 entries, 20 alternatives,
    // us for 1 / 2 / 4 / 32 CTAs a row: 1 row 15.8 / 13.6 / 10.9 / 9.5, 32 rows 16.5 / 14.6 /
    // 11.7 / 17.8, 100 rows 17.2 / 18.6 / 16.8 / 40, 300 rows 35.3 / 33.5 / 43 / 109, 400 rows
    // 40.2 / 56.6; 32000 entries, 1 row: 7.6 / 9.1).
    g.splits = 1;
    if (a.vocabulary >= 65536 && a.rows < 2 * c.sm_count)
        g.splits = a.rows <= 8 ? kMaxSplits : (int)std::min<int64_t>(4, (400 + a.rows - 1) / a.rows);
    g.chunk = ((a.vocabulary + g.splits - 1) / g.splits + 7) / 8 * 8;
    g.splits = (int)((a.vocabulary + g.chunk - 1) / g.chunk);
    const int64_t grid = a.rows * g.splits;
    switch (a.dtype) {
        case Q4LIN_DTYPE_F32: logprobs_kernel<Q4LIN_DTYPE_F32><<<(unsigned)grid, kThreads, 0, c.stream>>>(g); break;
        case Q4LIN_DTYPE_F16: logprobs_kernel<Q4LIN_DTYPE_F16><<<(unsigned)grid, kThreads, 0, c.stream>>>(g); break;
        default: logprobs_kernel<Q4LIN_DTYPE_BF16><<<(unsigned)grid, kThreads, 0, c.stream>>>(g); break;
    }
    return cudaGetLastError();
}

cudaError_t logprobs_backward_launch(const q4lin_logprobs_backward_t& a, const LaunchCtx& c) {
    LbArgs g;
    g.a = a;
    g.status = c.status_word;
    g.splits = splits_for(a.rows, a.vocabulary, 16 * c.sm_count, 8 * kThreads, 1 << 20);
    g.chunk = ((a.vocabulary + g.splits - 1) / g.splits + 7) / 8 * 8;
    g.splits = (int)((a.vocabulary + g.chunk - 1) / g.chunk);
    const int64_t grid = a.rows * g.splits;
    switch (a.dtype) {
        case Q4LIN_DTYPE_F32: logprobs_backward_kernel<Q4LIN_DTYPE_F32><<<(unsigned)grid, kThreads, 0, c.stream>>>(g); break;
        case Q4LIN_DTYPE_F16: logprobs_backward_kernel<Q4LIN_DTYPE_F16><<<(unsigned)grid, kThreads, 0, c.stream>>>(g); break;
        default: logprobs_backward_kernel<Q4LIN_DTYPE_BF16><<<(unsigned)grid, kThreads, 0, c.stream>>>(g); break;
    }
    return cudaGetLastError();
}

}  // namespace q4lin
