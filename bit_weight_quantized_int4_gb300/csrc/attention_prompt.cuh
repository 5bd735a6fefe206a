// attention_prompt.cuh -- attention of many query rows per key/value head over a paged cache
// (prompts and their chunks), on the tcgen05 tensor cores.  BITS: of the cache's codes
// (attention_prompt.cu has 8, kv4_attention_prompt.cu 4).
//
// A row is one query token of one head; the heads that share a key/value head are rows of one
// list (token-major), so grouped heads fill the MMA's 128 rows and share the keys.  A CTA
// takes two tiles of 128 rows and walks over 128 keys at a time:
//   widening warps      codes from global memory into fp16 K and V tiles in shared memory
//                       (code - 128 is exact in fp16; both are stored with the axis that the
//                       product sums over contiguous, 128-byte swizzled),
//   one issuing thread  S = Q K^T into tensor memory, then O += P V with P read from there,
//   softmax warps       one thread per row: the running maximum and sum in fp32, the weights
//                       back into tensor memory over the scores that they came from.
// The two tiles take turns: one's products run while the other's softmax does.  (Heads of 256, over 4 bits:
// one tile, whose outputs take the tensor memory of two.)
//
// The pages' scales stay out of the operands: a key page's multiplies its columns of S, a
// value page's (over the largest of the walk) joins the exponent of its weights.  O is
// only rescaled when a row's maximum has grown by 2^8 since the last time, which fp16's range
// leaves room for.  4-bit codes have a scale for each token: a key's multiplies its column of S, read
// from shared memory by every softmax warp.  A value's (over the largest of the walk) multiplies
// its weights in the same way where those have two terms; for bf16 outputs, where they have one,
// code - 8 times the scale is rounded to fp16 once as it is widened (11 bits as the weight's).  Walks whose values' scales
// are so far apart that fp16 would lose small ones (kWideFolded) take the scales' exponents into the weights'.
// Queries and weights enter as QT and PT fp16 terms, the rounded value and
// what the rounding left (22 bits), each term a product of its own: two of both in general; a
// weight of a bf16 output takes one (its 11 bits are finer than the output's 8), and bf16
// queries that are not rotated are exact in one.
//
// Few rows over many keys leave SMs idle (and, over 4 bits, few more walks than SMs the last round's): their
// walks over the keys are then cut into equal parts, one CTA each, that a second kernel joins in the order of
// the keys.
//
// Bound: the products, 2 head_dim flops a pair for each of QT + PT terms.  Measured (8 key/value
// heads of 128, 4 query heads each, the last 2048 of 8192 tokens): 240 us for rotated bf16
// queries (QT 2, PT 1: 361 Gflop, 1.5 Pflop/s, 0.79 of a large library product's rate), 336 us
// for fp16 (two terms of both), 479 us for fp32 (the same, and outputs taken out every 8 steps).
// While walks run the tensor pipes are busy for 77 % of the time; the scores' products, which read
// 8 KB of shared memory for 64 clocks of work, take the rest.
// (Leaving out the exponentials, or the loads or stores of the widened codes, changed the
// time by less than 4 %; two threads a row instead of one: 260 us; a share of the exponentials
// as polynomials on the FMA pipes: 249 us and up.)  Whole walks on 152 SMs leave 16 % of them
// idle at this size, and each has about 10 us around it: the queries, the first keys, the rows.
// Cutting the last round's walks so that all SMs end together took as long (239 us, and the
// joining kernel's time on top): busier SMs were slower ones.
// Over 4 bits, the same prompt: 271 us for bf16 queries as they are (QT 1), 316 us rotated, 407 us for
// fp16, 564 us for fp32; heads of 64, bf16, 215 us; the last 820 of 8192 tokens with heads of 256 365, 439,
// 540 and 705 us (on the kernel for few rows 1570).  The tensor pipes are busy for 35 % of the first:
// the softmax, with a scale for each key, and the widening take longer.  (With the values' scales multiplied
// into the weights, as for the other types, 305 us; that without the keys' scales 267, without any 213.  Four
// rows a thread, by loads of 16 rows, with an eighth of the reads of scales, against 279: 276 us, heads of 64
// 220 against 211; with that, half steps whose next scores are computed meanwhile: 286.)
#pragma once

#include <algorithm>
#include <type_traits>

#include "q4lin_internal.h"
#include "serving.cuh"

namespace q4lin {
namespace {
using namespace ptx;
using namespace serving;

constexpr int kQ = 128;     // rows per tile (MMA M = lanes of tensor memory)
constexpr int kKeys = 128;  // keys per step
// Five warpgroups: two of softmax, one that widens keys, one values, one whose first warp
// issues the MMAs.
constexpr int kSoftWarps = 8, kValueWarp = 12, kIssueWarp = 16;
constexpr int kWarps = 20, kThreads = 32 * kWarps;
// Registers of their threads: launched with 96 each.  Where values are multiplied by their scales as they are
// widened and heads have 128 channels, the widening warps need more (softmax / widening 176 / 48, 168 / 56, 160 /
// 64, 152 / 72, 2048 of 8192 tokens: 279, 272, 269, 310 us, rotated 326, 312, 306, 317; heads of 64 212, 214,
// 220, 220; two terms of weights, fp16, 400, 405, 414).
constexpr int kIssueRegs = 32;
__host__ __device__ constexpr int soft_regs(int D, bool folded) { return D == 256 || (folded && D == 128) ? 160 : 176; }
__host__ __device__ constexpr int widen_regs(int D, bool folded) { return D == 256 || (folded && D == 128) ? 64 : 48; }
constexpr bool regs_fit(int D, bool folded) {
    return 2 * soft_regs(D, folded) + 2 * widen_regs(D, folded) + kIssueRegs <= 5 * 96;
}
static_assert(regs_fit(128, true) && regs_fit(128, false), "registers of the launch");
constexpr int kMaxBatch = 1024;  // sequences per launch
constexpr int kScaleSlots = 5;  // steps whose scales are kept: the widening warps are up to four ahead
constexpr float kBase = 7.f;    // weights are kept as 2^7 p ...
// Tensor cores cut off what a product's sum has no room for, so an error of one sign grows with
// the steps that O adds up there (16384 keys: 3.6e-5 of the norm with two-term weights).  Outputs
// are taken out every `DRAIN` steps and added up with rounding, in memory:
//   fp32  in their own place or their part's, every 8 steps: 3e-6 at any length, about what sums in
//         plain fp32 have (every 16 steps: 5e-6);
//   fp16  in a slot of the workspace, every 64 steps, where the page table has room for more than
//         kFewKeys: below them the error stays at a third of what the rounding to fp16 leaves
//         (2.1e-4), at 131072 keys it was 2.6e-4.  (The code for it costs 336 -> 362 us on 2048 of
//         8192 tokens, 32 heads of 128, which never take anything out; walks of 131072 keys 5.2 -> 5.7 ms.)
//   bf16  not at all: 1.6e-4 at 131072 keys, against 1.7e-3 of the rounding.
constexpr int kDrainF32 = 8, kDrainF16 = 64;
constexpr int64_t kFewKeys = 32768;
constexpr int kDrainSlots = 256;  // at most; one for each CTA that runs
constexpr float kSlack = 8.f;   // ... with p up to 2^8 before O is rescaled (fp16: below 2^16)
// Undone before a logarithm, whose error grows with its distance from 0.
constexpr float kUnbase = 1.f / 128.f;
// (4 bits) A part's sums of values above 2^32 are kept over 2^32, so that those near fp32's largest have room.
constexpr float kLessBits = 32.f, kLess = 2.3283064365386963e-10f;
// A score's factor, its key's scale included, is at least about this, so that a masked score (-infinity) stays one.
constexpr float kLeastFactor = 1e-37f;
// (4 bits) Weights of a step that add up to no more than this are below fp16's 65504 each.
constexpr float kMostSum = 65000.f;
constexpr float kLeastRatio = 5.421010862427522e-20f;  // 2^-64
// (4 bits) A walk whose values' scales are further apart than this is wide.  fp16 has room for two terms
// of weights down to 2^-32 of the largest, and for folded values' 11 bits down to 2^-25 of the largest scale.
// Beyond, a row that sees only small values beside large ones behind it, or before its window, would lose them.
// In a wide walk the exponents of the values' scales join those of the weights, so that a row's maximum, a
// whole number there, is that of the products, which have the upper end of fp16's range; and values are not
// folded.  What is below 2^-80 of the walk's largest scale counts as that in the maximum, so that the sum of
// the weights alone stays in fp32's range.  (Such walks take 1.4 to 3.5 times as long: 2048 of 8192 tokens in
// bf16 819 us, in fp32 1026.)
constexpr float kWideFolded = 16777216.f, kWideWeights = 1024.f;  // 2^24, 2^10
constexpr int kLeastExponent = -80;
constexpr int64_t kDrainNs = 4000000000LL;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kScoreCol = 256;  // O of the two tiles in columns 0 and 128, S from here

// Rows of a CTA, a pair of tiles: of heads of 256 channels, whose outputs fill the columns of two, one tile.
__host__ __device__ constexpr int pair_rows_of(int64_t D) { return D == 256 ? kQ : 2 * kQ; }

struct PromptArgs {
    q4lin_kv_cache_t cache;
    q4lin_attention_t a;
    int page_shift, pair_rows, bits;
    int64_t rows_min;  // sequences of more rows than this per key/value head are taken
    int q_vec;
    int slots, most_parts;  // CTAs that run at a time; parts of a walk at most
    int pairs_most;         // records that the plan has room for
    float* parts;           // [unit][2 kQ (D + 2)]: unfinished walks; [slot][2 kQ D]: fp16 outputs taken out
    int* taken;             // [drain_slots]: slots in use
    int drain_slots;
    int4* plan;             // parts, steps of each, pairs; then of each pair: sequence, tokens,
                            // length, tile; first and last step, first token
    int* status;
    int64_t wait_ns;
    int skip_first_copy;  // test hook: no keys come, and the waits for them run out
};

// What one sequence asks of this kernel.
struct Prompt {
    int tq, len, pairs;  // pairs of row tiles
    bool bad;
};
__device__ __forceinline__ Prompt prompt_of(const PromptArgs& g, int64_t b) {
    const int64_t o0 = __ldg(g.a.offsets + b), o1 = __ldg(g.a.offsets + b + 1), len = __ldg(g.a.lengths + b);
    const int64_t rows = (o1 - o0) * (g.a.heads / g.cache.kv_heads);
    Prompt p;
    p.bad = o0 < 0 || o1 < o0 || o1 > g.a.tokens || o1 - o0 > g.a.max_query ||
            len > g.cache.pages_per_sequence << g.page_shift || (g.a.rope.cos && len > g.a.rope.positions);
    p.tq = (int)(o1 - o0), p.len = (int)(len > 0 ? len : 0);
    p.pairs = !p.bad && rows > g.rows_min ? (int)((rows + g.pair_rows - 1) / g.pair_rows) : 0;
    return p;
}
// The steps over keys of a pair of row tiles: 128 first .. 128 last - 1.
__device__ __forceinline__ void walk_of(const PromptArgs& g, const Prompt& p, int pair, int* first, int* last) {
    const int group = (int)(g.a.heads / g.cache.kv_heads), rows = p.tq * group, row0 = pair * g.pair_rows;
    const int first_pos = p.len - p.tq + row0 / group;
    const int last_pos = p.len - p.tq + (min(rows, row0 + g.pair_rows) - 1) / group;
    const int last_key = g.a.causal ? last_pos : p.len - 1;
    const int64_t low = g.a.window > 0 ? (int64_t)first_pos - g.a.window + 1 : 0;
    *first = low > 0 ? (int)(low / kKeys) : 0;
    *last = last_key < 0 || p.len == 0 ? *first : max(*first, last_key / kKeys + 1);
}
template <int D>
__device__ __forceinline__ float* part_at(const PromptArgs& g, int64_t unit) {
    return g.parts + unit * (pair_rows_of(D) * (D + 2));
}

// Shared memory.  A step's K tile is D / 64 blocks of 64 channels, its V tile two blocks of 64
// keys; both come and go by block through rings, as much as fits (three of each beside 128
// channels of two terms: half a tile is widened while the other's products run; of heads of 256 one
// block of values).
template <int D, int QT, bool KEYED>
struct Layout {
    static constexpr int kBlock = 128 * 128;           // 128 rows of 128 bytes
    static constexpr int kBlocks = D / 64;             // of a Q or K tile
    static constexpr int vBlock = D * 128;
    static constexpr bool kTight = QT == 2 && D >= 128;
    // (KEYED: scales of each key and value take the place of a block of values.)
    static constexpr int kRing = kTight ? 3 : 4;
    static constexpr int vRing = D == 256 ? (kTight ? 1 : 2) : kTight && KEYED ? 2 : kRing;
    static constexpr uint32_t q = 0;                                  // [tile][term][block]
    static constexpr uint32_t k = q + pair_rows_of(D) / kQ * QT * kBlocks * kBlock;      // [slot]
    static constexpr uint32_t v = k + kRing * kBlock;                 // [slot]
    static constexpr uint32_t bytes = v + vRing * vBlock;
};

// What a CTA does, left in shared memory by its prologue: the warpgroups read what each needs
// into its own registers (values kept across their register shares are spilled, and the issuing
// warp then waits for local memory behind the codes' loads: 351 against 243 us for the case at
// the head of this file).
struct Job {
    int64_t o0;
    int b, h, tq, len, row0, row_end, step0, n, cut;
    int page_low;  // the first page that a window leaves
    int slot;      // for outputs taken out, -1: none
};

// Scales of the steps between widening and softmax.  8 bits: of 16 keys each, with the values' as
// logarithms and inverses; KEYED: of each key, the values' as ratios.  K blocks of up to two steps
// more are widened while a step's scores are read, of four with 64 channels (kScaleSlots).
template <int D, bool KEYED>
struct StepScales {
    static constexpr int kSlots = kScaleSlots;
    float k_scale[kSlots][8], v_log[kSlots][8], v_inv[kSlots][8];
};
template <int D>
struct StepScales<D, true> {
    static constexpr int kSlots = D == 64 ? kScaleSlots : 3;
    alignas(16) float k_scale[kSlots][kKeys];
    alignas(16) float v_ratio[kSlots][kKeys];
};

template <int D, bool KEYED>
struct PromptShared {
    Job job;
    float factor[2 * kQ];
    StepScales<D, KEYED> scales;
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4], s_full[2], p_full[2], o_full[2];
    float v_max[kWarps], v_min[kWarps], k_max[kWarps];  // (4 bits) v_min: of those above 0
    int failed;
    uint32_t tmem;
};

// The MMAs are issued by one lane of a warp that runs as a whole, so that addresses and
// descriptors stay in uniform registers (a lone thread's have to be moved there one by one,
// which took longer than the MMAs: 100 against 64 clocks each).
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t leader;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(leader));
    return leader;
}
// D (tensor memory) (+)= A B^T, both fp16 operands from shared memory.
__device__ __forceinline__ void mma_f16_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           bool acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc), "r"(leader)
        : "memory");
}
// The same with A in tensor memory.
__device__ __forceinline__ void mma_f16_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           bool acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t leader, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(leader)
        : "memory");
}
// 8 or 16 columns of this warp's lanes, without waiting for completion.
__device__ __forceinline__ void tmem_st8_async(uint32_t addr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st16_async(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
// 64 columns of this warp's lanes; the load and its wait are one statement, so that no use of
// the registers is scheduled between them.
__device__ __forceinline__ void tmem_ld64(uint32_t addr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(addr)
        : "memory");
}
// 32 columns of this warp's lanes, without waiting; and the wait for them, which the registers go
// through so that no use of them is scheduled before it.
__device__ __forceinline__ void tmem_ld32_async(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
// `bytes` from shared to global memory, both 16-byte aligned, and until they have been read.
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile(
        "cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\t"
        "cp.async.bulk.commit_group;\n\t"
        "cp.async.bulk.wait_group 0;" ::"l"(reinterpret_cast<uint64_t>(dst)),
        "r"(src), "r"(bytes)
        : "memory");
}
// Values' scales over the walk's reference, taken apart: exponent, 2^-exponent, and what that leaves, at most 1.
struct Apart2 {
    float2 exponent, inverse, rest;
};
__device__ __forceinline__ Apart2 apart2(float2 ratio) {
    auto exponent = [](float r) { return min(max((int)(__float_as_uint(r) >> 23 & 255u) - 126, kLeastExponent), 126); };
    const int a = exponent(ratio.x), b = exponent(ratio.y);
    Apart2 p;
    p.exponent = make_float2((float)a, (float)b);
    p.inverse = make_float2(__uint_as_float((uint32_t)(127 - a) << 23), __uint_as_float((uint32_t)(127 - b) << 23));
    p.rest = fmul2(ratio, p.inverse);
    return p;
}
// m + log2(l); over 4 bits with the exponent of an l above 2 (far above, where values' scales are far apart) added
// apart, as lg2's result would be rounded where m cancels it.
__device__ __forceinline__ float log2_sum(float m, float l, bool apart) {
    if (!(apart && l >= 2.f && l <= 3.4028235e38f)) return m + lg2(l);
    const uint32_t bits = __float_as_uint(l);
    return m + (float)((int)(bits >> 23) - 127) + lg2(__uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u));
}
// This thread's number, read where it stands.
__device__ __forceinline__ int thread_number() {
    int t;
    asm volatile("mov.u32 %0, %%tid.x;" : "=r"(t));
    return t;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 16 bytes, issued where it stands (a plain load may sink to its use, behind the waits).
__device__ __forceinline__ void ld_codes(const uint8_t* p, uint4& v) {
    asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
}
// Pairs times pairs of scales of two terms, rounded once to fp16 (but for the lower term's product).
__device__ __forceinline__ uint32_t scaled_f16(uint32_t x, uint32_t hi, uint32_t lo) {
    const __half2 v = *reinterpret_cast<const __half2*>(&x);
    const __half2 y = __hfma2(v, *reinterpret_cast<const __half2*>(&hi), __hmul2(v, *reinterpret_cast<const __half2*>(&lo)));
    return *reinterpret_cast<const uint32_t*>(&y);
}
// Byte of 16-byte chunk `chunk` of row `row` in a 128-byte-swizzled block.
__device__ __forceinline__ uint32_t swizzled(int row, int chunk) {
    return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4));
}

// The queries of a pair of tiles: rotated, scaled to fp16's upper range by a power of two, as
// QT fp16 terms in swizzled tiles; and what undoes the scaling, with the scores' own scale.
template <int D, int QT, int DT, int BITS>
__device__ __noinline__ void put_queries(const PromptArgs& g, uint8_t* gbase, float* factor, int64_t o0, int h,
                                         int tq, int len, int row0, int row_end) {
    using L = Layout<D, QT, false>;  // (where the queries are is the same with KEYED)
    const int tid = threadIdx.x, group = (int)(g.a.heads / g.cache.kv_heads);
    constexpr int kUnitsRow = D / 8, kPer = kThreads / kUnitsRow;  // 16 or 8 lanes a row
    const int u = tid % kUnitsRow;
    bool turned;
    int cl, ch;
    rope_channels(g.a.rope, u, &turned, &cl, &ch);
    // Rows in batches whose loads are in flight together.
    constexpr int kRows = pair_rows_of(D), kPasses = (kRows + kPer - 1) / kPer, kTogether = 4;
#pragma unroll 1
    for (int p0 = 0; p0 < kPasses && p0 * kPer < row_end - row0; p0 += kTogether) {
        float x[kTogether][8], c[kTogether][4], sn[kTogether][4];
#pragma unroll
        for (int k = 0; k < kTogether; ++k) {
            const int r = (p0 + k) * kPer + tid / kUnitsRow, row = row0 + r;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[k][e] = 0.f;
            if (r < kRows && row < row_end) {
                const int token = (uint32_t)row / (uint32_t)group, head = h * group + row - token * group;
                const int64_t e = (o0 + token) * g.a.q_token_stride + head * g.a.q_head_stride;
                const int position = len - tq + token;
                load_four(g.a.query, DT, e + cl, g.q_vec, x[k]);
                load_four(g.a.query, DT, e + ch, g.q_vec, x[k] + 4);
                if (turned && position >= 0)
                    rope_load(g.a.rope, position, u, c[k], sn[k]);
                else
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[k][e] = 1.f, sn[k][e] = 0.f;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) c[k][e] = 1.f, sn[k][e] = 0.f;
            }
        }
#pragma unroll
        for (int k = 0; k < kTogether; ++k) {
            const int r = (p0 + k) * kPer + tid / kUnitsRow;
            if (turned) rope_apply(g.a.rope, c[k], sn[k], x[k]);
            float m = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[k][e]));
#pragma unroll
            for (int o = kUnitsRow / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            // 2^up brings the row's largest |x| to [2^14, 2^15); the scale's sign goes with it,
            // so that larger scores stay larger after the factor.  With an infinity the whole row
            // becomes NaN (a lone term of it could give scores of -infinity, as if masked).
            const int ex = min(max((int)(__float_as_uint(m) >> 23), 30), 254) - 127;
            const uint32_t up_bits = m == INFINITY ? 0x7FC00000u : (uint32_t)(127 + 14 - ex) << 23;
            const float up = copysignf(__uint_as_float(up_bits), g.a.scale);
            const float down = __uint_as_float((uint32_t)(127 - 14 + ex) << 23);
            if (r < kRows) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    split_f16(x[k][2 * e] * up, x[k][2 * e + 1] * up, &hi[e], &lo[e]);
                if constexpr (BITS == 4) {
                    // Channels 0, 4, 1, 5, 2, 6, 3, 7 of a chunk of eight, as nibbles are widened.
                    const uint32_t tile = L::q + (uint32_t)((r / kQ) * QT * L::kBlocks) * L::kBlock;
                    if (ch == cl + 4) {
                        const uint32_t at = tile + cl / 64 * L::kBlock + swizzled(r % kQ, cl % 64 / 8);
#pragma unroll
                        for (int term = 0; term < QT; ++term) {
                            const uint32_t(&h)[4] = term ? lo : hi;
                            *reinterpret_cast<uint4*>(gbase + at + term * L::kBlocks * L::kBlock) =
                                make_uint4(prmt(h[0], h[2], 0x5410u), prmt(h[0], h[2], 0x7632u),
                                           prmt(h[1], h[3], 0x5410u), prmt(h[1], h[3], 0x7632u));
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int d = (e < 4 ? cl : ch) + e % 4;
                            const uint32_t at = tile + d / 64 * L::kBlock + swizzled(r % kQ, d % 64 / 8) +
                                                d % 4 * 4 + (d >> 2 & 1) * 2;
                            const int shift = e % 2 * 16;
                            *reinterpret_cast<uint16_t*>(gbase + at) = (uint16_t)(hi[e / 2] >> shift);
                            if (QT == 2)
                                *reinterpret_cast<uint16_t*>(gbase + at + L::kBlocks * L::kBlock) =
                                    (uint16_t)(lo[e / 2] >> shift);
                        }
                    }
                } else {
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const int d = w ? ch : cl;  // channels d .. d + 3: half a 16-byte chunk
                        const uint32_t at = L::q + (uint32_t)((r / kQ) * QT * L::kBlocks + d / 64) * L::kBlock +
                                            swizzled(r % kQ, (d % 64) / 8) + (d % 8) * 2;
                        *reinterpret_cast<uint2*>(gbase + at) = make_uint2(hi[2 * w], hi[2 * w + 1]);
                        if (QT == 2)
                            *reinterpret_cast<uint2*>(gbase + at + L::kBlocks * L::kBlock) =
                                make_uint2(lo[2 * w], lo[2 * w + 1]);
                    }
                }
                if (u == 0) factor[r] = fabsf(g.a.scale) * kLog2e * down;
            }
        }
    }
}

// What walks of `longest` steps cost in n parts: rounds of CTAs times their steps, with 4 more for what comes
// before and after, 3 for a join.
__host__ __device__ inline int64_t cost_of(int64_t walks, int64_t slots, int64_t longest, int64_t n) {
    return (n * walks + slots - 1) / slots * ((longest + n - 1) / n + (n > 1 ? 7 : 4));
}

// One CTA, before the prompts' kernel: which pairs there are, and in how many parts their walks
// are cut.
constexpr int kPlanThreads = 256;
__global__ void __launch_bounds__(kPlanThreads) attention_prompt_plan_kernel(const PromptArgs g, int units_most) {
    __shared__ int s_longest[kPlanThreads / 32], s_scan[kPlanThreads / 32], s_prefix[kMaxBatch + 1];
    griddep_launch_dependents();  // (the prompts' kernel waits for this one's end)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int Hkv = (int)g.cache.kv_heads, group = (int)(g.a.heads / g.cache.kv_heads);
    int pairs = 0, longest = 0;
    if (tid < g.drain_slots) g.taken[tid] = 0;
    for (int64_t b0 = 0; b0 < g.cache.batch; b0 += kPlanThreads) {
        const int64_t b = b0 + tid;
        int sum = 0;
        if (b < g.cache.batch) {
            const Prompt p = prompt_of(g, b);
            if (p.bad) atomicCAS(g.status, 0, kStatusIndex);
            sum = p.pairs;
            if (p.pairs) {
                int first, last;
                // Causal: without a window the last pair's walk is the longest; with one, none is
                // longer than `window`.  Else all walks end together, and the first pair's begins
                // before the others.
                walk_of(g, p, g.a.causal ? p.pairs - 1 : 0, &first, &last);
                const int64_t window = (g.a.window + g.pair_rows / group + kKeys) / kKeys + 1;
                const bool behind = g.a.causal && g.a.window > 0;
                longest = max(longest, behind ? (int)min((int64_t)p.len / kKeys + 1, window) : last - first);
            }
        }
        const int own = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += n;
        }
        __syncthreads();
        if (lane == 31) s_scan[warp] = sum;
        __syncthreads();
        int before = pairs;
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            if (w < warp) before += s_scan[w];
            pairs += s_scan[w];
        }
        if (b < g.cache.batch) s_prefix[b] = before + sum - own;
    }
    // Offsets that only rise have no more pairs than there is room for. Where some decrease (which
    // has been reported above) the others may overlap: then none are taken.
    if (pairs > g.pairs_most) pairs = 0;
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) s_longest[warp] = longest;
    if (tid == 0) s_prefix[g.cache.batch] = pairs;
    __syncthreads();
    for (int i = tid; i < pairs; i += kPlanThreads) {
        int lo = 0, hi = (int)g.cache.batch;  // prefix[lo] <= i < prefix[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_prefix[mid] <= i)
                lo = mid;
            else
                hi = mid;
        }
        const Prompt p = prompt_of(g, lo);
        const int tile = p.pairs - 1 - (i - s_prefix[lo]);  // the longest walks first
        int first, last;
        walk_of(g, p, tile, &first, &last);
        g.plan[1 + 2 * i] = make_int4(lo, p.tq, p.len, tile);
        g.plan[2 + 2 * i] = make_int4(first, last, __ldg(g.a.offsets + lo), 0);
    }
    if (warp != 0) return;
    for (int w = 0; w < kPlanThreads / 32; ++w) longest = max(longest, s_longest[w]);
    // Walks in `parts` parts of `each` steps where whole ones leave SMs idle.  Lane i weighs i + 1 and
    // i + 33 parts.
    uint32_t best = 0xFFFFFFFFu;
    for (int n = lane + 1; n <= g.most_parts; n += 32) {
        const int64_t units = (int64_t)n * pairs * Hkv;
        if (n > 1 && units > units_most) break;
        const int64_t cost = cost_of((int64_t)pairs * Hkv, g.slots, longest, n);
        best = min(best, (uint32_t)min(cost, (int64_t)0x3FFFFFF) << 6 | (uint32_t)(n - 1));
    }
    const int parts = (int)(__reduce_min_sync(0xffffffffu, best) & 63u) + 1;
    if (lane == 0) *g.plan = make_int4(parts, max(1, (longest + parts - 1) / parts), pairs, 0);
}

// A free slot, for a CTA of a whole walk that outputs of 16 bits are taken out of; -1 for others.
// There are as many as CTAs run at a time (each holds all of an SM's tensor memory), so one is
// free; which one does not change the results.  Without (the search is bounded) outputs stay.
template <int DT, int DRAIN>
__device__ __forceinline__ int take_slot(const PromptArgs& g, int n, bool cut) {
    if (DT == Q4LIN_DTYPE_F32 || DRAIN == 0 || cut || n <= DRAIN) return -1;
    int slot = (int)(blockIdx.x % g.drain_slots);
    for (int i = 0; i < 64 * kDrainSlots; ++i) {
        if (atomicCAS(g.taken + slot, 0, 1) == 0) {
            __threadfence();
            return slot;
        }
        slot = slot + 1 < g.drain_slots ? slot + 1 : 0;
    }
    return -1;
}

// Where row `row` of a job (row r of its pair of tiles) has its fp32 outputs, its sums where the
// walk is cut, or what was taken out of its fp16 outputs.
template <int D, int DT>
__device__ __forceinline__ float* out_row(const PromptArgs& g, const volatile Job& job, int row, int r) {
    if (job.cut) return part_at<D>(g, blockIdx.x) + r * D;
    if (DT != Q4LIN_DTYPE_F32) return g.parts + ((int64_t)job.slot * pair_rows_of(D) + r) * D;
    const int group = (int)(g.a.heads / g.cache.kv_heads), token = row / group;
    const int64_t index = (job.o0 + token) * g.a.heads + job.h * group + (row - token * group);
    return static_cast<float*>(g.a.out) + index * D;
}
// y += keep * to[0 .. 15] where something is there, and back to it if it is to stay.
__device__ __forceinline__ void add_16(float* to, uint32_t (&y)[16], float keep, bool there, bool stays) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float4 v = make_float4(__uint_as_float(y[4 * e]), __uint_as_float(y[4 * e + 1]), __uint_as_float(y[4 * e + 2]),
                               __uint_as_float(y[4 * e + 3]));
        if (there) {
            const float4 old = reinterpret_cast<const float4*>(to)[e];
            v.x = fmaf(old.x, keep, v.x), v.y = fmaf(old.y, keep, v.y);
            v.z = fmaf(old.z, keep, v.z), v.w = fmaf(old.w, keep, v.w);
        }
        if (stays)
            reinterpret_cast<float4*>(to)[e] = v;
        else
            y[4 * e] = __float_as_uint(v.x), y[4 * e + 1] = __float_as_uint(v.y), y[4 * e + 2] = __float_as_uint(v.z),
                  y[4 * e + 3] = __float_as_uint(v.w);
    }
}

template <int D, int QT, int PT, int DT, int DRAIN, int BITS>
__global__ void __launch_bounds__(kThreads, 1) attention_prompt_kernel(const PromptArgs g) {
    constexpr bool kKeyed = BITS == 4, kFolded = BITS == 4 && PT == 1;  // what becomes of scales
    using L = Layout<D, QT, kKeyed>;
    using Scales = StepScales<D, kKeyed>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ PromptShared<D, kKeyed> S;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - smem_u32(smem_raw));
    const q4lin_kv_cache_t& C = g.cache;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, ps = g.page_shift;
    const int Hkv = (int)C.kv_heads, group = (int)(g.a.heads / C.kv_heads);
    const int h = (int)(blockIdx.x % Hkv);
    griddep_launch_dependents();  // (the joining kernel waits for this one's end)
    griddep_wait();               // for the plan
    {
    const int4 plan = __ldcg(g.plan);
    const int parts = plan.x, each = plan.y, pair = (int)(blockIdx.x / Hkv) / parts;
    if (pair >= plan.z) return;
    const int part = (int)(blockIdx.x / Hkv) % parts;
    const int4 j0 = __ldcg(g.plan + 1 + 2 * pair), j1 = __ldcg(g.plan + 2 + 2 * pair);
    const int b = j0.x, tq = j0.y, len = j0.z, tile = j0.w;
    const int64_t o0 = j1.z;
    if (tid == 0) S.failed = 0;
    const int rows = tq * group, row0 = tile * pair_rows_of(D);
    const int row_end = min(rows, row0 + pair_rows_of(D));
    const int step0 = min(j1.x + part * each, j1.y), step1 = min(step0 + each, j1.y);
    const int n = step1 - step0;
    if (n == 0 && part > 0) return;  // a shorter walk has fewer parts
    const int64_t low = g.a.window > 0 ? (int64_t)len - tq + row0 / group - g.a.window + 1 : 0;
    const int page_low = low > 0 ? (int)(low >> ps) : 0;
    if (tid == 0)
        S.job = {o0, b, h, tq, len, row0, row_end, step0, n, parts > 1, page_low, take_slot<DT, DRAIN>(g, n, parts > 1)};
    const int32_t* table = C.page_table + b * C.table_stride;
    const int pages = (len + (1 << ps) - 1) >> ps;

    // ---- prologue: barriers, tensor memory, the largest value scale, queries
    if (tid == 0) {
        for (int s = 0; s < 4; ++s) {
            mbar_init(smem_u32(&S.k_full[s]), 128);
            mbar_init(smem_u32(&S.v_full[s]), 128);
            mbar_init(smem_u32(&S.k_empty[s]), 1);
            mbar_init(smem_u32(&S.v_empty[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&S.s_full[s]), 1);
            mbar_init(smem_u32(&S.p_full[s]), kQ);
            mbar_init(smem_u32(&S.o_full[s]), 1);
        }
        mbar_init_fence();
    }
    if (warp == kIssueWarp) tmem_alloc(smem_u32(&S.tmem), kTmemCols);
    float v_max = 0.f;
    [[maybe_unused]] float v_min = INFINITY, k_max = 0.f;
    const int page_first = max((step0 * kKeys) >> ps, page_low);
    const int page_last = (int)min((int64_t)pages, ((int64_t)step1 * kKeys) >> ps);  // (the last step may end past 2^31)
    if constexpr (BITS == 8) {
        for (int p = page_first + tid; p < page_last; p += kThreads) {
            const int id = __ldg(table + p);
            if (id < 0 || id >= C.num_pages)
                atomicCAS(g.status, 0, kStatusIndex);
            else
                v_max = fmaxf(v_max, __ldg(C.v_scales + (int64_t)id * Hkv + h));
        }
    } else {
        // Four tokens' scales a thread.
        const int fours = ps - 2;
#pragma unroll 4
        for (int i = (page_first << fours) + tid; i < page_last << fours; i += kThreads) {
            const int p = i >> fours, e = (i & ((1 << fours) - 1)) * 4, id = __ldg(table + p);
            const int left = len - (p << ps) - e;  // (what is behind the sequence may be anything)
            if (id < 0 || id >= C.num_pages) {
                atomicCAS(g.status, 0, kStatusIndex);
            } else {
                const int64_t at = (((int64_t)id * Hkv + h) << ps) + e;
                const float4 s = __ldg(reinterpret_cast<const float4*>(C.v_scales + at));
                const float v[4] = {s.x, s.y, s.z, s.w};
                if constexpr (!kFolded) {
                    const float4 k = __ldg(reinterpret_cast<const float4*>(C.k_scales + at));
                    k_max = fmaxf(k_max, fmaxf(fmaxf(0 < left ? k.x : 0.f, 1 < left ? k.y : 0.f), fmaxf(2 < left ? k.z : 0.f, 3 < left ? k.w : 0.f)));
                }
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float x = n < left ? v[n] : 0.f;
                    v_max = fmaxf(v_max, x), v_min = fminf(v_min, x > 0.f ? x : INFINITY);
                }
            }
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) v_max = fmaxf(v_max, __shfl_xor_sync(0xffffffffu, v_max, o));
    if (lane == 0) S.v_max[warp] = v_max;
    if constexpr (BITS == 4) {
#pragma unroll
        for (int o = 16; o; o >>= 1) v_min = fminf(v_min, __shfl_xor_sync(0xffffffffu, v_min, o));
        if (lane == 0) S.v_min[warp] = v_min;
        if constexpr (!kFolded) {
#pragma unroll
            for (int o = 16; o; o >>= 1) k_max = fmaxf(k_max, __shfl_xor_sync(0xffffffffu, k_max, o));
            if (lane == 0) S.k_max[warp] = k_max;
        }
    }
    put_queries<D, QT, DT, BITS>(g, gbase, S.factor, o0, h, tq, len, row0, row_end);
    }
    fence_async_shared();  // the queries are read by the tensor cores
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // All of the SM's tensor memory is this CTA's, so it begins at 0.
    constexpr uint32_t tmem = 0;
    const volatile Job& job = S.job;
    // The first step before which outputs are taken out, so that O begins anew there.
    auto first_drain = [&]() {
        return DRAIN > 0 && (DT == Q4LIN_DTYPE_F32 || job.cut || job.slot >= 0) ? DRAIN : INT_MAX;
    };
    // What the values' scales are taken relative to: the largest of the walk, folded ones a power of
    // two that brings it to [2^11, 2^12), so that codes times scales fill fp16's range.
    auto value_ref = [&]() {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v = fmaxf(v, const_cast<volatile float&>(S.v_max[w]));
        if constexpr (kFolded) return __uint_as_float(min(max((int)(__float_as_uint(v) >> 23) - 11, 1), 253) << 23);
        return v > 0.f ? v : 1.f;  // 1: values that are all zero
    };
    // What the keys' scales are taken relative to where they multiply scores before the row's factor does: 1, or for
    // scales above 2^64 a power of two that brings the largest there, as a score may be an ordinary one where neither
    // that nor the factor is.
    auto key_ref = [&]() {
        if constexpr (kFolded || BITS == 8) return 1.f;
        const uint32_t most = __reduce_max_sync(0xffffffffu, lane < kWarps ? __float_as_uint(S.k_max[lane]) : 0u);
        return __uint_as_float((max(most >> 23, 127u + 64u) - 64u) << 23);
    };
    // (By a whole warp; positive floats are ordered as their bits.)
    auto wide_walk = [&]() {
        if constexpr (BITS == 8) return false;
        const uint32_t most = __reduce_max_sync(0xffffffffu, lane < kWarps ? __float_as_uint(S.v_max[lane]) : 0u);
        const uint32_t least = __reduce_min_sync(0xffffffffu, lane < kWarps ? __float_as_uint(S.v_min[lane]) : 0x7F800000u);
        return __uint_as_float(least) * (kFolded ? kWideFolded : kWideWeights) < __uint_as_float(most);
    };
    volatile int* failed = &S.failed;
    auto bar = [](uint64_t& x) { return smem_u32(&x); };
    // In line (a call would tie the warpgroups' registers together), bounded as everywhere.
    auto wait_for = [&](uint64_t& x, uint32_t parity, int64_t limit, const volatile int* stop) {
        if (mbar_try_wait(bar(x), parity)) return true;
        const uint64_t t0 = global_timer();
        while (!mbar_try_wait(bar(x), parity))
            if ((stop && *stop) || (int64_t)(global_timer() - t0) > limit) return false;
        return true;
    };
    auto wait = [&](uint64_t& x, uint32_t parity) {
        if (wait_for(x, parity, g.wait_ns, failed)) return true;
        record_failure(g.status, failed);
        return false;
    };

    if (warp < kSoftWarps) {
        // -------------------------------------------------------------- softmax
        more_registers<soft_regs(D, kFolded)>();
        const int tq = job.tq, len = job.len, row0 = job.row0, row_end = job.row_end;
        const int n = job.n, step0 = job.step0;
        const int tile = warp >> 2;
        const int r = tile * kQ + (warp & 3) * 32 + lane, row = row0 + r;
        const bool in = row < row_end;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lanes + kScoreCol + tile * kKeys, o_at = tmem + lanes + tile * 128;
        const int token = row / group, position = len - tq + token;
        const int limit = !in ? -1 : g.a.causal ? position : len - 1;
        const int low = g.a.window > 0 ? (int)max((int64_t)0, (int64_t)position - g.a.window + 1) : 0;
        float factor = S.factor[r];
        if constexpr (kKeyed && !kFolded) {  // (not so small that a masked score would not stay -infinity)
            factor *= key_ref();
            factor = factor < kLeastFactor ? kLeastFactor : factor;  // (a NaN stays one)
        }
        int drain = first_drain();
        float m = -INFINITY, l = 0.f, m_out = -INFINITY;  // m_out: of what was taken out
        bool ok = true;
        const int steps = tile == 0 || row_end - row0 > kQ ? n : 0;
        [[maybe_unused]] auto ratios_of = [&](int slot) -> const float2* {
            if constexpr (kKeyed)
                return reinterpret_cast<const float2*>(S.scales.v_ratio[slot]);
            else
                return nullptr;
        };
        auto walk = [&](auto is_wide) {
            constexpr bool kWide = decltype(is_wide)::value;
            for (int i = 0; i < steps; ++i) {
                ok = __all_sync(0xffffffffu, wait(S.s_full[tile], i & 1));
                if (!ok) break;
                tc_fence_after();
                const int key0 = (step0 + i) * kKeys, slot = i % Scales::kSlots;
                const int hi = min(limit - key0, kKeys), lo = max(low - key0, 0);
                if constexpr (kKeyed && kWide) {
                    // Sixteen scores at a time, twice, in little code: unrolled, it made ordinary walks, which do not
                    // run it, 12 % slower.
                    auto sixteen = [&](int c, const uint32_t (&x)[16], float from, auto&& take) {  // take(pair, exponents, scales)
                        const float2* ks = reinterpret_cast<const float2*>(S.scales.k_scale[slot]) + 8 * c;
                        const float2* ratios = ratios_of(slot) + 8 * c;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int key = 16 * c + 2 * e;
                            const float2 s = make_float2(key > hi || key < lo ? -INFINITY : __uint_as_float(x[2 * e]),
                                                         key + 1 > hi || key + 1 < lo ? -INFINITY : __uint_as_float(x[2 * e + 1]));
                            const float2 f = ffma2(ks[e], make_float2(factor, factor), make_float2(kLeastFactor, kLeastFactor));
                            const Apart2 v = apart2(ratios[e]);
                            take(e, ffma2(s, f, fadd2(make_float2(from, from), v.exponent)), v);
                        }
                    };
                    float top = -INFINITY;
#pragma unroll 1
                    for (int c = 0; c < 8; ++c) {
                        uint32_t x[16];
                        tmem_ld16(s_at + 16 * c, x);
                        sixteen(c, x, 0.f, [&](int, float2 t, const Apart2&) { top = max3(top, t.x, t.y); });
                    }
                    top = ceilf(top);
                    if (__any_sync(0xffffffffu, top > m + kSlack)) {
                        const float now = fmaxf(m, top), alpha = now == -INFINITY ? 1.f : ex2(m - now);
                        m = now, l *= alpha;
#pragma unroll 1
                        for (int c = 0; c < (i > 0 ? D / 16 : 0); ++c) {
                            uint32_t y[16];
                            tmem_ld16(o_at + 16 * c, y);
#pragma unroll
                            for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * alpha);
                            tmem_st16_async(o_at + 16 * c, y);
                        }
                    }
                    if (DRAIN > 0 && i == drain) {
                        drain += DRAIN;
                        tmem_wait_st();  // as below
                        float* to = out_row<D, DT>(g, job, row, r);
                        const float keep = m_out == -INFINITY ? 0.f : ex2(m_out - m);
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t y[16];
                            __syncwarp();
                            tmem_ld16(o_at + 16 * c, y);
                            if (in) add_16(to + 16 * c, y, keep, i > DRAIN, true);
                        }
                        __syncwarp();
                        m_out = m;
                    }
                    const float origin = kBase - (m == -INFINITY ? 0.f : m);
                    float2 sum = make_float2(0.f, 0.f);
                    auto weigh = [&](int c, const uint32_t (&x)[16]) {
                        uint32_t p[8], rest[8];
                        sixteen(c, x, origin, [&](int e, float2 t, const Apart2& v) {
                            const float2 y = make_float2(ex2(t.x), ex2(t.y)), w = fmul2(y, v.rest);
                            sum = ffma2(y, v.inverse, sum);
                            split_f16(w.x, w.y, &p[e], &rest[e]);
                        });
                        tmem_st8_async(s_at + 8 * c, p);
                        if (PT == 2) tmem_st8_async(s_at + 64 + 8 * c, rest);
                    };
                    // Weights go over scores that have been read.  Their lower terms lie from column 64 on, so with two
                    // terms those scores are taken first (32 of them) or from the end.
                    [[maybe_unused]] uint32_t kept[2][16];
                    if constexpr (PT == 2) {
                        tmem_ld16(s_at + 64, kept[0]);
                        tmem_ld16(s_at + 80, kept[1]);
                    }
#pragma unroll 1
                    for (int k = 0; k < (PT == 2 ? 6 : 8); ++k) {
                        const int c = PT == 2 && k >= 4 ? 11 - k : k;
                        uint32_t x[16];
                        tmem_ld16(s_at + 16 * c, x);
                        weigh(c, x);
                    }
                    if constexpr (PT == 2) weigh(4, kept[0]), weigh(5, kept[1]);
                    l += sum.x + sum.y;
                } else if constexpr (kFolded) {
                    // The scores in quarters, the next one on its way.  The weights by the maximum that there
                    // is: as long as their sum stays in fp16's range, so does each of them, and no maximum is
                    // looked for.  They wait in registers until that is known; rows that have seen nothing yet
                    // and those whose sum has grown too far (each for itself) get a new maximum first.
                    const float4* ks = reinterpret_cast<const float4*>(S.scales.k_scale[slot]);
                    const float2 factor2 = make_float2(factor, factor), least2 = make_float2(kLeastFactor, kLeastFactor);
                    const bool masked = __any_sync(0xffffffffu, hi < kKeys - 1 || lo > 0);
                    auto quarters = [&](auto&& take) {  // take(quarter, its 32 scores)
                        uint32_t x[2][32];
                        tmem_ld32_async(s_at, x[0]);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            tmem_wait_ld32(x[c % 2]);
                            if (c < 3) tmem_ld32_async(s_at + 32 * (c + 1), x[(c + 1) % 2]);
                            if (masked) {
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (32 * c + e > hi || 32 * c + e < lo) x[c % 2][e] = 0xFF800000u;
                            }
                            take(c, x[c % 2]);
                        }
                    };
                    auto column_factors = [&](int e, float2& a, float2& b) {  // of columns 4 e .. 4 e + 3
                        const float4 k = ks[e];
                        a = ffma2(make_float2(k.x, k.y), factor2, least2), b = ffma2(make_float2(k.z, k.w), factor2, least2);
                    };
                    uint32_t p[kKeys / 2];
                    float2 sum;
                    bool need = in && m == -INFINITY;
#pragma unroll 1
                    for (int pass = 0; pass < 2; ++pass) {
                        if (__any_sync(0xffffffffu, need)) {
                            float top = -INFINITY;
                            quarters([&](int c, const uint32_t (&x)[32]) {
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    float2 a, b;
                                    column_factors(8 * c + e, a, b);
                                    a = fmul2(make_float2(__uint_as_float(x[4 * e]), __uint_as_float(x[4 * e + 1])), a);
                                    b = fmul2(make_float2(__uint_as_float(x[4 * e + 2]), __uint_as_float(x[4 * e + 3])), b);
                                    top = max3(max3(top, a.x, a.y), b.x, b.y);
                                }
                            });
                            const float now = need ? fmaxf(m, top) : m, alpha = now == -INFINITY ? 1.f : ex2(m - now);
                            m = now, l *= alpha;
                            if (i > 0) {
#pragma unroll
                                for (int c = 0; c < D / 16; ++c) {
                                    uint32_t y[16];
                                    tmem_ld16(o_at + 16 * c, y);
#pragma unroll
                                    for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * alpha);
                                    tmem_st16_async(o_at + 16 * c, y);
                                }
                                tmem_wait_st();  // a second pass may read them; loads do not wait for stores
                            }
                        }
                        const float origin = kBase - (m == -INFINITY ? 0.f : m);
                        const float2 off2 = make_float2(origin, origin);
                        sum = make_float2(0.f, 0.f);
                        quarters([&](int c, const uint32_t (&x)[32]) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                float2 w[2];
                                column_factors(8 * c + e, w[0], w[1]);
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    w[h] = ffma2(make_float2(__uint_as_float(x[4 * e + 2 * h]), __uint_as_float(x[4 * e + 2 * h + 1])), w[h], off2);
                                    w[h].x = ex2(w[h].x), w[h].y = ex2(w[h].y);
                                    sum = fadd2(sum, w[h]);
                                    const __half2 v = __floats2half2_rn(w[h].x, w[h].y);
                                    p[16 * c + 2 * e + h] = *reinterpret_cast<const uint32_t*>(&v);
                                }
                            }
                        });
                        need = sum.x + sum.y > kMostSum;
                        if (!__any_sync(0xffffffffu, need)) break;
                    }
                    l += sum.x + sum.y;
#pragma unroll
                    for (int c = 0; c < 8; ++c) tmem_st8_async(s_at + 8 * c, *reinterpret_cast<uint32_t(*)[8]>(p + 8 * c));
                } else {
                    uint32_t x[kKeys];
                    tmem_ld64(s_at, x);
                    tmem_ld64(s_at + 64, x + 64);
                    if constexpr (kKeyed) {
                        const float4* ks = reinterpret_cast<const float4*>(S.scales.k_scale[slot]);
#pragma unroll
                        for (int e = 0; e < kKeys / 4; ++e) {
                            const float4 s = ks[e];
                            const float2 a = fmul2(make_float2(__uint_as_float(x[4 * e]), __uint_as_float(x[4 * e + 1])), make_float2(s.x, s.y));
                            const float2 b = fmul2(make_float2(__uint_as_float(x[4 * e + 2]), __uint_as_float(x[4 * e + 3])), make_float2(s.z, s.w));
                            x[4 * e] = __float_as_uint(a.x), x[4 * e + 1] = __float_as_uint(a.y);
                            x[4 * e + 2] = __float_as_uint(b.x), x[4 * e + 3] = __float_as_uint(b.y);
                        }
                    }
                    // Columns [lo, hi] of the step are seen; all of them in most steps.
                    if (__any_sync(0xffffffffu, hi < kKeys - 1 || lo > 0)) {
#pragma unroll
                        for (int e = 0; e < kKeys; ++e)
                            if (e > hi || e < lo) x[e] = 0xFF800000u;
                    }
                    float top = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        float mx = max3(__uint_as_float(x[16 * c]), __uint_as_float(x[16 * c + 1]), __uint_as_float(x[16 * c + 2]));
#pragma unroll
                        for (int e = 3; e < 15; e += 2)
                            mx = max3(mx, __uint_as_float(x[16 * c + e]), __uint_as_float(x[16 * c + e + 1]));
                        mx = fmaxf(mx, __uint_as_float(x[16 * c + 15]));
                        if constexpr (BITS == 8)
                            top = fmaxf(top, mx * fmaxf(factor * S.scales.k_scale[slot][c], kLeastFactor));
                        else
                            top = fmaxf(top, mx);
                    }
                    if constexpr (BITS == 4) top *= factor;
                    if (__any_sync(0xffffffffu, top > m + kSlack)) {
                        // Some row's maximum grew too far: O and l over to the new one.  (The product
                        // that read the last weights is complete: this step's scores came after it.)
                        const float now = fmaxf(m, top);
                        const float alpha = now == -INFINITY ? 1.f : ex2(m - now);
                        m = now, l *= alpha;
                        if (i > 0) {
#pragma unroll
                            for (int c = 0; c < D / 16; ++c) {
                                uint32_t y[16];
                                tmem_ld16(o_at + 16 * c, y);
#pragma unroll
                                for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * alpha);
                                tmem_st16_async(o_at + 16 * c, y);
                            }
                        }
                    }
                    if (DRAIN > 0 && i == drain) {
                        drain += DRAIN;
                        tmem_wait_st();  // O may just have been rescaled; loads do not wait for stores
                        float* to = out_row<D, DT>(g, job, row, r);
                        const float keep = m_out == -INFINITY ? 0.f : ex2(m_out - m);
#pragma unroll DT == Q4LIN_DTYPE_F32 ? 4 : 8
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t y[16];
                            __syncwarp();  // the load is the whole warp's
                            tmem_ld16(o_at + 16 * c, y);
                            if (in) add_16(to + 16 * c, y, keep, i > DRAIN, true);
                        }
                        __syncwarp();
                        m_out = m;
                    }
                    const float origin = kBase - (m == -INFINITY ? 0.f : m);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        float f = factor, off = origin;
                        if constexpr (BITS == 8)
                            f = fmaxf(factor * S.scales.k_scale[slot][c], kLeastFactor), off = origin + S.scales.v_log[slot][c];
                        const float2 f2 = make_float2(f, f), off2 = make_float2(off, off);
                        float2 sum = make_float2(0.f, 0.f);
                        [[maybe_unused]] float4 ratio = make_float4(0.f, 0.f, 0.f, 0.f);
                        uint32_t p[8], rest[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float2 y = ffma2(make_float2(__uint_as_float(x[16 * c + 2 * e]), __uint_as_float(x[16 * c + 2 * e + 1])), f2, off2);
                            y.x = ex2(y.x), y.y = ex2(y.y);
                            sum = fadd2(sum, y);
                            if constexpr (kKeyed) {
                                if (e % 2 == 0) ratio = *reinterpret_cast<const float4*>(&S.scales.v_ratio[slot][16 * c + 2 * e]);
                                y = fmul2(y, e % 2 ? make_float2(ratio.z, ratio.w) : make_float2(ratio.x, ratio.y));
                            }
                            if (PT == 2) {
                                split_f16(y.x, y.y, &p[e], &rest[e]);
                            } else {
                                const __half2 v = __floats2half2_rn(y.x, y.y);
                                p[e] = *reinterpret_cast<const uint32_t*>(&v);
                            }
                        }
                        if constexpr (BITS == 8)
                            l = fmaf(sum.x + sum.y, S.scales.v_inv[slot][c], l);
                        else
                            l += sum.x + sum.y;
                        tmem_st8_async(s_at + 8 * c, p);  // over the scores
                        if (PT == 2) tmem_st8_async(s_at + 64 + 8 * c, rest);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(S.p_full[tile]));
            }
        };
        if (kKeyed && wide_walk())
            walk(std::bool_constant<kKeyed>{});
        else
            walk(std::false_type{});
        if (ok && steps > 0) {
            ok = __all_sync(0xffffffffu, wait(S.o_full[tile], 0));
            tc_fence_after();
        }
        // (A second tile without rows has nothing to store, and the first one's products may
        // still read the shared memory that the rows go through.)
        if (ok && (tile == 0 || row_end - row0 > kQ)) {
            // (Everything about the row anew: the loop has no registers to keep it in.)
            const int tid = thread_number(), r = tid, row = job.row0 + r;  // threads are rows
            const bool in = row < job.row_end, cut = job.cut;
            const int group = (int)(g.a.heads / C.kv_heads), token = row / group;
            const int64_t index = (job.o0 + token) * g.a.heads + job.h * group + (row - token * group);
            const float v_ref = value_ref(), inv = l != 0.f ? v_ref / l : 0.f;
            const uint32_t o_at = ((uint32_t)((tid >> 5) & 3) << 21) + (uint32_t)(r / kQ) * 128;
            float* unit = part_at<D>(g, blockIdx.x);
            // A thread's row goes through shared memory, where nothing else is wanted any more (its
            // pitch keeps the rows of a quarter-warp on banks of their own), and leaves by one
            // bulk copy: rows stored by their threads took 6 us more.
            const bool wide = cut || DT == Q4LIN_DTYPE_F32;
            const uint32_t row_bytes = wide ? 4 * D : 2 * D, out = base + (uint32_t)r * (4 * D + 16);
            static_assert(pair_rows_of(D) * (4 * D + 16) <= L::bytes, "the rows fit");
            float f = l == 0.f ? 0.f : cut ? v_ref : inv;
            if (BITS == 4 && cut && v_ref > 4294967296.f) {
                // (What the maximum loses as it is rounded goes into the sums.)
                const float more = m + kLessBits, by = fmaf((more - kLessBits) - m, -kLn2, 1.f) * kLess;
                if (m != -INFINITY) m = more, l *= by, f *= by;
            }
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t x[32];
                __syncwarp();  // the load is the whole warp's
                if (steps > 0) {
                    tmem_ld32(o_at + 32 * c, x);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = 0u;
                }
                if (DRAIN > 0 && drain > DRAIN && drain < INT_MAX && in) {
                    const float keep = m_out == -INFINITY ? 0.f : ex2(m_out - m);
                    float* from = out_row<D, DT>(g, job, row, r) + 32 * c;
                    add_16(from, *reinterpret_cast<uint32_t(*)[16]>(x), keep, true, false);
                    add_16(from + 16, *reinterpret_cast<uint32_t(*)[16]>(x + 16), keep, true, false);
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(l == 0.f ? 0.f : __uint_as_float(x[e]) * f);
                if (wide) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        st_shared_v4(out + 128 * c + 16 * e, x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            w[j] = to_16x2(__uint_as_float(x[8 * e + 2 * j]), __uint_as_float(x[8 * e + 2 * j + 1]),
                                           DT);
                        st_shared_v4(out + 64 * c + 16 * e, w[0], w[1], w[2], w[3]);
                    }
                }
            }
            // (What was taken out went through the generic proxy to the same place.)
            if (DRAIN > 0) asm volatile("fence.proxy.async;" ::: "memory");
            fence_async_shared();
            if (in) {
                void* to = cut ? static_cast<void*>(unit + r * D)
                               : static_cast<void*>(static_cast<uint8_t*>(g.a.out) + index * row_bytes);
                bulk_store(to, out, row_bytes);
            }
            if (in && cut) {
                unit[pair_rows_of(D) * D + r] = m, unit[pair_rows_of(D) * (D + 1) + r] = l;
            } else if (in && g.a.lse) {
                g.a.lse[index] = l != 0.f ? log2_sum(m == -INFINITY ? 0.f : m, l * kUnbase, BITS == 4) * kLn2 : -INFINITY;
            }
        }
    } else if (warp < kIssueWarp) {
        // ------------------------- codes into fp16 blocks: keys, and values, 128 threads each
        fewer_registers<widen_regs(D, kFolded)>();
        const int n = job.n, step0 = job.step0, pages = (job.len + (1 << ps) - 1) >> ps;
        const int page_low = job.page_low;
        const int32_t* table = C.page_table + job.b * C.table_stride;
        const bool keys = warp < kValueWarp;
        const float ref = value_ref();
        [[maybe_unused]] const bool wide = wide_walk();
        [[maybe_unused]] const float key_inverse = 1.f / key_ref();
        const int t = tid & 127;
        // One ring each, a step's blocks in the order of their use.
        auto walk = [&](auto&& widen) {
            if (keys)
                widen(S.k_full, S.k_empty, base + L::k, L::kBlock, L::kRing, L::kBlocks, C.k_codes);
            else
                widen(S.v_full, S.v_empty, base + L::v, L::vBlock, L::vRing, 2, C.v_codes);
        };
        // Head's share of the page of group `lane` of 16 keys of step i, -1 past the end and
        // before the window.
        auto fetch_pages = [&](int i) {
            const int p = ((step0 + i) * kKeys + lane * 16) >> ps;
            if (lane >= 8 || i >= n || p < page_low || p >= pages) return -1;
            const int id = __ldg(table + p);
            return (id < 0 || id >= C.num_pages ? 0 : id) * Hkv + h;
        };
        walk([&](uint64_t* full, uint64_t* empty, uint32_t ring, uint32_t block, int depth, int blocks,
                 const uint8_t* codes) {
            // 8 bits: a thread's pieces of 16 codes: of a block of keys, 16 channels of key t / 4 + 32 j
            // (t % 4); of a block of values, 16 keys of a channel, in the order of the page.
            // 4 bits: pieces of 32 codes: of a block of keys, of key t / 2 + 64 j (t % 2); of a block of
            // values, of whole tokens, in the order of the page.
            [[maybe_unused]] const int count = keys ? 4 : D / 32;  // (8 bits) pieces per thread and block
            const uint32_t page_bytes = (uint32_t)(D * BITS / 8) << ps;
            // A value's scale over the reference; 1 in wide walks.
            [[maybe_unused]] const float inverse = wide ? 0.f : 1.f / ref, one = wide ? 1.f : 0.f;
            uint4 reg[BITS == 4 && D < 256 ? 2 : 4];
            // 16-byte chunks of a token's 4-bit codes; values' rows of a block that a thread has a chunk of.
            [[maybe_unused]] constexpr int kChunks = D / 32, kValueRows = D / 64;
            [[maybe_unused]] float scale[D == 256 ? 4 : 2];  // of the values
            int pages_now = fetch_pages(0), pages_next = fetch_pages(1);
            auto load = [&](int page_ids, int blk) {
                if constexpr (BITS == 4) {
                    constexpr uint32_t kRow = D / 2;  // bytes of a token's codes
                    if (keys) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t key = t / 2 + 64 * j;
                            const int page = __shfl_sync(0xffffffffu, page_ids, key / 16);
                            reg[j] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
                            if (page >= 0)
                                ld_codes(codes + (uint64_t)(uint32_t)page * page_bytes + (key & (1u << ps) - 1) * kRow +
                                             blk * 32 + t % 2 * 16, reg[j]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < kValueRows; ++j) {
                            const uint32_t key = 64 * blk + t / kChunks + 128 / kChunks * j;
                            const int page = __shfl_sync(0xffffffffu, page_ids, key / 16);
                            const uint32_t in_page = key & (1u << ps) - 1;
                            reg[j] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
                            if constexpr (kFolded) scale[j] = 0.f;
                            if (page >= 0) {
                                ld_codes(codes + (uint64_t)(uint32_t)page * page_bytes + in_page * kRow + t % kChunks * 16, reg[j]);
                                if constexpr (kFolded) scale[j] = __ldg(C.v_scales + ((int64_t)page << ps) + in_page);
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (j >= count) continue;
                        uint32_t group, at;
                        if (keys) {
                            const uint32_t key = t / 4 + 32 * j;
                            group = key / 16, at = (key & (1u << ps) - 1) * D + blk * 64 + t % 4 * 16;
                        } else {
                            const uint32_t q = t + 128 * j;
                            group = q / D, at = q * 16 & page_bytes - 1;
                            group += 4 * blk;
                        }
                        const int page = __shfl_sync(0xffffffffu, page_ids, group);
                        reg[j] = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
                        if (page >= 0) ld_codes(codes + (uint64_t)(uint32_t)page * page_bytes + at, reg[j]);
                    }
                }
            };
            // (first: the block's first key, for scales that are behind the sequence.)
            auto store = [&](uint32_t to, [[maybe_unused]] int first) {
                if constexpr (BITS == 4) {
                    if (keys) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t w[4] = {reg[j].x, reg[j].y, reg[j].z, reg[j].w};
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                uint32_t f[4];
                                nibbles_f16(w[c], f[0], f[1], f[2], f[3]);
                                st_shared_v4(to + swizzled(t / 2 + 64 * j, t % 2 * 4 + c), f[0], f[1], f[2], f[3]);
                            }
                        }
                    } else {
                        // Rows of a key's 64 channels, as the products take them with this operand the other
                        // way round; every further 64 channels in rows of their own behind the first, every
                        // second 64 written in another order so that all banks are.
                        const int chunk = t % kChunks, half = chunk / 2, odd = half % 2;
#pragma unroll
                        for (int j = 0; j < kValueRows; ++j) {
                            const int row = t / kChunks + 128 / kChunks * j;
                            const uint32_t w[4] = {odd ? reg[j].z : reg[j].x, odd ? reg[j].w : reg[j].y,
                                                   odd ? reg[j].x : reg[j].z, odd ? reg[j].y : reg[j].w};
                            [[maybe_unused]] uint32_t hi, lo;
                            if constexpr (kFolded) {
                                const float s = first + row < job.len ? fmaf(scale[j], inverse, one) : 0.f;
                                split_f16(s, s, &hi, &lo);
                            }
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                uint32_t f[4];
                                nibbles_f16(w[c], f[0], f[1], f[2], f[3]);
                                if constexpr (kFolded) {
#pragma unroll
                                    for (int n = 0; n < 4; ++n) f[n] = scaled_f16(f[n], hi, lo);
                                }
                                st_shared_v4(to + half * (64 * 128) + swizzled(row, chunk % 2 * 4 + (c ^ 2 * odd)),
                                             prmt(f[0], f[1], 0x5410u), prmt(f[2], f[3], 0x5410u),
                                             prmt(f[0], f[1], 0x7632u), prmt(f[2], f[3], 0x7632u));
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (j >= count) continue;
                        uint32_t row, c;  // of 128 bytes, and its 32-byte piece
                        if (keys) {
                            row = t / 4 + 32 * j, c = t % 4;
                        } else {
                            const uint32_t q = t + 128 * j, rem = q & (page_bytes >> 4) - 1;
                            row = rem >> ps - 4, c = q / D & ~((1u << ps - 4) - 1) | rem & (1u << ps - 4) - 1;
                        }
                        uint32_t f[8];
                        codes_f16(reg[j].x, &f[0], &f[1]);
                        codes_f16(reg[j].y, &f[2], &f[3]);
                        codes_f16(reg[j].z, &f[4], &f[5]);
                        codes_f16(reg[j].w, &f[6], &f[7]);
                        const uint32_t chunk = to + swizzled(row, 2 * c);
                        st_shared_v4(chunk, f[0], f[1], f[2], f[3]);
                        st_shared_v4(chunk ^ 16, f[4], f[5], f[6], f[7]);
                    }
                }
            };
            int slot = 0;
            uint32_t par = 1;  // nothing to wait for in the ring's first round
            load(pages_now, 0);
            for (int i = 0; i < n && !(keys && g.skip_first_copy); ++i) {
                for (int blk = 0; blk < blocks; ++blk) {
                    // (With the keys: the softmax needs both scales once the scores are there.)
                    const bool scales = keys && blk == 0 && (BITS == 4 || t < 8);
                    float ks = 0.f, vs = 0.f;
                    if constexpr (kKeyed) {
                        // Key t of the step; 0 for those behind the sequence and before the window.
                        if (keys && blk == 0) {
                            const int page = __shfl_sync(0xffffffffu, pages_now, t / 16), key = (step0 + i) * kKeys + t;
                            if (page >= 0 && key < job.len) {
                                const int64_t at = ((int64_t)page << ps) + (key & (1 << ps) - 1);
                                ks = __ldg(C.k_scales + at);
                                if (!kFolded || wide) vs = __ldg(C.v_scales + at);
                            }
                        }
                    } else if (scales && pages_now >= 0) {
                        ks = __ldg(C.k_scales + pages_now), vs = __ldg(C.v_scales + pages_now);
                    }
                    if (!__all_sync(0xffffffffu, wait(empty[slot], par))) return;
                    if (scales) {
                        // Far below fp16's range a weight is 0 in the product; in l it counts.
                        const int at = i % Scales::kSlots;
                        if constexpr (kKeyed) {
                            S.scales.k_scale[at][t] = kFolded ? ks : ks * key_inverse;
                            if (!kFolded || wide) S.scales.v_ratio[at][t] = vs / ref;
                        } else if constexpr (BITS == 8) {
                            const float ratio = fmaxf(vs / ref, kLeastRatio);
                            S.scales.k_scale[at][t] = ks, S.scales.v_log[at][t] = lg2(ratio), S.scales.v_inv[at][t] = 1.f / ratio;
                        }
                    }
                    store(ring + (uint32_t)slot * block, (step0 + i) * kKeys + 64 * blk);
                    fence_async_shared();
                    mbar_arrive(bar(full[slot]));
                    if (++slot == depth) slot = 0, par ^= 1u;
                    if (blk + 1 < blocks) {
                        load(pages_now, blk + 1);
                    } else {
                        load(pages_next, 0);
                        pages_now = pages_next, pages_next = fetch_pages(i + 2);
                    }
                }
            }
        });
    } else {
        // ------------------------------------------------------------ MMA issue
        fewer_registers<kIssueRegs>();
        const int n = job.n;
        const bool two = job.row_end - job.row0 > kQ;
        if (warp == kIssueWarp && n > 0) {
            const uint32_t leader = elect_one();
            // (4 bits: values as rows of channels, so that the summed axis is the other one.)
            const uint32_t idesc_s = f16_idesc(kQ, kKeys), idesc_o = f16_idesc(kQ, D) | (BITS == 4 ? 1u << 16 : 0u);
            // Low words of the descriptors; 32 bytes along a swizzled row are 2 in their address
            // field, a block of 64 channels (keys) is kBlock / 16 (the high words are all alike).
            const uint64_t desc0 = sw128_desc(base);
            const uint32_t high = (uint32_t)(desc0 >> 32), low0 = (uint32_t)desc0;
            auto desc = [&](uint32_t low_word) { return (uint64_t)high << 32 | low_word; };
            bool ok = true;
            int k_slot = 0, v_slot = 0;  // of the first block of this step's tile
            int drain = first_drain();
            bool begins = true;  // O begins anew at this step
            uint32_t k_par = 0, v_par = 0;
            // One tile's products of a step.  The step's first tile waits for the blocks, its last
            // one releases them and moves on in the ring.
            auto scores = [&](int tile, bool first, bool last) {
                int slot = k_slot;
                uint32_t par = k_par;
#pragma unroll
                for (int kb = 0; kb < L::kBlocks; ++kb) {
                    if (first) {
                        ok = ok && __all_sync(0xffffffffu, wait(S.k_full[slot], par));
                        if (!ok) return;
                        tc_fence_after();
                    }
                    const uint32_t k_low = low0 + ((L::k + (uint32_t)slot * L::kBlock) >> 4);
#pragma unroll
                    for (int term = 0; term < QT; ++term) {
                        const uint32_t q_low =
                            low0 + ((L::q + (uint32_t)((tile * QT + term) * L::kBlocks + kb) * L::kBlock) >> 4);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_f16_ss(leader, tmem + kScoreCol + tile * kKeys, desc(q_low + 2 * kk),
                                       desc(k_low + 2 * kk), idesc_s, kb + term + kk > 0);
                    }
                    if (last) mma_commit(leader, bar(S.k_empty[slot]));
                    if (++slot == L::kRing) slot = 0, par ^= 1u;
                }
                if (last) k_slot = slot, k_par = par;
                mma_commit(leader, bar(S.s_full[tile]));
            };
            auto outputs = [&](int tile, int i, bool first, bool last) {
                int slot = v_slot;
                uint32_t par = v_par;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (first) {
                        ok = ok && __all_sync(0xffffffffu, wait(S.v_full[slot], par));
                        if (!ok) return;
                    }
                    if (half == 0) {
                        ok = ok && __all_sync(0xffffffffu, wait(S.p_full[tile], i & 1));
                        if (!ok) return;
                    }
                    tc_fence_after();
                    // Of 16 keys: 32 bytes of a channel's row; or 16 rows, with the second half of the
                    // channels (in the descriptor, where rows along the summed axis have a 1) 8 KB away, and so on.
                    constexpr uint32_t kStep = BITS == 4 ? 16 * 128 / 16 : 2, kOther = BITS == 4 ? 64 * 128 / 16 - 1 : 0;
                    const uint32_t v_low = low0 + (kOther << 16) + ((L::v + (uint32_t)slot * L::vBlock) >> 4);
#pragma unroll
                    for (int term = 0; term < PT; ++term)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_f16_ts(leader, tmem + tile * 128,
                                       tmem + kScoreCol + tile * kKeys + term * 64 + (half * 4 + kk) * 8,
                                       desc(v_low + kStep * kk), idesc_o,
                                       !begins || half + term + kk > 0);
                    if (last) mma_commit(leader, bar(S.v_empty[slot]));
                    if (++slot == L::vRing) slot = 0, par ^= 1u;
                }
                if (last) v_slot = slot, v_par = par;
            };
            scores(0, true, !two);
            if (ok && two) scores(1, false, true);
            for (int i = 0; ok && i < n; ++i) {
                const bool more = i + 1 < n;
                if (DRAIN > 0 && i == drain) begins = true, drain += DRAIN;
                outputs(0, i, true, !two);
                if (ok && more) scores(0, true, !two);
                if (ok && two) outputs(1, i, false, true);
                begins = false;
                if (ok && two && more) scores(1, false, true);
            }
            // Everything issued has completed when these arrive; tensor memory is freed after.
            mma_commit(leader, bar(S.o_full[0]));
            mma_commit(leader, bar(S.o_full[1]));
            wait_for(S.o_full[1], 0, kDrainNs, nullptr);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kIssueWarp) tmem_dealloc(tmem, kTmemCols);
    if (DRAIN > 0 && DT != Q4LIN_DTYPE_F32 && thread_number() == 0 && S.job.slot >= 0) {
        __threadfence();  // (the rows' threads have read what was theirs before the barrier)
        atomicExch(g.taken + S.job.slot, 0);
    }
}

// The rows of walks that were cut: a warp takes PER rows of a pair of tiles, ROWS at a time with
// AHEAD parts of each in flight, in the order of the keys.
constexpr int kJoinWarps = 4;
template <int D, int PER, int ROWS, int AHEAD>
__device__ __forceinline__ void join_rows(const PromptArgs& g, int64_t unit0, int stride, int count, int r0, int rows,
                                          int64_t index0, int head0, int group) {
    const int lane = threadIdx.x & 31;
    const bool on = lane < D / 4;
    // (128 channels at a time.)
#pragma unroll 1
    for (int v = 0; v < PER * (D == 256 ? 2 : 1); v += ROWS) {
        const int r = r0 + v % PER, unit4 = v / PER * 32 + lane;
        float mx[ROWS], l[ROWS];
        float4 o[ROWS];
#pragma unroll
        for (int q = 0; q < ROWS; ++q) mx[q] = -INFINITY, l[q] = 0.f, o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int c = 0; c < count; c += AHEAD) {
            float pm[ROWS][AHEAD], pl[ROWS][AHEAD];
            float4 po[ROWS][AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const float* unit = part_at<D>(g, unit0 + (int64_t)(c + k) * stride);
#pragma unroll
                for (int q = 0; q < ROWS; ++q) {
                    pm[q][k] = -INFINITY, pl[q][k] = 0.f, po[q][k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (c + k < count && r + q < rows) {
                        pm[q][k] = __ldcg(unit + pair_rows_of(D) * D + r + q), pl[q][k] = __ldcg(unit + pair_rows_of(D) * (D + 1) + r + q);
                        if (on) po[q][k] = __ldcg(reinterpret_cast<const float4*>(unit + (r + q) * D) + unit4);
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < ROWS; ++q) {
                float top = mx[q];
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) top = fmaxf(top, pm[q][k]);
                const float from = top == -INFINITY ? 0.f : top, old = ex2(mx[q] - from);
                o[q].x *= old, o[q].y *= old, o[q].z *= old, o[q].w *= old, l[q] *= old, mx[q] = top;
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    const float w = ex2(pm[q][k] - from);
                    o[q].x = fmaf(po[q][k].x, w, o[q].x), o[q].y = fmaf(po[q][k].y, w, o[q].y);
                    o[q].z = fmaf(po[q][k].z, w, o[q].z), o[q].w = fmaf(po[q][k].w, w, o[q].w);
                    l[q] = fmaf(pl[q][k], w, l[q]);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
            if (r + q >= rows) break;
            const float inv = l[q] != 0.f ? 1.f / l[q] : 0.f;
            const int at = head0 + r + q, step = at / group;  // tokens from index0's
            const int64_t index = index0 + step * g.a.heads + (at - step * group);
            if (on && g.a.dtype == Q4LIN_DTYPE_F32)
                reinterpret_cast<float4*>(static_cast<float*>(g.a.out) + index * D)[unit4] =
                    make_float4(o[q].x * inv, o[q].y * inv, o[q].z * inv, o[q].w * inv);
            else if (on)
                reinterpret_cast<uint2*>(static_cast<unsigned short*>(g.a.out) + index * D)[unit4] =
                    make_uint2(to_16x2(o[q].x * inv, o[q].y * inv, g.a.dtype), to_16x2(o[q].z * inv, o[q].w * inv, g.a.dtype));
            if (unit4 == 0 && g.a.lse)
                g.a.lse[index] = l[q] != 0.f ? log2_sum(mx[q] == -INFINITY ? 0.f : mx[q], l[q] * kUnbase, g.bits == 4) * kLn2 : -INFINITY;
        }
    }
}
template <int D, int PER, int ROWS, int AHEAD>
__global__ void __launch_bounds__(32 * kJoinWarps) attention_prompt_join_kernel(const PromptArgs g) {
    const int i = ((int)blockIdx.x * kJoinWarps + (int)(threadIdx.x >> 5)) * PER;
    const int Hkv = (int)g.cache.kv_heads, group = (int)(g.a.heads / g.cache.kv_heads);
    const int u = i / pair_rows_of(D), r0 = i % pair_rows_of(D), h = u % Hkv;
    griddep_wait();
    // (The launch has no more pairs than the plan has room for: their records come with it.)
    const int pair = u / Hkv;
    const int4 plan = __ldcg(g.plan), j0 = __ldcg(g.plan + 1 + 2 * pair), j1 = __ldcg(g.plan + 2 + 2 * pair);
    const int parts = plan.x, each = plan.y;
    if (parts == 1 || pair >= plan.z) return;
    const int row0 = j0.w * pair_rows_of(D), rows = min(j0.y * group - row0, pair_rows_of(D));
    if (r0 >= rows) return;
    const int count = max(1, (j1.y - j1.x + each - 1) / each);
    // Row r is head head0 + r of the pair's first token, the heads of a group counted on.
    const int token = row0 / group, head0 = row0 - token * group;
    const int64_t index0 = ((int64_t)j1.z + token) * g.a.heads + h * group;
    join_rows<D, PER, ROWS, AHEAD>(g, (int64_t)pair * parts * Hkv + h, Hkv, count, r0, rows, index0, head0, group);
}

template <int D, int QT, int PT, int DT, int DRAIN, int BITS>
cudaError_t launch(PromptArgs& g, int64_t pairs_most, const LaunchCtx& c) {
    constexpr bool kKeyed = BITS == 4;
    constexpr int bytes = Layout<D, QT, kKeyed>::bytes + 1024;
    static_assert(bytes + sizeof(PromptShared<D, kKeyed>) <= 227 * 1024, "shared memory of one SM");
    // One CTA holds an SM (it takes all of its tensor memory).
    constexpr int asked = bytes > 116 * 1024 ? bytes : 116 * 1024;
    cudaError_t e = kernel_smem_once<attention_prompt_kernel<D, QT, PT, DT, DRAIN, BITS>>(asked);
    if (e != cudaSuccess) return e;
    // Parts only where whole walks leave SMs idle, and as the workspace allows.
    const int64_t units = std::max<int64_t>(1, pairs_most) * g.cache.kv_heads;
    const int64_t head = kDrainSlots + 4 + 8 * pairs_most;  // floats, a multiple of 4
    if (head > c.ws_floats / 2) return cudaErrorInvalidValue;
    const int64_t room = (c.ws_floats - head) / (pair_rows_of(D) * (D + 2));
    g.slots = c.sm_count;
    g.pairs_most = (int)pairs_most;
    g.taken = reinterpret_cast<int*>(c.ws);
    g.drain_slots = (int)std::min<int64_t>(room, std::min(kDrainSlots, c.sm_count));
    g.plan = reinterpret_cast<int4*>(c.ws + kDrainSlots);
    g.parts = c.ws + head;
    g.most_parts = units <= c.sm_count ? 64 : 1;
    int64_t grid = g.most_parts == 1 ? units : std::min(std::max<int64_t>(units, 2 * c.sm_count), room);
    if (BITS == 4 && units > c.sm_count) {
        // Where few more walks than SMs leave most SMs idle in the last round, too (1280 tokens, 4 heads on each
        // of 8 of 128, 160 walks: after 6912 others in bf16 277 -> 254 us, in fp32 538 -> 432, after 64000
        // 2300 -> 1618), if walks as long as the page table allows would be cut: the launch costs 3 us where the
        // plan then finds that they are too short.
        const int64_t longest = g.cache.pages_per_sequence * g.cache.page_size / kKeys + 1;
        int64_t best = 1;
        for (int64_t n = 2; n <= 64 && n * units <= room; ++n)
            if (cost_of(units, g.slots, longest, n) < cost_of(units, g.slots, longest, best)) best = n;
        g.most_parts = best > 1 ? 64 : 1, grid = best * units;
    }
    if (grid < units) g.most_parts = 1;
    const int64_t ctas = std::max(grid, units);
    attention_prompt_plan_kernel<<<1, kPlanThreads, 0, c.stream>>>(g, (int)std::min<int64_t>(ctas, INT32_MAX));
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // The launches of the next kernels overlap the ones before; they wait for their ends on the
    // device.
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t main = {};
    main.gridDim = dim3((unsigned)ctas);
    main.blockDim = dim3(kThreads);
    main.dynamicSmemBytes = asked;
    main.stream = c.stream;
    main.attrs = &attr;
    main.numAttrs = 1;
    e = cudaLaunchKernelEx(&main, attention_prompt_kernel<D, QT, PT, DT, DRAIN, BITS>, g);
    if (e != cudaSuccess || g.most_parts == 1) return e;
    // A row a warp while all of them fit on the SMs at once, more beyond (8 key/value heads of 128,
    // 4 query heads each, us for 1 / 4 rows a warp: 32 queries on 8192 keys 25.9 / 34.9, 128 40.1 /
    // 42.8, 300 on 2000 39.4 / 36.6, 512 on 8192 91.4 / 86.8, in fp32, without what is taken
    // out, 130.5 / 125.5).
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.stream = c.stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (g.a.tokens * g.a.heads <= 40 * c.sm_count) {
        cfg.gridDim = dim3((unsigned)(units * (pair_rows_of(D) / kJoinWarps)));
        return cudaLaunchKernelEx(&cfg, attention_prompt_join_kernel<D, 1, 1, 8>, g);
    }
    cfg.gridDim = dim3((unsigned)(units * (pair_rows_of(D) / (4 * kJoinWarps))));
    return cudaLaunchKernelEx(&cfg, attention_prompt_join_kernel<D, 4, 2, 4>, g);
}

// Sequences of more than `rows_min` query rows per key/value head.
template <int BITS>
cudaError_t prompt_launch(const q4lin_kv_cache_t& cache, const q4lin_attention_t& a, int64_t rows_min,
                          const LaunchCtx& c) {
    const int64_t rows = a.tokens * (a.heads / cache.kv_heads);
    cudaError_t e = cudaSuccess;
    for (int64_t b = 0; b < cache.batch && e == cudaSuccess; b += kMaxBatch) {
        PromptArgs g;
        g.cache = cache;
        g.a = a;
        g.cache.batch = std::min<int64_t>(kMaxBatch, cache.batch - b);
        g.cache.page_table += b * cache.table_stride;
        g.a.offsets += b;
        g.a.lengths += b;
        g.page_shift = cache.page_size == 16 ? 4 : cache.page_size == 32 ? 5 : 6;
        g.bits = BITS;
        g.rows_min = rows_min;
        g.q_vec = reinterpret_cast<uintptr_t>(a.query) % (4 * dtype_size(a.dtype)) == 0 &&
                  a.q_token_stride % 4 == 0 && a.q_head_stride % 4 == 0;
        g.status = c.status_word;
        g.wait_ns = c.wait_limit_ns;
        g.skip_first_copy = c.tc_skip_first_copy;
        // Pairs of all sequences at most: each taken one has more than rows_min rows.
        g.pair_rows = pair_rows_of(cache.head_dim);
        const int64_t pairs = rows / g.pair_rows + std::min(g.cache.batch, rows / (rows_min + 1));
        const bool few = cache.pages_per_sequence * cache.page_size <= kFewKeys;
        auto typed = [&](auto dim) {
            // One term where it is exact (see the head of this file).
            constexpr int f32 = Q4LIN_DTYPE_F32, f16 = Q4LIN_DTYPE_F16, bf16 = Q4LIN_DTYPE_BF16, D = decltype(dim)::value;
            if (a.dtype == bf16 && !a.rope.cos) return launch<D, 1, 1, bf16, 0, BITS>(g, pairs, c);
            if (a.dtype == bf16) return launch<D, 2, 1, bf16, 0, BITS>(g, pairs, c);
            if (a.dtype == f16 && few) return launch<D, 2, 2, f16, 0, BITS>(g, pairs, c);
            if (a.dtype == f16) return launch<D, 2, 2, f16, kDrainF16, BITS>(g, pairs, c);
            return launch<D, 2, 2, f32, kDrainF32, BITS>(g, pairs, c);
        };
        if (cache.head_dim == 64)
            e = typed(std::integral_constant<int, 64>{});
        else if (cache.head_dim == 128)
            e = typed(std::integral_constant<int, 128>{});
        else if constexpr (BITS == 4)
            e = typed(std::integral_constant<int, 256>{});
    }
    return e;
}

}  // namespace
}  // namespace q4lin
