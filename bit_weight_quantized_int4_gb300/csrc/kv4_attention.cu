// kv4_attention.cu -- attention of a few query rows per key/value head over the paged 4-bit
// cache: single tokens, draft tokens, short chunks.
//
// The keys of all sequences and heads are one list of 64-key tiles, cut evenly over the GPU's warps
// (attention_split.cuh); a warp works alone, with its own ring of copies.
//
// Bound: the codes and scales, head_dim + 8 bytes per key and key/value head; at half the bytes of an
// 8-bit cache also the instructions of a tile, about 1150 a warp, 576 of which widen codes.  Measured (8
// key/value heads of 128, 4 query heads each): 64 sequences of up to 8192 tokens, 347 MB, 74.5 us: 4.7
// TB/s, 0.69 of a copy's bandwidth (without widening any code 11 us less); one sequence of 131071 tokens, 143
// MB, 39.3 us, 8 of it the start and the join; one of 701 tokens 8.7 us.  Heads of 64 / 256: 51 us (0.53)
// and 127 us (0.78); eight and sixteen query heads a key head 108 and 205 us.
//
// Products on the tensor cores (m16n8k16, fp16 operands, fp32 sums), transposed: keys (channels of
// the values) are the MMA's 16 rows, and a query row takes two of its 8 columns, the rounded value
// and what the rounding left (22 bits).  So four query rows, a key head's in most models, fill a
// tile, where as the MMA's rows they would fill half of one.  Codes - 8 are exact in fp16; a token's
// scales multiply its score and its weight in fp32.  Both kinds lie in memory as rows of a token's
// codes, so a page is copied as it is, by tensor copies that swizzle 16-byte chunks: a lane reads
// its keys' chunks, and the values come by ldmatrix.trans, which pairs the same four channels of
// neighbouring keys, without bank conflicts.  A masked nibble is widened by one addition: 0x6400 | c
// is 1024 + c in fp16, 0x6400 | 16 c is 1024 + 16 c.  Channels are permuted alike in queries and keys
// so that the nibbles of a word that lie 16 bits apart are neighbours along the summed axis.
#include "attention_split.cuh"

namespace q4lin {
namespace {

// CT tiles of 8 columns, 4 query rows each.  Warps in fours: one too many for a scheduler holds all of
// them up (64 sequences as above, 8 / 12 / 16 warps: 78, 73, 77 us, 10 and 14 more than any; two tiles, 8
// and 12: 108, 133; heads of 64, 12 / 16 / 20: 54, 54, 62, two tiles 74 with 12, 79 with 16, four 121 with
// 8, 167 with 12).
__host__ __device__ constexpr int warps_of(int D, int CT) {
    return D == 64 ? (CT <= 2 ? 12 : 8) : D == 128 && CT == 1 ? 12 : 8;
}

// Weights are 2 to the power of scores less a maximum that they may have passed by up to 2^10.  For the product
// with the values' codes a row's, times the values' scales, are brought to fp16's upper range by a power of two
// for each tile: of the largest of them, in which only keys that the row sees have a part, so that two terms
// leave 2^-22 of that however small a value is beside those that the row does not see.  Sums of values are kept
// over 2^20, so that those near fp32's largest have room.
constexpr float kMostWeight = 1024.f, kLess = 1.f / 1048576.f, kMore = 1048576.f;

struct KvMaps {
    CUtensorMap k, v;  // [page and head][token][bytes of a token]
};

template <int D, int CT>
struct Mine {  // of one warp
    uint2 q[CT][D / 16][32];  // B fragments
    RowInfo row[CT * 4];
    float scales[2][kTile];  // of a tile's keys, and values over 2^20
};
template <int D, int CT>
struct Layout {
    static constexpr int W = warps_of(D, CT);
    static constexpr uint32_t codes = kTile * D / 2;  // of half a tile: keys or values
    static constexpr int other = W * ((int)sizeof(Mine<D, CT>) + 4) + 4 * (kMaxBatch + 1) + 64 + 1024;
    // Half tiles in a warp's ring: three, where they fit (with more the first copies of all warps hold one
    // another up: one sequence of 131071 tokens 38.6 us, with four 40.6; 64 sequences of heads of 64 with
    // 2, 3, 4, 8: 50.7, 50.3, 50.5, 53.6).
    static constexpr int fit = (227 * 1024 - other) / (W * (int)(codes + 8)), slots = fit < 3 ? fit : 3;
    static_assert(slots >= 2, "a tile's keys and values fit");
};
template <int D, int CT>
struct Shared {
    using L = Layout<D, CT>;
    Mine<D, CT> mine[L::W];
    uint64_t full[L::W][L::slots];
    int prefix[kMaxBatch + 1];
    uint32_t sums[L::W];
    int failed;
};

__device__ __forceinline__ void ldmatrix_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// The 8 x 8 matrix of which lane 4 i + j holds elements 2 j and 2 j + 1 of row i, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <int N>
__device__ __forceinline__ void ld_words(uint32_t addr, uint32_t (&w)[N]) {
    if constexpr (N == 2)
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
    else
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
}
__device__ __forceinline__ float ld_shared_f(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}
// Byte of 16-byte chunk `chunk` of token `row` of a tile, as the tensor copies lay it down: rows of
// D / 2 bytes, chunks swizzled within spans of as many.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int row, int chunk) {
    constexpr int kChunks = D / 32, kShiftRow = D == 64 ? 2 : D == 128 ? 1 : 0;
    return (uint32_t)(row * (D / 2) + ((chunk ^ ((row >> kShiftRow) & (kChunks - 1))) << 4));
}

template <int D, int CT>
__global__ void __launch_bounds__(32 * warps_of(D, CT), 1)
    kv4_attention_kernel(const __grid_constant__ KvMaps maps, const SplitArgs g) {
    using L = Layout<D, CT>;
    constexpr int W = L::W, T = 32 * W, R = 4 * CT, kSlots = L::slots;
    constexpr int kLaneWords = D / 32;                  // of a key, a lane's
    constexpr int kWords = kLaneWords < 4 ? kLaneWords : 4;  // read at a time
    constexpr int kChunks = D / 32;                     // of a token's codes
    constexpr int kSteps = D / 16;                      // MMAs along the channels
    constexpr bool kHeld = CT * kSteps <= 16;           // queries stay in registers
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    Shared<D, CT>& S = *reinterpret_cast<Shared<D, CT>*>(smem_raw + (base - smem_u32(smem_raw)) + W * kSlots * L::codes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, t = lane & 3;
    const uint32_t ring = base + (uint32_t)(warp * kSlots) * L::codes;
    Mine<D, CT>& mine = S.mine[warp];
    const q4lin_kv4_cache_t& C = g.cache;
    const int Hkv = (int)C.kv_heads, group = (int)(g.a.heads / C.kv_heads), ps = g.page_shift;
    const int tile_shift = 6 - ps, ppt = 1 << tile_shift;  // pages per tile

    if (tid == 0) {
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.v);
        S.prefix[0] = 0;
        S.failed = 0;
        for (int w = 0; w < W; ++w)
            for (int s = 0; s < kSlots; ++s) mbar_init(smem_u32(&S.full[w][s]), 1);
        mbar_init_fence();
    }
    follow_stream();  // (the joining kernel, launched next, waits for this one's end)
    const int batch = (int)C.batch;
    const uint32_t sum = scan_tiles<R, W>(g, S.prefix, S.sums);
    // A list that would be too long is empty, and a share of all numbers tells the joining kernel
    // that no head was cut.
    const bool too_many = sum == kTooMany;
    const int total = too_many ? 0 : (int)sum;
    const int share = max(1, (total + g.workers - 1) / g.workers);
    if (blockIdx.x == 0) {
        for (int b = tid; b < batch; b += T) g.list[1 + b] = too_many ? 0 : S.prefix[b];
        if (tid == 0) g.list[0] = too_many ? INT_MAX : share;
    }
    // Neighbouring shares to different SMs: a short list is spread over all of them.
    const int worker = warp * (int)gridDim.x + (int)blockIdx.x;
    const int64_t begin = (int64_t)worker * share;
    const int end = (int)min((int64_t)total, begin + share);
    if (begin >= end) return;

    // The piece's tiles `first`, first + 1, ...; with the pages of the next 32 / ppt of them in
    // the lanes: lane i holds page i % ppt of tile i / ppt.
    const uint32_t page_bytes = (uint32_t)(D / 2) << ps;
    const int batch_tiles = 32 >> tile_shift, page_of_lane = lane & (ppt - 1), tile_of_lane = lane >> tile_shift;
    const int32_t* table = nullptr;
    int first = 0, cnt = 0, page_low = 0, pages = 0, head = 0, ids = 0, issued = 0, slot_in = 0, in_flight = 0;
    // (-1 is no page and none of the cache's: it is told apart from one in the table by its place.)
    auto load_ids = [&](int i) {
        const int p = ((first + i) << tile_shift) + lane;
        ids = i + tile_of_lane < cnt && p >= page_low && p < pages ? __ldg(table + p) : -1;
    };
    auto check_ids = [&](int i) {
        if ((uint32_t)ids >= (uint32_t)C.num_pages) {
            const int p = ((first + i) << tile_shift) + lane;
            if (i + tile_of_lane < cnt && p >= page_low && p < pages) {
                atomicCAS(g.status, 0, kStatusIndex);
                ids = 0;  // read something of the cache rather than nothing
            }
        }
    };
    // Next half tile of the piece (keys of a tile, then its values) into the ring, a page a lane.
    auto issue = [&]() {
        if (issued >= 2 * cnt) return;
        const int i = issued >> 1, in_batch = i & (batch_tiles - 1);
        if ((issued & 1) == 0 && i > 0 && in_batch == 0) load_ids(i), check_ids(i);
        const int id = __shfl_sync(0xffffffffu, ids, (in_batch << tile_shift) + page_of_lane);
        const bool some = lane < ppt && id >= 0;
        const int count = __popc(__ballot_sync(0xffffffffu, some));
        const uint32_t bar = smem_u32(&S.full[warp][slot_in]);
        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)count * page_bytes + g.missing);
        __syncwarp();
        if (some)
            tma_load_3d(ring + (uint32_t)slot_in * L::codes + page_of_lane * page_bytes, issued & 1 ? &maps.v : &maps.k, 0, 0,
                        id * Hkv + head, bar);
        ++issued, ++in_flight;
        slot_in = slot_in + 1 == kSlots ? 0 : slot_in + 1;
    };
    // Four scales a lane, keys' in the lower half of the warp and values' in the upper one, on their way
    // a tile ahead, their page's index two.
    const int scale_key = (lane & 15) * 4;
    const float* const scale_base = lane < 16 ? C.k_scales : C.v_scales;
    int scale_page = -1;
    float4 scales_next = make_float4(0.f, 0.f, 0.f, 0.f);
    auto fetch_page = [&](int i) {
        const int p = ((first + i) << tile_shift) + (scale_key >> ps);
        scale_page = i < cnt && p >= page_low && p < pages ? __ldg(table + p) : -1;
        if ((uint32_t)scale_page >= (uint32_t)C.num_pages && i < cnt && p >= page_low && p < pages) scale_page = 0;  // (reported)
    };
    auto fetch_scales = [&]() {
        scales_next = make_float4(0.f, 0.f, 0.f, 0.f);
        if (scale_page >= 0)
            scales_next = __ldg(reinterpret_cast<const float4*>(
                scale_base + (((int64_t)scale_page * Hkv + head) << ps) + (scale_key & ((1 << ps) - 1))));
    };
    uint32_t phase = 0;  // parity bit of each slot's next wait
    int slot_out = 0;
    bool ok = true;
    auto await = [&]() {  // the oldest half tile in flight; its slot
        const uint32_t bar = smem_u32(&S.full[warp][slot_out]);
        ok = __all_sync(0xffffffffu, wait_bounded(bar, (phase >> slot_out) & 1u, g.wait_ns, &S.failed));
        const uint32_t at = (uint32_t)slot_out;
        if (ok) {
            phase ^= 1u << slot_out, --in_flight;
            slot_out = slot_out + 1 == kSlots ? 0 : slot_out + 1;
        }
        return at;
    };

    int pos = (int)begin;
    Piece P = piece_of<R>(g, S.prefix, pos, end);
    while (true) {
        // ---- queries: rotated, scaled to fp16's upper range by a power of two, split into two
        // terms.  A lane holds 8 channels of a row, kPer rows at a time.  Their loads and the
        // pages' go first: behind the rings of all SMs they would wait for microseconds.
        cnt = P.len > 0 ? P.n : 0;
        first = P.tile0 + P.k0;
        table = C.page_table + P.b * C.table_stride;
        pages = (P.len + (1 << ps) - 1) >> ps;
        // Pages before the window of the piece's first token are not read.
        page_low = 0;
        if (g.a.window > 0)
            page_low = (int)(max((int64_t)P.len - P.tq + P.row0 / group - g.a.window + 1, (int64_t)0) >> ps);
        head = P.h;
        issued = 0;
        load_ids(0);
        fetch_page(0);
        int limit_min = INT_MAX, low_max = 0;
        {
            constexpr int kUnits = D / 8, kPer = 32 / kUnits, kPasses = R / kPer;
            const int unit = lane % kUnits;
            const int64_t o0 = __ldg(g.a.offsets + P.b);
            bool turned;
            int cl, ch;
            rope_channels(g.a.rope, unit, &turned, &cl, &ch);
            constexpr int kTogether = kPasses < 2 ? kPasses : 2;  // passes whose loads overlap
            const int valid = min(R, P.tq * group - P.row0);  // rows (the others stay unread)
            if (lane >= valid && lane < R) mine.row[lane] = {0.f, -1, 0, -1};
            const uint32_t token0 = (uint32_t)P.row0 / (uint32_t)group, rest0 = P.row0 - token0 * group;
#pragma unroll 1
            for (int p0 = 0; p0 * kPer < valid; p0 += kTogether) {
                float x[kTogether][8], c[kTogether][4], s[kTogether][4];
#pragma unroll
                for (int k = 0; k < kTogether; ++k) {
                    const uint32_t r = (p0 + k) * kPer + lane / kUnits, step = (rest0 + r) / (uint32_t)group;
                    const int token = token0 + step, position = P.len - P.tq + token;
                    if (r < valid) {
                        const int64_t e = (o0 + token) * g.a.q_token_stride +
                                          (P.h * group + (int)(rest0 + r - step * group)) * g.a.q_head_stride;
                        load_four(g.a.query, g.a.dtype, e + cl, g.q_vec, x[k]);
                        load_four(g.a.query, g.a.dtype, e + ch, g.q_vec, x[k] + 4);
                        if (turned && position >= 0) rope_load(g.a.rope, position, unit, c[k], s[k]);
                    }
                }
                if (p0 == 0) {
                    check_ids(0);
                    fetch_scales();
                    fetch_page(1);
#pragma unroll 1
                    for (int i = 0; i < kSlots; ++i) issue();
                }
#pragma unroll
                for (int k = 0; k < kTogether; ++k) {
                    if ((p0 + k) * kPer >= valid) break;
                    const uint32_t r = (p0 + k) * kPer + lane / kUnits, step = (rest0 + r) / (uint32_t)group;
                    const int token = token0 + step, position = P.len - P.tq + token;
                    const bool in = r < valid;
                    if (in && turned && position >= 0) rope_apply(g.a.rope, c[k], s[k], x[k]);
                    float m = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[k][e]));
#pragma unroll
                    for (int o = kUnits / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                    // 2^up brings the row's largest |x| to [2^14, 2^15), with its exponent kept within
                    // what both 2^up and 2^-up can hold; the scale's sign goes with it, so that
                    // larger scores stay larger after the factor.
                    const int ex = min(max((int)(__float_as_uint(m) >> 23), 30), 254) - 127;
                    const float up = copysignf(__uint_as_float((uint32_t)(127 + 14 - ex) << 23), g.a.scale);
                    const float down = __uint_as_float((uint32_t)(127 - 14 + ex) << 23);
                    if (!in) continue;
                    // Channel n of a word of eight is in the lower half of its pair for n < 4, in the
                    // upper one for n >= 4; pair n % 4 of a word is half n % 2 of step n % 4 / 2.
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int d = (e < 4 ? cl : ch) + e % 4, word = d / 8;
                        const float v = x[k][e] * up;
                        const __half hi = __float2half_rn(v), lo = __float2half_rn(v - __half2float(hi));
                        // Columns 2 r and 2 r + 1 of row r: lanes 4 columns apart.
                        __half* f = reinterpret_cast<__half*>(
                            &mine.q[r / 4][2 * (word % kLaneWords) + e % 4 / 2][r % 4 * 8 + word / kLaneWords]);
                        f[e % 2 * 2 + (d >> 2 & 1)] = hi, f[16 + e % 2 * 2 + (d >> 2 & 1)] = lo;
                    }
                    RowInfo i;
                    i.factor = fabsf(g.a.scale) * kLog2e * down;
                    i.limit = g.a.causal ? position : P.len - 1;
                    const int64_t low = g.a.window > 0 ? (int64_t)position - g.a.window + 1 : 0;
                    i.low = low > 0 ? (int)low : 0;
                    i.index = (int)((o0 + token) * g.a.heads + P.h * group + (rest0 + r - step * group));
                    if (unit == 0) mine.row[r] = i;
                    limit_min = min(limit_min, i.limit), low_max = max(low_max, i.low);
                }
            }
            limit_min = __reduce_min_sync(0xffffffffu, limit_min);
            low_max = __reduce_max_sync(0xffffffffu, low_max);
            __syncwarp();
        }

        // Lane (gq, t) has row 4 ct + t of everything.  O: channels 32 c + 4 gq + 2 n, + 1 in [2 c + n].
        float2 O[CT][2 * kChunks];
        float m_run[CT], l_run[CT], factor[CT];
        int limit[CT], low[CT];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            m_run[ct] = -INFINITY, l_run[ct] = 0.f;
            const RowInfo& row = mine.row[4 * ct + t];
            factor[ct] = row.factor, limit[ct] = row.limit, low[ct] = row.low;
#pragma unroll
            for (int i = 0; i < 2 * kChunks; ++i) O[ct][i] = make_float2(0.f, 0.f);
        }
        uint2 held_q[CT][kHeld ? kSteps : 1];
        if constexpr (kHeld) {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int k = 0; k < kSteps; ++k) held_q[ct][k] = mine.q[ct][k][lane];
        }
        for (int i = 0; i < cnt; ++i) {
            const int tile_key = (first + i) * kTile;
            // The tile's scales, through shared memory to the lanes that want them; 0 for keys behind the
            // sequence, whose slots may hold anything.
            {
                const int left = P.len - tile_key - scale_key;
                float4 v = scales_next;
                v.x = left > 0 ? v.x : 0.f, v.y = left > 1 ? v.y : 0.f, v.z = left > 2 ? v.z : 0.f, v.w = left > 3 ? v.w : 0.f;
                const float less = lane < 16 ? 1.f : kLess;
                v.x *= less, v.y *= less, v.z *= less, v.w *= less;
                *reinterpret_cast<float4*>(&mine.scales[lane >> 4][scale_key]) = v;
                fetch_scales();
                fetch_page(i + 2);
                __syncwarp();
            }
            // Of this lane's keys, 16 m + gq and + 8.
            auto scales_of = [&](int kind, float2 (&s)[4]) {
                const uint32_t at = smem_u32(mine.scales[kind]) + gq * 4;
#pragma unroll
                for (int m = 0; m < 4; ++m) s[m] = make_float2(ld_shared_f(at + m * 64), ld_shared_f(at + m * 64 + 32));
            };
            // ---- scores
            const uint32_t k_slot = await();
            if (!ok) break;
            const uint32_t k_at = ring + k_slot * L::codes;
            float sc[CT][4][4];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[ct][m][e] = 0.f;
            // (Steps of the four blocks of 16 keys side by side: a block's own wait for one another.)
#pragma unroll
            for (int c = 0; c < kLaneWords / kWords; ++c) {
                const int byte = t * kLaneWords * 4 + c * kWords * 4;
                uint32_t w[8][kWords];
#pragma unroll
                for (int j = 0; j < 8; ++j) ld_words(k_at + chunk_at<D>(8 * j + gq, byte >> 4) + (byte & 15), w[j]);
#pragma unroll
                for (int k = 0; k < kWords; ++k) {
                    const int step = 2 * (c * kWords + k);
                    uint2 q0[CT], q1[CT];
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) {
                        if constexpr (kHeld)
                            q0[ct] = held_q[ct][step], q1[ct] = held_q[ct][step + 1];
                        else
                            q0[ct] = mine.q[ct][step][lane], q1[ct] = mine.q[ct][step + 1][lane];
                    }
                    uint4 a[4], b[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        nibbles_f16(w[2 * m][k], a[m].x, a[m].z, b[m].x, b[m].z);
                        nibbles_f16(w[2 * m + 1][k], a[m].y, a[m].w, b[m].y, b[m].w);
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) mma_f16(sc[ct][m], a[m], q0[ct].x, q0[ct].y);
                    }
#pragma unroll
                    for (int m = 0; m < 4; ++m)
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) mma_f16(sc[ct][m], b[m], q1[ct].x, q1[ct].y);
                }
            }
            __syncwarp();
            issue();  // the slot of the keys is free

            // ---- softmax: weights by the maximum that there is, as long as they stay in fp16's range; a row
            // that has seen nothing yet or whose scores have grown too far gets a new maximum first.  Then
            // times the values' scales, as two fp16 terms.
            float2 sk[4], sv[4];
            scales_of(0, sk);
            scales_of(1, sv);
            const bool inside = tile_key >= low_max && tile_key + kTile - 1 <= limit_min;
            uint2 pf[CT][4];  // B fragments
            float unit[CT];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                float2 x[4], p[4];
                // (Factors and keys' scales first: a score may be an ordinary one where neither is.)
                const float2 f2 = make_float2(factor[ct], factor[ct]);
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    x[m] = fmul2(make_float2(sc[ct][m][0] + sc[ct][m][1], sc[ct][m][2] + sc[ct][m][3]), fmul2(sk[m], f2));
                if (!inside) {
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const int key = tile_key + 16 * m + gq;
                        if (key < low[ct] || key > limit[ct]) x[m].x = -INFINITY;
                        if (key + 8 < low[ct] || key + 8 > limit[ct]) x[m].y = -INFINITY;
                    }
                }
                auto weights = [&]() {
                    const float off = m_run[ct] == -INFINITY ? 0.f : -m_run[ct];
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        p[m] = fadd2(x[m], make_float2(off, off));
                        p[m].x = ex2(p[m].x), p[m].y = ex2(p[m].y);
                    }
                };
                weights();
                float most = fmaxf(fmaxf(fmaxf(p[0].x, p[0].y), fmaxf(p[1].x, p[1].y)), fmaxf(fmaxf(p[2].x, p[2].y), fmaxf(p[3].x, p[3].y)));
                const bool sees = limit[ct] >= tile_key && low[ct] < tile_key + kTile;
                const unsigned far = __ballot_sync(0xffffffffu, most > kMostWeight || (m_run[ct] == -INFINITY && sees));
                if (far) {  // (each row for itself)
                    float mx = fmaxf(fmaxf(fmaxf(x[0].x, x[0].y), fmaxf(x[1].x, x[1].y)), fmaxf(fmaxf(x[2].x, x[2].y), fmaxf(x[3].x, x[3].y)));
#pragma unroll
                    for (int o = 4; o < 32; o *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    const float old = m_run[ct];
                    if (far & 0x11111111u << t) m_run[ct] = fmaxf(mx, old);
                    const float alpha = m_run[ct] == -INFINITY ? 1.f : ex2(old - m_run[ct]);
                    l_run[ct] *= alpha;
#pragma unroll
                    for (int n = 0; n < 2 * kChunks; ++n) O[ct][n] = fmul2(O[ct][n], make_float2(alpha, alpha));
                    weights();
                }
                float2 sum = make_float2(0.f, 0.f);
                most = 0.f;
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    sum = fadd2(sum, p[m]);
                    p[m] = fmul2(p[m], sv[m]);
                    most = fmaxf(fmaxf(most, fabsf(p[m].x)), fabsf(p[m].y));
                }
                // The largest of the row (a lane's other columns are other rows) to [2^14, 2^15).
#pragma unroll
                for (int o = 4; o < 32; o *= 2) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                const uint32_t ex = min(max(__float_as_uint(most) >> 23, 15u), 254u);
                const float up = __uint_as_float((268u - ex) << 23);
                unit[ct] = __uint_as_float((ex - 14u) << 23);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    p[m] = fmul2(p[m], make_float2(up, up));
                    // Rows of a transposed fragment: both terms of a key's weight.
                    uint32_t hi, lo;
                    split_f16(p[m].x, p[m].y, &hi, &lo);
                    pf[ct][m].x = transposed(prmt(hi, lo, 0x5410u));
                    pf[ct][m].y = transposed(prmt(hi, lo, 0x7632u));
                }
                l_run[ct] += sum.x + sum.y;
            }
            const uint32_t v_slot = await();
            if (!ok) break;

            // ---- outputs: 64 channels at a time, the tile's 64 keys in 4 steps
            const uint32_t v_at = ring + v_slot * L::codes;
#pragma unroll
            for (int c0 = 0; c0 < kChunks; c0 += 2) {
                float acc[CT][4][4];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[ct][n][e] = 0.f;
#pragma unroll
                for (int k2 = 0; k2 < 2; ++k2) {
                    uint32_t w[2][4];  // of keys 32 k2 + 8 i + 2 t, + 1: channels 4 gq .. 4 gq + 3 of the chunk
                    ldmatrix_trans(v_at + chunk_at<D>(32 * k2 + lane, c0), w[0]);
                    ldmatrix_trans(v_at + chunk_at<D>(32 * k2 + lane, c0 + 1), w[1]);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint4 a, b;  // channels 4 gq, + 1; 4 gq + 2, + 3
                            nibbles_f16(w[c][2 * k], a.x, a.y, b.x, b.y);
                            nibbles_f16(w[c][2 * k + 1], a.z, a.w, b.z, b.w);
#pragma unroll
                            for (int ct = 0; ct < CT; ++ct) {
                                mma_f16(acc[ct][2 * c], a, pf[ct][2 * k2 + k].x, pf[ct][2 * k2 + k].y);
                                mma_f16(acc[ct][2 * c + 1], b, pf[ct][2 * k2 + k].x, pf[ct][2 * k2 + k].y);
                            }
                        }
                    }
                }
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const float2 v = make_float2(acc[ct][n][0] + acc[ct][n][1], acc[ct][n][2] + acc[ct][n][3]);
                        O[ct][2 * c0 + n] = ffma2(v, make_float2(unit[ct], unit[ct]), O[ct][2 * c0 + n]);
                    }
            }
            __syncwarp();
            issue();
        }
        if (!ok) {
            // A wait ran out: copies still in flight must land before the CTA leaves, and the
            // warp ends here (outputs are undefined).
            if (lane == 0) record_failure(g.status, &S.failed);
            const int64_t limit = g.missing ? g.wait_ns : kDrainNs;
            for (; in_flight > 0; --in_flight) {
                wait_bounded(smem_u32(&S.full[warp][slot_out]), (phase >> slot_out) & 1u, limit, nullptr);
                phase ^= 1u << slot_out;
                slot_out = slot_out + 1 == kSlots ? 0 : slot_out + 1;
            }
            return;
        }

        // ---- results: this lane has 4 channels of each chunk of rows 4 ct + t
        const bool complete = P.n == P.tiles;
        float* part = part_at<D, R>(g, worker, P.k0 == 0);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            float l = l_run[ct];
#pragma unroll
            for (int o = 4; o < 32; o *= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
            const int r = 4 * ct + t;
            const int64_t index = mine.row[r].index;
            if (index < 0) continue;
            const float f = !complete ? 1.f : l != 0.f ? kMore / l : 0.f;  // l == 0: the row sees no key
            const bool wide = !complete || g.a.dtype == Q4LIN_DTYPE_F32;
            float* to = complete ? static_cast<float*>(g.a.out) + index * D : part + r * D;
            unsigned short* to16 = static_cast<unsigned short*>(g.a.out) + index * D;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const float2 x = fmul2(O[ct][2 * c], make_float2(f, f)), y = fmul2(O[ct][2 * c + 1], make_float2(f, f));
                if (wide)
                    *reinterpret_cast<float4*>(to + 32 * c + 4 * gq) = make_float4(x.x, x.y, y.x, y.y);
                else
                    *reinterpret_cast<uint2*>(to16 + 32 * c + 4 * gq) =
                        make_uint2(to_16x2(x.x, x.y, g.a.dtype), to_16x2(y.x, y.y, g.a.dtype));
            }
            if (gq != 0) continue;
            if (!complete)
                part[R * D + r] = m_run[ct], part[R * D + R + r] = l * kLess;
            else if (g.a.lse)
                g.a.lse[index] = l != 0.f ? ((m_run[ct] == -INFINITY ? 0.f : m_run[ct]) + lg2(l)) * kLn2
                                          : -INFINITY;
        }
        pos += P.n;
        if (pos >= end) return;
        P = piece_of<R>(g, S.prefix, pos, end);
        __syncwarp();  // every lane has read the queries and rows of this piece
    }
}

// A map of the codes: boxes of one page of one head, 16-byte chunks of a token's codes swizzled.
bool map_codes(CUtensorMap* map, const q4lin_kv4_cache_t& C, const uint8_t* codes) {
    EncodeTiledFn encode = tensor_map_encoder();
    if (!encode) return false;
    const cuuint64_t row = (cuuint64_t)C.head_dim / 2;
    const cuuint64_t dims[3] = {row, (cuuint64_t)C.page_size, (cuuint64_t)(C.num_pages * C.kv_heads)};
    const cuuint64_t strides[2] = {row, row * (cuuint64_t)C.page_size};
    const cuuint32_t box[3] = {(cuuint32_t)row, (cuuint32_t)C.page_size, 1}, steps[3] = {1, 1, 1};
    const CUtensorMapSwizzle swizzle = row == 32   ? CU_TENSOR_MAP_SWIZZLE_32B
                                       : row == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                   : CU_TENSOR_MAP_SWIZZLE_128B;
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(codes), dims, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int CT>
cudaError_t launch(SplitArgs& g, const SplitSize& size, const KvMaps& maps, const LaunchCtx& c) {
    using L = Layout<D, CT>;
    constexpr int R = 4 * CT;
    constexpr int bytes = L::W * L::slots * (int)L::codes + (int)sizeof(Shared<D, CT>) + 1024;
    static_assert(bytes <= 227 * 1024, "shared memory of one SM");
    cudaError_t e = kernel_smem_once<kv4_attention_kernel<D, CT>>(bytes);
    if (e != cudaSuccess) return e;
    // One CTA per SM, and no more than the longest possible list has tiles for.
    const int64_t grid = std::min<int64_t>(c.sm_count, size.segments * size.tiles);
    g.workers = (int)grid * L::W;
    g.list = reinterpret_cast<int*>(c.ws);
    g.parts = c.ws + kMaxBatch + 4;  // 16-byte aligned
    if ((int64_t)g.workers * 2 * R * (D + 2) + kMaxBatch + 4 > c.ws_floats) return cudaErrorInvalidValue;
    e = launch_early(kv4_attention_kernel<D, CT>, dim3((unsigned)grid), 32 * L::W, bytes, c.stream, maps, g);
    if (e != cudaSuccess) return e;
    return join_launch<D, R>(g, size, c);
}

}  // namespace

bool kv4_attention_split_countable(const q4lin_kv4_cache_t& cache, const q4lin_attention_t& a, int64_t rows_max) {
    return split_countable(cache, a, rows_max, 4);
}

cudaError_t kv4_attention_split_launch(const q4lin_kv4_cache_t& cache, const q4lin_attention_t& a, int64_t rows_max,
                                       const LaunchCtx& c) {
    KvMaps maps;
    if (!map_codes(&maps.k, cache, cache.k_codes) || !map_codes(&maps.v, cache, cache.v_codes))
        return cudaErrorInvalidValue;
    return in_groups(cache, a, rows_max, 4, c, [&](SplitArgs& g, const SplitSize& size) {
        g.unshift = kMore;
        auto rows = [&](auto dim) {
            constexpr int D = decltype(dim)::value;
            if constexpr (D < 256)
                if (size.rows > 8) return launch<D, 4>(g, size, maps, c);
            return size.rows > 4 ? launch<D, 2>(g, size, maps, c) : launch<D, 1>(g, size, maps, c);
        };
        if (cache.head_dim == 64) return rows(std::integral_constant<int, 64>{});
        if (cache.head_dim == 128) return rows(std::integral_constant<int, 128>{});
        return rows(std::integral_constant<int, 256>{});
    });
}

}  // namespace q4lin
