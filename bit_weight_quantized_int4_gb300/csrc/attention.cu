// attention.cu -- attention of a few query rows per key/value head over the paged 8-bit
// cache: single tokens, draft tokens, short chunks.
//
// Bound: the codes, 2 head_dim bytes per key and key/value head, read once for up to 16 query
// rows of that head (8 with 256 channels; more rows walk over them again, from L2).  The keys of all sequences and heads form one list of 64-key tiles that
// is cut evenly over all warps of the GPU, whatever the sequences' lengths; a warp's share of
// one head's keys is a piece.  A warp works alone: it has its own ring of bulk copies (a
// page's keys or values of one head are contiguous), its own queries, running maximum, sum
// and outputs, and a piece's first copies are on their way while its queries are rotated.
// (CTAs that joined their warps after every piece spent 5 to 8 us on each: the latencies of
// a loaded memory system, one after another, with nothing in flight.)  Heads that lie in one
// share are stored at once; the others leave sums in the handle's workspace, which a second
// kernel adds in the order of the keys, so the result does not depend on the schedule.
//
// Measured (8 key/value heads of 128, 4 query heads each): 64 sequences of up to 8192 tokens,
// 652 MB, 110 to 114 us: 5.8 TB/s, 0.86 of a copy's bandwidth; one sequence of 131071 tokens, 269
// MB, 56 us: 4.8 TB/s, the start and the join a sixth of it.  One of 701 tokens (0.7 MB) 8.9 us,
// 9 drafts of up to 5 tokens behind a window of 1024 (10 MB, 7 query heads) 22.0 us: the chain of
// dependent loads, from the offsets to the page table to the first keys, and two launches.
//
// Products on the tensor cores (m16n8k16, fp16 operands, fp32 sums): codes - 128 are exact
// in fp16; a query row and a row of probabilities take two of the MMA's 16 rows each, the
// rounded value and what the rounding left (22 bits), so 8 rows fill a tile at no cost over
// one-term operands.  Both operands' summed axes are permuted so that a lane reads 16
// consecutive bytes of a key (of a channel of the values) at a time and the scores leave
// the first product in the layout that the second one takes.
#include "attention_split.cuh"

namespace q4lin {
namespace {
using namespace ptx;
using namespace serving;

constexpr int kRows = 8;   // query rows per MMA tile (two of its 16 rows each)
constexpr int kSlots = 3;  // half tiles (keys or values) in a warp's ring

// Warps of the one CTA on an SM: what registers, rings and queries leave room for.
__host__ __device__ constexpr int warps_of(int D, int RT) {
    return D == 256 ? 4 : D == 64 ? (RT == 1 ? 12 : 8) : (RT == 1 ? 8 : 7);
}

template <int D, int RT>
struct Mine {  // of one warp
    uint4 q[RT][D / 16][32];  // A fragments
    RowInfo row[RT * kRows];
};
template <int D, int RT>
struct Shared {
    static constexpr int W = warps_of(D, RT);
    Mine<D, RT> mine[W];
    uint64_t full[W][kSlots];
    int prefix[kMaxBatch + 1];
    uint32_t sums[W];
    int failed;
};

template <int D, int RT>
__global__ void __launch_bounds__(32 * warps_of(D, RT), 1) attention_split_kernel(const SplitArgs g) {
    constexpr int W = warps_of(D, RT), T = 32 * W, R = RT * kRows, kNt = D / 8;
    constexpr uint32_t kHalf = kTile * D;  // bytes of a tile's keys (values)
    extern __shared__ __align__(128) uint8_t smem_raw[];
    // After the rings, in dynamic shared memory too (more than 48 KiB with two row tiles).
    Shared<D, RT>& S = *reinterpret_cast<Shared<D, RT>*>(smem_raw + W * kSlots * kHalf);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_u32(smem_raw) + (uint32_t)(warp * kSlots) * kHalf;
    Mine<D, RT>& mine = S.mine[warp];
    const q4lin_kv_cache_t& C = g.cache;
    const int Hkv = (int)C.kv_heads, group = (int)(g.a.heads / C.kv_heads), ps = g.page_shift;
    const int ppt = kTile >> ps;  // pages per tile
    griddep_launch_dependents();  // (the joining kernel waits for this one's end)

    // ---- the list: an inclusive scan of the sequences' tiles
    if (tid == 0) {
        S.prefix[0] = 0;
        S.failed = 0;
        for (int w = 0; w < W; ++w)
            for (int s = 0; s < kSlots; ++s) mbar_init(smem_u32(&S.full[w][s]), 1);
        mbar_init_fence();
    }
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

    auto piece_at = [&](int pos) { return piece_of<R>(g, S.prefix, pos, end); };

    // The piece's tiles `first`, first + 1, ...; with the pages of the next 32 / ppt of them in
    // the lanes: lane i holds page i % ppt of tile i / ppt.
    const uint32_t page_bytes = (uint32_t)(D << ps);
    const int batch_tiles = 32 / ppt;
    const int32_t* table = nullptr;
    int first = 0, cnt = 0, page_low = 0, pages = 0, head = 0, ids = 0, issued = 0, slot_in = 0, in_flight = 0;
    // (-1 is no page and none of the cache's: it is told apart from one in the table by its place.)
    auto load_ids = [&](int i) {
        const int p = (first + i) * ppt + lane;
        ids = i + lane / ppt < cnt && p >= page_low && p < pages ? __ldg(table + p) : -1;
    };
    auto check_ids = [&](int i) {
        if ((uint32_t)ids >= (uint32_t)C.num_pages) {
            const int p = (first + i) * ppt + lane;
            if (i + lane / ppt < cnt && p >= page_low && p < pages) {
                atomicCAS(g.status, 0, kStatusIndex);
                ids = 0;  // read something of the cache rather than nothing
            }
        }
    };
    // Next half tile of the piece (keys of a tile, then its values) into the ring.
    auto issue = [&]() {
        if (issued >= 2 * cnt) return;
        const int i = issued >> 1;
        if ((issued & 1) == 0 && i > 0 && i % batch_tiles == 0) load_ids(i), check_ids(i);
        const int id = __shfl_sync(0xffffffffu, ids, (i % batch_tiles) * ppt + lane % ppt);
        const bool some = lane < ppt && id >= 0;
        const int count = __popc(__ballot_sync(0xffffffffu, some));
        const uint32_t bar = smem_u32(&S.full[warp][slot_in]);
        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)count * page_bytes + g.missing);
        __syncwarp();
        if (some) {
            const uint8_t* codes = issued & 1 ? C.v_codes : C.k_codes;
            bulk_load(ring + (uint32_t)slot_in * kHalf + lane * page_bytes,
                      codes + ((int64_t)id * Hkv + head) * page_bytes, page_bytes, bar);
        }
        ++issued, ++in_flight;
        slot_in = slot_in + 1 == kSlots ? 0 : slot_in + 1;
    };
    // The scales of this lane's 16 keys of tile i (one page each).
    float sk_next = 0.f, sv_next = 0.f;
    auto fetch_scales = [&](int i) {
        const int p = (first + i) * ppt + ((t * 16) >> ps);
        sk_next = sv_next = 0.f;
        if (i < cnt && p >= page_low && p < pages) {
            int id = __ldg(table + p);
            if (id < 0 || id >= C.num_pages) id = 0;
            sk_next = __ldg(C.k_scales + (int64_t)id * Hkv + head);
            sv_next = __ldg(C.v_scales + (int64_t)id * Hkv + head);
        }
    };
    uint32_t phase = 0;  // parity bit of each slot's next wait
    int slot_out = 0;
    bool ok = true;
    auto await = [&]() {  // the oldest half tile in flight; its place in the ring
        const uint32_t bar = smem_u32(&S.full[warp][slot_out]);
        ok = __all_sync(0xffffffffu, wait_bounded(bar, (phase >> slot_out) & 1u, g.wait_ns, &S.failed));
        const uint32_t at = ring + (uint32_t)slot_out * kHalf;
        if (ok) {
            phase ^= 1u << slot_out, --in_flight;
            slot_out = slot_out + 1 == kSlots ? 0 : slot_out + 1;
        }
        return at;
    };

    int pos = (int)begin;
    Piece P = piece_at(pos);
    while (true) {
        // ---- queries: rotated, scaled to fp16's upper range by a power of two, split into two
        // terms.  A lane holds 8 channels of a row, kPer rows at a time.  Their loads, the pages'
        // and the scales' go first: behind the rings of all SMs (29 MB) they would wait for 4 us.
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
        int limit_min = INT_MAX, low_max = 0;
        {
            constexpr int kUnits = D / 8, kPer = 32 / kUnits, kPasses = R / kPer;
            const int unit = lane % kUnits;
            const int64_t o0 = __ldg(g.a.offsets + P.b);
            bool turned;
            int cl, ch;
            rope_channels(g.a.rope, unit, &turned, &cl, &ch);
            // Passes whose loads overlap (with four, 128 channels spill in the kernel of 8 rows: 113
            // against 110 us for 64 sequences; drafts 22.5 against 21.8, where 16 rows spill 108 bytes
            // all the same, as 56 do with 256 channels).
            constexpr int kTogether = kPasses < 2 ? kPasses : 2;
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
                    fetch_scales(0);
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
                    // 2^up brings the row's largest |x| to [2^14, 2^15); its exponent is kept
                    // within what both 2^up and 2^-up can hold.
                    const int ex = min(max((int)(__float_as_uint(m) >> 23), 30), 254) - 127;
                    const float up = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
                    const float down = __uint_as_float((uint32_t)(127 - 14 + ex) << 23);
                    if (!in) continue;
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const int d = w ? ch : cl;  // channels d .. d + 3
                        uint4 f;
                        split_f16(x[k][4 * w] * up, x[k][4 * w + 1] * up, &f.x, &f.y);
                        split_f16(x[k][4 * w + 2] * up, x[k][4 * w + 3] * up, &f.z, &f.w);
                        mine.q[r / kRows][(d / 64) * 4 + (d % 16) / 4][(r % kRows) * 4 + (d % 64) / 16] = f;
                    }
                    RowInfo i;
                    i.factor = g.a.scale * kLog2e * down;
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

        float O[RT][kNt][2], m_run[RT], l_run[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            m_run[rt] = -INFINITY, l_run[rt] = 0.f;
#pragma unroll
            for (int i = 0; i < kNt; ++i) O[rt][i][0] = O[rt][i][1] = 0.f;
        }
        const RowInfo* rows = mine.row;
        for (int i = 0; i < cnt; ++i) {
            const float sk = sk_next, sv = sv_next;
            fetch_scales(i + 1);
            const int tile_key = (first + i) * kTile;
            const int key0 = tile_key + t * 16;  // first of this lane's 16 keys
            // ---- scores: 8 column tiles of 8 keys; key of column c of tile j:
            // (c / 2) 16 + 2 j + c % 2, so that this lane's are key0 .. key0 + 15
            const uint32_t k_at = await();
            if (!ok) break;
            float sc[RT][8][4];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[rt][j][e] = 0.f;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                uint4 qf[RT][4];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int k = 0; k < 4; ++k) qf[rt][k] = mine.q[rt][4 * c + k][lane];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int key = (gq >> 1) * 16 + 2 * j + (gq & 1);
                    const uint4 w = ld_shared_v4(k_at + (uint32_t)(key * D + c * 64 + t * 16));
                    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t b0, b1;
                        codes_f16(words[k], &b0, &b1);
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) mma_f16(sc[rt][j], qf[rt][k], b0, b1);
                    }
                }
            }
            __syncwarp();
            issue();  // the slot of the keys is free

            // ---- softmax: running maximum and sum; weights of the values, two fp16 terms
            float sv_max = sv;
            if (ppt > 1) {
                sv_max = fmaxf(sv_max, __shfl_xor_sync(0xffffffffu, sv_max, 1));
                sv_max = fmaxf(sv_max, __shfl_xor_sync(0xffffffffu, sv_max, 2));
            }
            const float ratio = ppt > 1 ? (sv_max > 0.f ? __fdividef(sv, sv_max) : 0.f) : 1.f;
            const bool inside = tile_key >= low_max && tile_key + kTile - 1 <= limit_min;
            uint4 pf[RT][4];
            float alpha[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const RowInfo& row = rows[rt * kRows + gq];
                const float f = row.factor * sk;
                float p[8][2], mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) p[j][e] = (sc[rt][j][e] + sc[rt][j][2 + e]) * f;
                if (!inside) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int key = key0 + 2 * j + e;
                            if (key < row.low || key > row.limit) p[j][e] = -INFINITY;
                        }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fmaxf(p[j][0], p[j][1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                mx = fmaxf(mx, m_run[rt]);
                const float base = mx == -INFINITY ? 0.f : mx;  // a row that has seen nothing yet
                alpha[rt] = ex2(m_run[rt] - base);
                m_run[rt] = mx;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        p[j][e] = ex2(p[j][e] - base + kShift);
                        sum += p[j][e];
                        p[j][e] *= ratio;
                    }
                l_run[rt] = fmaf(l_run[rt], alpha[rt], sum);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    split_f16(p[2 * k][0], p[2 * k][1], &pf[rt][k].x, &pf[rt][k].y);
                    split_f16(p[2 * k + 1][0], p[2 * k + 1][1], &pf[rt][k].z, &pf[rt][k].w);
                }
            }

            // ---- outputs: channel tile nt of 8, the tile's 64 keys in 4 steps
            const uint32_t v_at = await() + (uint32_t)((((t * 16) >> ps) * (D << ps)) +
                                                       ((t * 16) & ((1 << ps) - 1)) + (gq << ps));
            if (!ok) break;
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) {
                const uint4 w = ld_shared_v4(v_at + (uint32_t)((nt * 8) << ps));
                const uint32_t words[4] = {w.x, w.y, w.z, w.w};
                float acc[RT][4];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[rt][e] = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t b0, b1;
                    codes_f16(words[k], &b0, &b1);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) mma_f16(acc[rt], pf[rt][k], b0, b1);
                }
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        O[rt][nt][e] = fmaf(acc[rt][e] + acc[rt][2 + e], sv_max, O[rt][nt][e] * alpha[rt]);
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

        // ---- results: lane (gq, t) holds channels 8 nt + 2 t, + 1 of rows rt 8 + gq
        const bool whole = P.n == P.tiles;
        float* part = part_at<D, R>(g, worker, P.k0 == 0);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            float l = l_run[rt];
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            const int r = rt * kRows + gq;
            const int64_t index = rows[r].index;
            if (index < 0) continue;
            if (!whole) {
#pragma unroll
                for (int nt = 0; nt < kNt; ++nt)
                    *reinterpret_cast<float2*>(part + r * D + nt * 8 + 2 * t) =
                        make_float2(O[rt][nt][0], O[rt][nt][1]);
                if (t == 0) part[R * D + r] = m_run[rt], part[R * D + R + r] = l;
                continue;
            }
            const float inv = l != 0.f ? 1.f / l : 0.f;  // l == 0: the row sees no key
            if (g.a.dtype == Q4LIN_DTYPE_F32) {
                float* out = static_cast<float*>(g.a.out) + index * D + 2 * t;
#pragma unroll
                for (int nt = 0; nt < kNt; ++nt)
                    *reinterpret_cast<float2*>(out + nt * 8) = make_float2(O[rt][nt][0] * inv, O[rt][nt][1] * inv);
            } else {
                unsigned short* out = static_cast<unsigned short*>(g.a.out) + index * D + 2 * t;
#pragma unroll
                for (int nt = 0; nt < kNt; ++nt)
                    *reinterpret_cast<uint32_t*>(out + nt * 8) =
                        to_16x2(O[rt][nt][0] * inv, O[rt][nt][1] * inv, g.a.dtype);
            }
            if (t == 0 && g.a.lse)
                g.a.lse[index] = l != 0.f ? ((m_run[rt] == -INFINITY ? 0.f : m_run[rt]) + lg2(l * kUnshift)) * kLn2
                                          : -INFINITY;
        }
        pos += P.n;
        if (pos >= end) return;
        P = piece_at(pos);
        __syncwarp();  // every lane has read the queries and rows of this piece
    }
}

template <int D, int RT>
cudaError_t launch(SplitArgs& g, const SplitSize& size, const LaunchCtx& c) {
    constexpr int W = warps_of(D, RT), R = RT * kRows;
    constexpr int bytes = W * kSlots * kTile * D + (int)sizeof(Shared<D, RT>);
    static_assert(bytes <= 227 * 1024, "shared memory of one SM");
    cudaError_t e = kernel_smem_once<attention_split_kernel<D, RT>>(bytes);
    if (e != cudaSuccess) return e;
    // One CTA per SM, and no more than the longest possible list has tiles for.
    const int64_t grid = std::min<int64_t>(c.sm_count, size.segments * size.tiles);
    g.workers = (int)grid * W;
    g.list = reinterpret_cast<int*>(c.ws);
    g.parts = c.ws + kMaxBatch + 4;  // 16-byte aligned
    if ((int64_t)g.workers * 2 * R * (D + 2) + kMaxBatch + 4 > c.ws_floats) return cudaErrorInvalidValue;
    attention_split_kernel<D, RT><<<(unsigned)grid, 32 * W, bytes, c.stream>>>(g);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return join_launch<D, R>(g, size, c);
}

}  // namespace

bool attention_split_countable(const q4lin_kv_cache_t& cache, const q4lin_attention_t& a, int64_t rows_max) {
    return split_countable(cache, a, rows_max, kRows);
}

cudaError_t attention_split_launch(const q4lin_kv_cache_t& cache, const q4lin_attention_t& a,
                                   int64_t rows_max, const LaunchCtx& c) {
    return in_groups(cache, a, rows_max, kRows, c, [&](SplitArgs& g, const SplitSize& size) {
        switch (cache.head_dim) {
            case 64: return size.rows > kRows ? launch<64, 2>(g, size, c) : launch<64, 1>(g, size, c);
            case 128: return size.rows > kRows ? launch<128, 2>(g, size, c) : launch<128, 1>(g, size, c);
            default: return launch<256, 1>(g, size, c);
        }
    });
}

}  // namespace q4lin
