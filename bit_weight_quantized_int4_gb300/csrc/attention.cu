// attention.cu -- attention of a few query rows per key/value head over the paged 8-bit
// cache: single tokens, draft tokens, short chunks.
//
// Bound: the codes, 2 head_dim bytes per key and key/value head, read once for all query
// rows of that head.  The keys of all sequences and heads form one list of 64-key tiles that
// is cut evenly over the CTAs, whatever the sequences' lengths; a CTA's share of one
// sequence's keys, for `heads_per` of its key/value heads, is a piece.  The warps of a head
// take its tiles in turn, each with its own ring of bulk copies (a page's keys or values of
// one head are contiguous), its own running maximum and sum and its own outputs; they are
// joined through shared memory at the end of the piece, while the next piece's first copies
// and queries are on their way.  A head that is cut joins its pieces through the handle's
// workspace: every CTA has at most two unfinished pieces (its first and its last), the CTA
// that arrives last adds them in order, so the result does not depend on the schedule.
// Short lists are not cut at all where the join would cost more than it saves.
//
// Products on the tensor cores (m16n8k16, fp16 operands, fp32 sums): codes - 128 are exact
// in fp16; a query row and a row of probabilities take two of the MMA's 16 rows each, the
// rounded value and what the rounding left (22 bits), so 8 rows fill a tile at no cost over
// one-term operands.  Both operands' summed axes are permuted so that a lane reads 16
// consecutive bytes of a key (of a channel of the values) at a time and the scores leave
// the first product in the layout that the second one takes.
#include <algorithm>

#include "q4lin_internal.h"
#include "serving.cuh"

namespace q4lin {
namespace {
using namespace ptx;
using namespace serving;

constexpr int kTile = 64;        // keys per tile
constexpr int kRows = 8;         // query rows per MMA tile (two of its 16 rows each)
constexpr int kSlots = 3;        // half tiles (keys or values) in a warp's ring
constexpr int kMaxBatch = 1024;  // sequences per launch
constexpr float kShift = 14.f;   // probabilities are kept as 2^14 p: fp16's range downwards
constexpr int64_t kDrainNs = 4000000000LL;

// CTAs of four warps, as many per SM as their rings and registers allow: while one joins its
// warps or waits for its first keys, the others stream.
constexpr int kWarps = 4;
__host__ __device__ constexpr int ctas_of(int D, int RT) { return D == 256 ? 1 : D == 64 && RT == 1 ? 3 : 2; }

struct SplitArgs {
    q4lin_kv_cache_t cache;
    q4lin_attention_t a;
    int page_shift;
    int64_t rows_max;
    int q_vec;
    int heads_per;  // key/value heads of a CTA at a time: 1, 2 or 4 (RT * heads_per <= 4)
    float* ws;
    int* tickets;
    int* status;
    int64_t wait_ns;
};

// Per query row of a piece.
struct RowInfo {
    float factor;        // of the MMA's scores, without the keys' scale, in powers of two
    int limit, low;      // keys [low, limit] are seen
    int64_t index;       // token * heads + head, or -1
};

// Largest heads_per * RT: what the queries' fragments leave of the shared memory.
__host__ __device__ constexpr int max_group(int D) { return D == 64 ? 4 : 2; }

enum { kCut, kParts, kWhole };  // how the list is shared, see the kernel

struct List {
    int mode, share, tiles, grid, groups, end;  // end: of this CTA's share
};

// A CTA's share of one sequence's keys.
struct Piece {
    int b, len, tq, h0, row0, tile, n;  // n tiles from `tile`; first head, first row
    int after, more;                    // list position past the piece; whether the CTA goes on
    int cut, later, c0, c1;             // not a head's only piece; not its first; its CTAs
    int64_t o0;
};

template <int D, int RT>
struct Shared {
    static constexpr int W = kWarps, kGroup = max_group(D);
    uint4 q[kGroup][D / 16][32];  // A fragments, [head * RT + row tile]
    RowInfo row[2][kGroup * kRows];  // of this piece and the next
    float m[W][RT * kRows], l[W][RT * kRows];
    uint32_t merge[W];  // where a warp left its outputs
    uint64_t full[W][kSlots];
    List list;
    Piece piece[3];  // this one, the next, and the one after that in the making
    int prefix[kMaxBatch + 1];
    int sums[3][W], scan[2][W];
    int limit_min[2][kGroup], low_max[2][kGroup];  // per head of a piece
    int failed, last;
};

struct Sequence {
    int tq, len, tile0, tiles, row_tiles;
};

// What one sequence asks of this kernel; nothing where its indices are bad or its rows are
// too many for it.
template <int RT>
__device__ __forceinline__ Sequence sequence_of(const SplitArgs& g, int64_t b, bool* bad) {
    Sequence s;
    const int64_t o0 = __ldg(g.a.offsets + b), o1 = __ldg(g.a.offsets + b + 1);
    const int64_t group = g.a.heads / g.cache.kv_heads;
    s.len = __ldg(g.a.lengths + b);
    s.tq = (int)(o1 - o0);
    *bad = o0 < 0 || o1 < o0 || o1 > g.a.tokens || s.tq > g.a.max_query ||
           (int64_t)s.len > g.cache.pages_per_sequence << g.page_shift ||
           (g.a.rope.cos && s.len > g.a.rope.positions);
    if (*bad || s.tq * group > g.rows_max) s.tq = 0;
    if (s.len < 0) s.len = 0;
    const int64_t first = g.a.window > 0 ? (int64_t)s.len - s.tq - g.a.window + 1 : 0;
    s.tile0 = first > 0 ? (int)(first / kTile) : 0;
    s.tiles = max((s.len + kTile - 1) / kTile - s.tile0, 1);
    s.row_tiles = (int)((s.tq * group + RT * kRows - 1) / (RT * kRows));
    return s;
}

// A head's parts, one per CTA, in proportion to its tiles.
__device__ __forceinline__ int parts_of(int tiles, int grid, int all) {
    return max(1, (int)((int64_t)tiles * grid / max(all, 1)));
}
// Units of one head in the list.
__device__ __forceinline__ int units_of(const List& list, const Sequence& s) {
    return list.mode == kCut ? s.tiles : list.mode == kParts ? parts_of(s.tiles, list.grid, list.tiles) : 1;
}
// What a CTA does from list position pos on, in sequence b that begins at list_begin (one thread).
template <int RT>
__device__ __noinline__ void fill_piece(const SplitArgs& g, const List& list, int pos, int b, int list_begin,
                                        const Sequence& s, Piece& p) {
    p.b = b, p.len = s.len, p.tq = s.tq;
    const int of_head = units_of(list, s), local = pos - list_begin, seg = local / of_head;
    const int unit = local - seg * of_head, done = min(of_head - unit, list.end - pos);
    p.h0 = seg / s.row_tiles * g.heads_per, p.row0 = seg % s.row_tiles * (RT * kRows);
    p.after = pos + done;
    p.more = p.after < list.end;
    p.cut = done < of_head;
    int k0 = 0;
    p.n = s.tiles;
    if (list.mode == kCut) {
        k0 = unit, p.n = done;
    } else if (list.mode == kParts) {
        const int each = (s.tiles + of_head - 1) / of_head;
        k0 = unit * each, p.n = max(0, min(each, s.tiles - k0));
    }
    p.tile = s.tile0 + k0;
    p.later = unit > 0;
    p.c0 = (pos - unit) / list.share, p.c1 = (pos - unit + of_head - 1) / list.share;
    p.o0 = __ldg(g.a.offsets + b);
}
template <int RT>
__device__ __noinline__ void make_piece(const SplitArgs& g, const List& list, const int* prefix, int pos, Piece& p) {
    int lo = 0, hi = (int)g.cache.batch;  // prefix[lo] <= pos < prefix[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= pos)
            lo = mid;
        else
            hi = mid;
    }
    bool bad;
    fill_piece<RT>(g, list, pos, lo, prefix[lo], sequence_of<RT>(g, lo, &bad), p);
}

// Four channels of a query row: the joined sums o and l, both as 2^kShift p, over the maximum
// `base` (a power of two's exponent).
__device__ __forceinline__ void emit(const SplitArgs& g, int64_t index, int D, int d, float4 o, float l,
                                     float base) {
    if (index < 0) return;
    const float inv = l != 0.f ? 1.f / l : 0.f;  // l == 0: the row sees no key
    const float v[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
    if (g.a.dtype == Q4LIN_DTYPE_F32)
        *reinterpret_cast<float4*>(static_cast<float*>(g.a.out) + index * D + d) =
            make_float4(v[0], v[1], v[2], v[3]);
    else
        *reinterpret_cast<uint2*>(static_cast<unsigned short*>(g.a.out) + index * D + d) =
            make_uint2(to_16x2(v[0], v[1], g.a.dtype), to_16x2(v[2], v[3], g.a.dtype));
    if (d == 0 && g.a.lse) g.a.lse[index] = l != 0.f ? (base + lg2(l) - kShift) * kLn2 : -INFINITY;
}

// A CTA's unfinished piece of one head: [R][D] sums, then R maxima and R sums of weights.
template <int D, int RT>
__device__ __forceinline__ float* part_at(const SplitArgs& g, int cta, int place, int hi) {
    constexpr int kPart = RT * kRows * (D + 2);
    return g.ws + ((int64_t)(cta * 2 + place) * g.heads_per + hi) * kPart;
}

// The parts of a piece's heads, added in their order by one CTA: four channels of a row per
// thread, kAhead loads in flight (what another SM has just written takes a microsecond or two
// to come).  Not in line: its registers are not the main loop's.
template <int D, int RT, int W>
__device__ __noinline__ void join_parts(const SplitArgs& g, const Piece& P, const RowInfo* rows) {
    constexpr int R = RT * kRows, T = 32 * W, kAhead = 16;
    const int group = (int)(g.a.heads / g.cache.kv_heads);
    const int valid = min(R, P.tq * group - P.row0), count = P.c1 - P.c0 + 1;
    for (int i = threadIdx.x; i < g.heads_per * valid * (D / 4); i += T) {
        const int row = i / (D / 4), d = i % (D / 4) * 4, hi = row / valid, r = row - hi * valid;
        float mx = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < count; c += kAhead) {
            float pm[kAhead], pl[kAhead];
            float4 po[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                pm[k] = -INFINITY, pl[k] = 0.f, po[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c + k < count) {
                    const float* src = part_at<D, RT>(g, P.c0 + c + k, c + k == 0, hi);
                    pm[k] = __ldcg(src + R * D + r), pl[k] = __ldcg(src + R * D + R + r);
                    po[k] = __ldcg(reinterpret_cast<const float4*>(src + r * D + d));
                }
            }
            float top = mx;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) top = fmaxf(top, pm[k]);
            const float from = top == -INFINITY ? 0.f : top, old = ex2(mx - from);
            o.x *= old, o.y *= old, o.z *= old, o.w *= old, l *= old;
            mx = top;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const float w = ex2(pm[k] - from);
                o.x = fmaf(po[k].x, w, o.x), o.y = fmaf(po[k].y, w, o.y);
                o.z = fmaf(po[k].z, w, o.z), o.w = fmaf(po[k].w, w, o.w);
                l = fmaf(pl[k], w, l);
            }
        }
        emit(g, rows[hi * R + r].index, D, d, o, l, mx == -INFINITY ? 0.f : mx);
    }
}

template <int D, int RT>
__global__ void __launch_bounds__(32 * kWarps, ctas_of(D, RT)) attention_split_kernel(const SplitArgs g) {
    constexpr int W = kWarps, T = 32 * W, R = RT * kRows, kGroup = max_group(D);
    constexpr int kNt = D / 8;
    constexpr uint32_t kHalf = kTile * D;  // bytes of a tile's keys (values)
    extern __shared__ uint8_t smem_raw[];
    __shared__ Shared<D, RT> S;
    const uint32_t ring = (smem_u32(smem_raw) + 127u) & ~127u;
    uint8_t* ring_ptr = smem_raw + (ring - smem_u32(smem_raw));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, t = lane & 3;
    const q4lin_kv_cache_t& C = g.cache;
    const int Hkv = (int)C.kv_heads, group = (int)(g.a.heads / C.kv_heads), ps = g.page_shift;
    const int ppt = kTile >> ps;  // pages per tile
    const int hp = g.heads_per, wph = W / hp;  // warps per head
    const int my_head = warp / wph, my_turn = warp % wph;

    // ---- the list: tiles of all sequences, row tiles and groups of heads, or their number
    // alone where nothing is cut.  First the totals, then an inclusive scan.
    if (tid == 0) {
        S.prefix[0] = 0;
        S.failed = 0;
        for (int w = 0; w < W; ++w)
            for (int s = 0; s < kSlots; ++s) mbar_init(smem_u32(&S.full[w][s]), 1);
        mbar_init_fence();
    }
    const int batch = (int)C.batch, groups = Hkv / hp;
    int tiles_all = 0, segments = 0, longest = 0;
    Sequence mine = {};  // of the thread's last sequence: its only one in most calls
    for (int b = tid; b < batch; b += T) {
        bool bad;
        mine = sequence_of<RT>(g, b, &bad);
        tiles_all += mine.tiles * mine.row_tiles * groups, segments += mine.row_tiles * groups;
        if (mine.row_tiles) longest = max(longest, mine.tiles);
        if (bad && blockIdx.x == 0) atomicCAS(g.status, 0, kStatusIndex);
    }
    const bool once = batch <= T;
    {
        const int a = __reduce_add_sync(0xffffffffu, tiles_all), b = __reduce_add_sync(0xffffffffu, segments);
        const int c = __reduce_max_sync(0xffffffffu, longest);
        if (lane == 0) S.sums[0][warp] = a, S.sums[1][warp] = b, S.sums[2][warp] = c;
    }
    __syncthreads();
    tiles_all = segments = longest = 0;
#pragma unroll
    for (int w = 0; w < W; ++w)
        tiles_all += S.sums[0][w], segments += S.sums[1][w], longest = max(longest, S.sums[2][w]);
    // Three ways to share the list, by the rounds that the warps of a CTA then take over its
    // tiles.  Cut: evenly, wherever that falls; a piece more and a join cost about three rounds.
    // Parts: every head in parts of its own, one per CTA; a join costs about two.  Whole: some
    // heads to their end.
    const int grid = (int)gridDim.x;
    int parts = 0, part_tiles = 0;
    for (int b = tid; b < batch; b += T) {
        bool bad;
        if (!once) mine = sequence_of<RT>(g, b, &bad);
        if (!mine.row_tiles) continue;
        const int n = parts_of(mine.tiles, grid, tiles_all);
        parts += n * mine.row_tiles * groups;
        part_tiles = max(part_tiles, (mine.tiles + n - 1) / n);
    }
    parts = __reduce_add_sync(0xffffffffu, parts);
    part_tiles = __reduce_max_sync(0xffffffffu, part_tiles);
    if (lane == 0) S.scan[0][warp] = parts, S.scan[1][warp] = part_tiles;
    __syncthreads();
    parts = part_tiles = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) parts += S.scan[0][w], part_tiles = max(part_tiles, S.scan[1][w]);
    const int cut_share = max(wph, (tiles_all + grid - 1) / grid), whole_share = (segments + grid - 1) / grid;
    const int cut_rounds = (cut_share + wph - 1) / wph + 3;
    const int whole_rounds = whole_share * ((longest + wph - 1) / wph);
    const int part_rounds = parts <= grid ? (part_tiles + wph - 1) / wph + 2 : INT_MAX;
    const int rounds = min(cut_rounds, min(whole_rounds, part_rounds));
    const int mode = rounds == whole_rounds ? kWhole : rounds == part_rounds ? kParts : kCut;
    const int share = mode == kCut ? cut_share : mode == kParts ? 1 : whole_share;
    const int total = mode == kCut ? tiles_all : mode == kParts ? parts : segments;
    const int64_t begin = (int64_t)blockIdx.x * share;
    const int end = (int)min((int64_t)total, begin + share);
    if (begin >= end) return;
    const List list = {mode, share, tiles_all, grid, groups, end};
    if (tid == 0) S.list = list;
    int carry = 0;
    for (int b0 = 0; b0 < batch; b0 += T) {
        const int b = b0 + tid;
        int v = 0;
        if (b < batch) {
            bool bad;
            if (!once) mine = sequence_of<RT>(g, b, &bad);
            v = mine.row_tiles ? units_of(list, mine) * mine.row_tiles * groups : 0;
        }
        int sum = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += n;
        }
        __syncthreads();
        if (lane == 31) S.scan[0][warp] = sum;
        __syncthreads();
        int before = carry;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w < warp) before += S.scan[0][w];
            carry += S.scan[0][w];
        }
        before += sum;
        if (b < batch) S.prefix[b + 1] = before;
        // The sequence that the CTA's share begins in.
        if (v && begin >= before - v && begin < before) fill_piece<RT>(g, list, (int)begin, b, before - v, mine, S.piece[0]);
    }

    // ---- pieces: S.piece[0] is there after the next barrier
    // This warp's tiles of a piece: `first`, `first` + wph, ...; with the pages of the next
    // 32 / ppt of them in the lanes: lane i holds page i % ppt of tile i / ppt.
    const uint32_t page_bytes = (uint32_t)(D << ps);
    const int batch_tiles = 32 / ppt;
    const int32_t* table = nullptr;
    int first = 0, cnt = 0, pages = 0, head = 0, ids = 0, issued = 0, slot_in = 0, in_flight = 0;
    auto fetch_ids = [&](int i) {
        const int tile = first + (i + lane / ppt) * wph, p = tile * ppt + lane % ppt;
        ids = -1;
        if (i + lane / ppt < cnt && p < pages) {
            ids = __ldg(table + p);
            if (ids < 0 || ids >= C.num_pages) {
                atomicCAS(g.status, 0, kStatusIndex);
                ids = 0;  // read something of the cache rather than nothing
            }
        }
    };
    auto enter = [&](const Piece& p) {
        cnt = p.len > 0 && p.n > my_turn ? (p.n - my_turn + wph - 1) / wph : 0;
        first = p.tile + my_turn;
        table = C.page_table + p.b * C.table_stride;
        pages = (p.len + (1 << ps) - 1) >> ps;
        head = p.h0 + my_head;
        issued = 0;
        fetch_ids(0);
    };
    // Next half tile of the piece (keys of a tile, then its values) into the ring.
    auto issue = [&]() {
        if (issued >= 2 * cnt) return;
        const int i = issued >> 1;
        if ((issued & 1) == 0 && i > 0 && i % batch_tiles == 0) fetch_ids(i);
        const int id = __shfl_sync(0xffffffffu, ids, (i % batch_tiles) * ppt + lane % ppt);
        const bool mine = lane < ppt && id >= 0;
        const int count = __popc(__ballot_sync(0xffffffffu, mine));
        const uint32_t bar = smem_u32(&S.full[warp][slot_in]);
        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)count * page_bytes);
        __syncwarp();
        if (mine) {
            const uint8_t* codes = issued & 1 ? C.v_codes : C.k_codes;
            bulk_load(ring + (uint32_t)(warp * kSlots + slot_in) * kHalf + lane * page_bytes,
                      codes + ((int64_t)id * Hkv + head) * page_bytes, page_bytes, bar);
        }
        ++issued, ++in_flight;
        slot_in = slot_in + 1 == kSlots ? 0 : slot_in + 1;
    };
    // The scales of this lane's 16 keys of tile i (one page each).
    float sk_next = 0.f, sv_next = 0.f;
    auto fetch_scales = [&](int i) {
        const int p = (first + i * wph) * ppt + ((t * 16) >> ps);
        sk_next = sv_next = 0.f;
        if (i < cnt && p < pages) {
            int id = __ldg(table + p);
            if (id < 0 || id >= C.num_pages) id = 0;
            sk_next = __ldg(C.k_scales + (int64_t)id * Hkv + head);
            sv_next = __ldg(C.v_scales + (int64_t)id * Hkv + head);
        }
    };

    // Queries of a piece: thread (row, unit of 8 channels), kPasses rows one after another.
    constexpr int kUnitsRow = D / 8, kPer = T / kUnitsRow;
    constexpr int kPasses = kGroup * kRows / kPer;  // of the most rows
    const int q_unit = tid % kUnitsRow;
    auto query_row = [&](const Piece& p, int r, int* token, int* h) {  // r: row of the piece
        const int row = p.row0 + r % R;
        const bool in = r < hp * R && row < p.tq * group;
        *token = in ? row / group : 0;
        *h = (p.h0 + r / R) * group + (in ? row - *token * group : 0);
        return in;
    };
    bool turned;
    int cl, ch;
    rope_channels(g.a.rope, q_unit, &turned, &cl, &ch);
    struct Query {
        float x[8], c[4], s[4];
    };
    auto load_query = [&](const Piece& p, int pass, Query& q) {
        float(&x)[8] = q.x;
        int token, h;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.f;
        if (query_row(p, pass * kPer + tid / kUnitsRow, &token, &h)) {
            const int64_t e = (p.o0 + token) * g.a.q_token_stride + h * g.a.q_head_stride;
            load_four(g.a.query, g.a.dtype, e + cl, g.q_vec, x);
            load_four(g.a.query, g.a.dtype, e + ch, g.q_vec, x + 4);
            const int position = p.len - p.tq + token;
            if (turned && position >= 0) rope_load(g.a.rope, position, q_unit, q.c, q.s);
        }
    };
    // Rotated, scaled to fp16's upper range by a power of two, split into two terms.
    auto put_query = [&](const Piece& p, int pass, Query& q, int which) {
        float(&x)[8] = q.x;
        const int r = pass * kPer + tid / kUnitsRow;
        int token, h;
        const bool in = query_row(p, r, &token, &h);
        const int position = p.len - p.tq + token;
        if (in && turned && position >= 0) rope_apply(g.a.rope, q.c, q.s, x);
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));
#pragma unroll
        for (int o = kUnitsRow / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        // 2^up brings the row's largest |x| to [2^14, 2^15); its exponent is kept within what
        // both 2^up and 2^-up can hold.
        const int ex = min(max((int)(__float_as_uint(m) >> 23), 30), 250) - 127;
        const float up = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
        const float down = __uint_as_float((uint32_t)(127 - 14 + ex) << 23);
        if (r >= hp * R) return;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const int d = w ? ch : cl;  // channels d .. d + 3
            uint4 f;
            split_f16(x[4 * w] * up, x[4 * w + 1] * up, &f.x, &f.y);
            split_f16(x[4 * w + 2] * up, x[4 * w + 3] * up, &f.z, &f.w);
            S.q[r / kRows][(d / 64) * 4 + (d % 16) / 4][(r % kRows) * 4 + (d % 64) / 16] = f;
        }
        if (q_unit == 0) {
            RowInfo i;
            i.factor = g.a.scale * kLog2e * down;
            i.limit = !in ? -1 : g.a.causal ? position : p.len - 1;
            const int64_t low = g.a.window > 0 ? (int64_t)position - g.a.window + 1 : 0;
            i.low = low > 0 ? (int)low : 0;
            i.index = in ? (p.o0 + token) * g.a.heads + h : -1;
            S.row[which][r] = i;
            if (in) {
                atomicMin(&S.limit_min[which][r / R], i.limit);
                atomicMax(&S.low_max[which][r / R], i.low);
            }
        }
    };
    auto clear_limits = [&](int which) {
        if (tid < hp) S.limit_min[which][tid] = INT_MAX, S.low_max[which][tid] = 0;
    };

    uint32_t phase = 0;  // parity bit of each slot's next wait
    int slot_out = 0, which = 0;
    bool ok = true;
    auto await = [&]() {  // the oldest half tile in flight; its place in the ring
        const uint32_t bar = smem_u32(&S.full[warp][slot_out]);
        ok = __all_sync(0xffffffffu, wait_bounded(bar, (phase >> slot_out) & 1u, g.wait_ns, &S.failed));
        const uint32_t at = ring + (uint32_t)(warp * kSlots + slot_out) * kHalf;
        if (ok) {
            phase ^= 1u << slot_out, --in_flight;
            slot_out = slot_out + 1 == kSlots ? 0 : slot_out + 1;
        }
        return at;
    };

    const int passes = (hp * R + kPer - 1) / kPer;  // of this call
    clear_limits(0);
    __syncthreads();
    {
        Query x[kPasses];
#pragma unroll
        for (int pass = 0; pass < kPasses; ++pass)
            if (pass < passes) load_query(S.piece[0], pass, x[pass]);
        enter(S.piece[0]);
        issue();
        issue();
        issue();
        fetch_scales(0);
#pragma unroll
        for (int pass = 0; pass < kPasses; ++pass)
            if (pass < passes) put_query(S.piece[0], pass, x[pass], 0);
    }
    if (tid == T - 1 && S.piece[0].more) make_piece<RT>(g, S.list, S.prefix, S.piece[0].after, S.piece[1]);
    __syncthreads();

    for (int turn = 0;; turn = turn == 2 ? 0 : turn + 1) {
        float O[RT][kNt][2], m_run[RT], l_run[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            m_run[rt] = -INFINITY, l_run[rt] = 0.f;
#pragma unroll
            for (int i = 0; i < kNt; ++i) O[rt][i][0] = O[rt][i][1] = 0.f;
        }
        const RowInfo* rows = S.row[which] + my_head * R;
        const int limit_min = S.limit_min[which][my_head], low_max = S.low_max[which][my_head];

        for (int i = 0; i < cnt; ++i) {
            const float sk = sk_next, sv = sv_next;
            fetch_scales(i + 1);
            const int tile_key = (first + i * wph) * kTile;
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
                    for (int k = 0; k < 4; ++k) qf[rt][k] = S.q[my_head * RT + rt][4 * c + k][lane];
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
            // A wait ran out: copies still in flight must land before the CTA leaves, and it
            // goes on without any (the tickets have to come out even; outputs are undefined).
            if (lane == 0) record_failure(g.status, &S.failed);
            for (; in_flight > 0; --in_flight) {
                wait_bounded(smem_u32(&S.full[warp][slot_out]), (phase >> slot_out) & 1u, kDrainNs, nullptr);
                phase ^= 1u << slot_out;
                slot_out = slot_out + 1 == kSlots ? 0 : slot_out + 1;
            }
        }

        const Piece& P = S.piece[turn];
        const int next = turn == 2 ? 0 : turn + 1;
        const Piece& N = S.piece[next];
        const bool more = P.more;
        // ---- the next piece's first copies take two of the ring's three slots, this one's
        // outputs the third
        const uint32_t keep = (uint32_t)(warp * kSlots + (slot_in + 2) % kSlots) * kHalf;
        if (more) {
            enter(N);
            if (!ok) cnt = 0;
            issue();
            issue();
            fetch_scales(0);
        }
        Query x[kPasses];
        if (more) {
#pragma unroll
            for (int pass = 0; pass < kPasses; ++pass)
                if (pass < passes) load_query(N, pass, x[pass]);
            clear_limits(which ^ 1);
        }
        if (lane == 0) S.merge[warp] = keep;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            float l = l_run[rt];
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            const int r = rt * kRows + gq;
            if (t == 0) S.m[warp][r] = m_run[rt], S.l[warp][r] = l;
            float* o = reinterpret_cast<float*>(ring_ptr + keep) + r * D + 2 * t;
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt)
                *reinterpret_cast<float2*>(o + nt * 8) = make_float2(O[rt][nt][0], O[rt][nt][1]);
        }
        __syncthreads();

        // ---- join a head's warps.  Partial pieces: slot 0 for the CTA's first (begun by an
        // earlier CTA), 1 for its last.
        constexpr int kQuads = R * D / 4;
        for (int i = tid - my_head * wph * 32; i < kQuads; i += wph * 32) {
            const int r = i / (D / 4), d = (i % (D / 4)) * 4, w0 = my_head * wph;
            float mx = -INFINITY;
            for (int w = w0; w < w0 + wph; ++w) mx = fmaxf(mx, S.m[w][r]);
            const float base = mx == -INFINITY ? 0.f : mx;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            float l = 0.f;
#pragma unroll 2
            for (int w = w0; w < w0 + wph; ++w) {
                const float c = ex2(S.m[w][r] - base);
                const float4 v = *reinterpret_cast<const float4*>(ring_ptr + S.merge[w] + (r * D + d) * 4);
                o.x = fmaf(v.x, c, o.x), o.y = fmaf(v.y, c, o.y);
                o.z = fmaf(v.z, c, o.z), o.w = fmaf(v.w, c, o.w);
                l = fmaf(S.l[w][r], c, l);
            }
            if (P.cut) {
                float* part = part_at<D, RT>(g, blockIdx.x, !P.later, my_head);
                *reinterpret_cast<float4*>(part + r * D + d) = o;
                if (d == 0) part[R * D + r] = mx, part[R * D + R + r] = l;
            } else {
                emit(g, S.row[which][my_head * R + r].index, D, d, o, l, base);
            }
        }
        if (P.cut) {
            const int c0 = P.c0, c1 = P.c1;  // the CTAs that share these heads' keys
            __syncthreads();
            if (tid == 0) {
                __threadfence();
                S.last = atomicAdd(g.tickets + c0, 1) == c1 - c0;
                __threadfence();
                if (S.last) g.tickets[c0] = 0;
            }
            __syncthreads();
            if (S.last) join_parts<D, RT, W>(g, P, S.row[which]);
        }
        if (!more) break;
        which ^= 1;
        if (tid == T - 1 && N.more)
            make_piece<RT>(g, S.list, S.prefix, N.after, S.piece[next == 2 ? 0 : next + 1]);
#pragma unroll
        for (int pass = 0; pass < kPasses; ++pass)
            if (pass < passes) put_query(N, pass, x[pass], which);
        // The next copies also write where the joined outputs were.
        fence_async_shared();
        __syncthreads();
        issue();
    }
}

template <int D, int RT>
cudaError_t launch(const SplitArgs& g, int64_t grid, cudaStream_t stream) {
    constexpr int bytes = kWarps * kSlots * kTile * D + 128;
    static_assert(ctas_of(D, RT) * (bytes + sizeof(Shared<D, RT>) + 1024) <= 228 * 1024, "shared memory of one SM");
    const cudaError_t e = kernel_smem_once<attention_split_kernel<D, RT>>(bytes);
    if (e != cudaSuccess) return e;
    attention_split_kernel<D, RT><<<(unsigned)grid, 32 * kWarps, bytes, stream>>>(g);
    return cudaGetLastError();
}

}  // namespace

cudaError_t attention_split_launch(const q4lin_kv_cache_t& cache, const q4lin_attention_t& a,
                                   int64_t rows_max, const LaunchCtx& c) {
    const int64_t group = a.heads / cache.kv_heads;
    const int64_t rows = std::min(rows_max, a.max_query * group);
    const int D = (int)cache.head_dim;
    const bool two = rows > kRows && D != 256;
    const int R = two ? 2 * kRows : kRows;
    cudaError_t err = cudaSuccess;
    // Sequences in groups that the kernel's list holds.
    for (int64_t b = 0; b < cache.batch && err == cudaSuccess; b += kMaxBatch) {
        SplitArgs g;
        g.cache = cache;
        g.a = a;
        g.cache.batch = std::min<int64_t>(kMaxBatch, cache.batch - b);
        g.cache.page_table += b * cache.table_stride;
        g.a.offsets += b;
        g.a.lengths += b;
        g.page_shift = cache.page_size == 16 ? 4 : cache.page_size == 32 ? 5 : 6;
        g.rows_max = rows_max;
        g.q_vec = reinterpret_cast<uintptr_t>(a.query) % (4 * dtype_size(a.dtype)) == 0 &&
                  a.q_token_stride % 4 == 0 && a.q_head_stride % 4 == 0;
        g.ws = c.ws;
        g.tickets = c.tickets;
        g.status = c.status_word;
        g.wait_ns = c.wait_limit_ns;
        // One or two CTAs per SM, and no more than the longest possible list has tiles for.
        const int64_t slots = (int64_t)c.sm_count * ctas_of(D, two ? 2 : 1);
        const int64_t tiles = (cache.pages_per_sequence * cache.page_size + kTile - 1) / kTile;
        const int64_t row_tiles = std::min((a.tokens * group + R - 1) / R + g.cache.batch,
                                           ((rows + R - 1) / R) * g.cache.batch);
        const int64_t grid = std::max<int64_t>(
            1, std::min<int64_t>(slots, (tiles * row_tiles * cache.kv_heads + kWarps - 1) / kWarps));
        // More heads at a time leave fewer joins of warps and fewer of them idle at the end of
        // a piece, as long as every CTA finds a piece of its own.
        g.heads_per = 1;
        for (int hp = 2; hp * (two ? 2 : 1) <= max_group(D) && cache.kv_heads % hp == 0 &&
                         row_tiles * cache.kv_heads / hp >= slots;
             hp *= 2)
            g.heads_per = hp;
        switch (D) {
            case 64: err = two ? launch<64, 2>(g, grid, c.stream) : launch<64, 1>(g, grid, c.stream); break;
            case 128: err = two ? launch<128, 2>(g, grid, c.stream) : launch<128, 1>(g, grid, c.stream); break;
            default: err = launch<256, 1>(g, grid, c.stream); break;
        }
    }
    return err;
}

}  // namespace q4lin
