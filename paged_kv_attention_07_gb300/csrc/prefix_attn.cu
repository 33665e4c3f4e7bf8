// prefix_attn.cu -- attention for groups of requests whose first tokens are the
// same: the keys of a group's common tokens are read once for all its query rows.
//
// Softmax over a set of keys splits over any partition of them: each part gives
// the normalised sum O_i of its values and L_i = log sum exp(s), and
//     out = sum_i e^(L_i - L) O_i,   L = log sum_i e^(L_i).
// The parts here are a group's common keys, whose query rows are those of all the
// group's tokens, and a request's own keys with the rows of its own tokens
// (causal among the new ones). Either way a row is a (token, query head) of one kv
// head's group of heads: 128 / G tokens make a tile of up to 128 rows, which
// lie in q as one box of [tokens, G heads, d].
//
// Work unit: (segment, kv head, one or two row tiles) x its key tiles of 128 keys.
// All units' key tiles, weighted by their cost, form one line that is cut into
// equal shares, one per CTA (one CTA per SM): every SM gets the same work however
// the groups, lengths and heads fall, and a unit is cut where a share ends. Each
// CTA finds its share by itself from the lengths (prefix sums, a few microseconds
// at a thousand requests): no planning launch. Pieces go to the workspace in 32 bits
// and a second kernel joins each token's.
//
// Per CTA, 12 warps: K and V producers (TMA boxes of pages through the block
// table), two MMA-issuing warps, two softmax warpgroups ("lanes" 0 and 1, one
// thread per row); over codes 4 warps more, which split the rows and widen V. With
// two row tiles in a unit, lane k has row tile k and every key tile serves both;
// with one, the lanes take alternate key tiles of the same rows, so that one's
// exponentials overlap the other's products, and leave two pieces. Tensor memory:
// S_k (128 columns, P_k written over it) and O_k.
// The tensor cores ask for P in the type of V, bf16. A weight is two bf16 numbers, off by 2^-15
// of it, and takes two products: the result's error is that of its own rounding (0.0017 against 64 bits; with
// one number 0.0023, and 24 groups of 8 beams took 3 % less time, 64 requests 6, 4 beams 1). Over codes
// P is one f16 number (below). The weights' sum is kept from the unrounded values in 32 bits.
//
// Measured, with the join: 24 groups of 8 (1000 to 8192 common tokens, 1 to 512 own, 8 kv heads of 128,
// G = 4) 97 us, 4.2 TB/s of what has to be read; 64 requests behind 16384 tokens 50 us; 4 beams
// behind 8192 21.5 us; 32 groups of 4 over an 8-bit cache 87 us, 2.9 TB/s. A full tile more of
// long groups takes 1.4 us of an SM (6.9 TB/s), of 8-bit codes 1.0 (5.0), with two row tiles 2.4 to 2.9 (0.9 PFLOP/s and
// more, without the weights' second product); lengths, shares and the join 12 us of each call. A
// request's own unit of a tile or two takes 2 to 3 us: it leaves the stages half empty, and its steps
// follow each other on one lane (first copies 2, S and softmax of an edge tile 2, P V 1, result 1).
#include <float.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "params.cuh"
#include "plan.cuh"
#include "tcgen05.cuh"

namespace pka {

namespace {

constexpr int kKeys = 128;  // keys of a key tile
constexpr int kPieces = 256;  // pieces of a list
constexpr int kMaxSegs = 2 * kMaxRequests;
constexpr int kChunks = kMaxSegs / 32;  // warp-sized runs of segments
// Costs on the line: a key tile for one row tile, for two, and what a unit takes besides
// (its first copies, its end, lanes that wait for one another), as measured: 24 groups of 8
// beams with (1, 2, 1) 97 us, (1, 2, 2) 104, (1, 2, 3) 112, 64 requests 50, 50 and 51; over an 8-bit
// cache 32 groups of 4 with (1, 2, 3) 87.6 us, (1, 2, 4) 91, (1, 2, 2) 89.4, (1, 2, 1) 103.
constexpr int kCostOne = 1, kCostTwo = 2;

struct Seg {
    int q0, n;      // its tokens
    int c0, c1;     // its keys
    int base;       // the first key tile's first key
    int nkt, nrt;   // key tiles; units per kv head
    int w, e;       // costs: of a key tile, and of a unit besides
};

// How a token's rows and a unit's key tiles come from a segment.
PKA_DEVICE Seg make_seg(const PrefixParams& p, int q0, int n, int c0, int c1) {
    Seg s;
    s.q0 = q0;
    s.n = n;
    s.c0 = c0;
    s.c1 = c1;
    s.base = c0 & ~(p.bs - 1);
    s.nkt = n > 0 && c1 > c0 ? (c1 - s.base + kKeys - 1) / kKeys : 0;
    s.nrt = s.nkt == 0 ? 0 : n <= p.upt ? 1 : (n + p.upt - 1) / p.upt;
    s.w = p.upt > p.tpt && n > p.tpt ? kCostTwo : kCostOne;
    s.e = p.cost_unit;
    return s;
}

// A group of one request has no common keys: they are its own.
PKA_DEVICE int common_keys(int r0, int r1, int prefix) { return r1 - r0 > 1 ? prefix : 0; }

// The last i in [0, n) with a[i] <= x (a[0] <= x).
PKA_DEVICE int last_at_most(const int32_t* a, int n, int x) {
    int lo = 0, hi = n - 1;
#pragma unroll 1
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The line in shares of `base` or base + 1.
struct Shares {
    int base, rem;
    PKA_DEVICE Shares(int total, int ncta) : base(total / ncta), rem(total % ncta) {}
    PKA_DEVICE int start(int cta) const { return cta * base + min(cta, rem); }
    PKA_DEVICE int cta_of(int x) const {
        const int cut = rem * (base + 1);
        return x < cut ? x / (base + 1) : rem + (x - cut) / base;
    }
};
PKA_DEVICE int unit_cost(const Seg& s) { return s.nkt > 0 ? s.e + s.nkt * s.w : 0; }
// The first key tile of a unit that starts at `us` whose place is at or past x
// (tile t's place: us + e + t w).
PKA_DEVICE int first_tile(int x, int us, const Seg& s) {
    const int d = x - us - s.e;
    return d <= 0 ? 0 : min(s.nkt, (d + s.w - 1) / s.w);
}

// Of a piece's key tiles from t0 on those behind position `end` (past the unit's
// last token) have nothing to see: they are left out, but for one.
PKA_DEVICE int seen_tiles(const Seg& s, int t0, int t1, int end) {
    return max(1, min(t1 - t0, (min(s.c1, end) - (s.base + t0 * kKeys) + kKeys - 1) / kKeys));
}

// Replaces the halves of w whose bits are all set where kMask's are (infinities and NaN) by zeros.
template <uint32_t kMask, int N>
PKA_DEVICE bool take_out(uint32_t (&w)[N]) {
    bool any = false;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if ((w[e] & kMask) == kMask) {
            w[e] &= 0xffff0000u;
            any = true;
        }
        if ((w[e] >> 16 & kMask) == kMask) {
            w[e] &= 0xffffu;
            any = true;
        }
    }
    return any;
}

// Two weights p >= 0 as two bf16 numbers each, p cut off, and the rest, rounded (2^-16 of p at most). 2^-17 of p more
// keeps the rest above 0 where p is (down to 2^-116), so that an infinite value is not multiplied by 0.
PKA_DEVICE void split_weights(float p0, float p1, uint32_t& high, uint32_t& rest) {
    const uint32_t b0 = __float_as_uint(p0), b1 = __float_as_uint(p1);
    high = __byte_perm(b0, b1, 0x7632);
    float d0, d1;
    fma2(d0, d1, p0, p1, 1.f + 1.f / 131072, __uint_as_float(b0 & 0xffff0000u | 0x80000000u),
         __uint_as_float(b1 & 0xffff0000u | 0x80000000u));
    rest = pack_bf16(d0, d1);
}

struct Piece {
    int table;      // the request whose block table row is read
    int h;          // kv head
    int q0, ntok;   // the unit's tokens
    int kb0, nkt;   // first key of the first tile, key tiles
    int c0, c1;     // visible keys of the segment
    int pos0;       // position of token q0 (past everything for common keys)
    int row;        // its result's first row in the workspace; common keys: bit 31
};

template <int D, bool kFp8>
struct PxCfg {
    // Registers by role: the launch gives every thread the same.
    static constexpr int kThreads = kFp8 ? 512 : 384;
    static constexpr int kRegsLaunch = kFp8 ? 128 : 168, kRegsIssue = kFp8 ? 64 : 80;
    static constexpr int kRegsSoftmax = kFp8 ? 176 : 208, kRegsWiden = 96;
    static_assert(128 * kRegsIssue + 256 * kRegsSoftmax + (kFp8 ? 128 * kRegsWiden : 0) <= kThreads * kRegsLaunch,
                  "register split");
    static constexpr int kRowTiles = 2;              // places for row tiles
    static constexpr int kChunk = D / 64;            // 64-wide swizzle chunks per row
    static constexpr int kChunkBytes = 128 * 128;    // 128 rows x 128 B
    static constexpr int kTileBytes = kChunk * kChunkBytes;
    static constexpr int kCodeBytes = kKeys * D;     // a key tile in 8 bits
    static constexpr int kStagesK = 2, kStageK = kFp8 ? kCodeBytes : kTileBytes;
    static constexpr int kStagesV = 2;               // of V in 16 bits
    static constexpr int kStagesCode = kFp8 ? 2 : 0;  // of V's codes
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kRowTiles * kTileBytes;
    static constexpr int kOffV = kOffK + kStagesK * kStageK;
    static constexpr int kOffCode = kOffV + kStagesV * kTileBytes;
    // the lengths, while a list is made, where the tiles go later
    static constexpr int kOffMeta = kOffK;
    static constexpr int kMetaBytes = (int)sizeof(int32_t) * (4 * kMaxRequests + 2);
    static constexpr int kOffTiles = kOffCode + kStagesCode * kCodeBytes;
    static constexpr int kOffPiece = kOffTiles > kOffMeta + kMetaBytes ? kOffTiles : (kOffMeta + kMetaBytes + 15) / 16 * 16;
    static constexpr int kOffSums = kOffPiece + kPieces * (int)sizeof(Piece);
    static constexpr int kOffUnit = kOffSums + (kChunks + 1) * 8;  // [4][128] of the row tiles' rows in 8 bits
    static constexpr int kOffBar = kOffUnit + (kFp8 ? 4 * 128 * 4 : 0);
    static constexpr int kSmem = kOffBar + 256 + 1024;
    static constexpr uint32_t kColS = 0, kColO = 256, kTmemCols = 512;
    static_assert(kSmem <= 232448, "shared memory");
};

// Entries [32 chunk, 32 chunk + 32) of the table from a piece's first page on, one per lane.
PKA_DEVICE int table_entry(const PrefixParams& p, const Piece& U, int chunk, int lane) {
    const int pos = U.kb0 + ((32 * chunk + lane) << p.bs_log2);
    return pos < U.c1 ? __ldg(p.block_table + (int64_t)U.table * p.max_blocks + (pos >> p.bs_log2)) : 0;
}

// The lengths of a call in shared memory.
struct Meta {
    int32_t* starts;  // [groups + 1]
    int32_t* prefix;  // [groups]
    int32_t* qsl;     // [B + 1]
    int32_t* lens;    // [B]
};

// Segment s: the groups, then, from own0 on, the requests (own0 is the number of
// groups, up to whole runs of 32).
PKA_DEVICE Seg seg_of(const PrefixParams& p, const Meta& m, int s, int& err) {
    if (s < p.groups) {
        const int r0 = m.starts[s], r1 = m.starts[s + 1], len = m.prefix[s];
        if (r0 > r1 || r0 < 0 || r1 > p.B) {
            err |= PKA_DEVERR_INDEX;
            return make_seg(p, 0, 0, 0, 0);
        }
        if (len < 0) err |= PKA_DEVERR_SEQ_LEN;
        const int q0 = m.qsl[r0], q1 = m.qsl[r1];
        return make_seg(p, q0, q1 - q0, 0, common_keys(r0, r1, len));
    }
    if (s < p.own0 || s >= p.own0 + p.B) return make_seg(p, 0, 0, 0, 0);
    const int r = s - p.own0;
    const int q0 = m.qsl[r], q1 = m.qsl[r + 1], len = m.lens[r];
    if (q0 < 0 || q1 < q0 || q1 > p.T || (r == 0 && q0 != 0)) err |= PKA_DEVERR_QUERY_START_LOC;
    const int n = q1 - q0;
    if (n <= 0) return make_seg(p, q0, 0, 0, 0);
    if (n > p.max_query) err |= PKA_DEVERR_QUERY_LEN;
    if (len < n || len > p.max_seq) err |= PKA_DEVERR_SEQ_LEN;
    const int g = last_at_most(m.starts, p.groups, r);
    const int have = m.prefix[g];
    if (have < 0 || have > len - n) err |= PKA_DEVERR_SEQ_LEN;
    return make_seg(p, q0, n, common_keys(m.starts[g], m.starts[g + 1], have), len);
}

// Inclusive sums over the warp's lanes.
PKA_DEVICE void warp_sums(int& a, int& b) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
            a += x;
            b += y;
        }
    }
}

// kSeveral: requests may have more than one new token. The code that keeps a later token's
// infinities from earlier ones costs 3 to 8 % where nothing calls for it (24 groups of 8 beams 105
// us with it, 97 without; 64 requests 51.1 and 49.7; 8-bit 90.6 and 87.2), by its size alone.
template <int D, bool kFp8, bool kSeveral>
__global__ void __launch_bounds__((PxCfg<D, kFp8>::kThreads), 1)
    prefix_attn_kernel(const __grid_constant__ PrefixMaps maps, const PrefixParams p) {
    using C = PxCfg<D, kFp8>;
    constexpr int kPxThreads = C::kThreads;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint64_t* q_full = bars + 0;    // [2] per row tile's place: landed
    uint64_t* q_empty = bars + 2;   // [2] its unit's last S product is done
    uint64_t* k_full = bars + 4;    // [2] per K stage
    uint64_t* k_empty = bars + 6;
    uint64_t* v_full = bars + 8;    // [2] per V stage
    uint64_t* v_empty = bars + 10;
    uint64_t* s_full = bars + 12;   // [2] per lane: its S tile is in tensor memory
    uint64_t* p_full = bars + 14;   // [2] its P is (4 warp arrivals)
    uint64_t* pv_done = bars + 16;  // [2] the product that read its P is done
    uint64_t* o_free = bars + 18;   // [2] its O has been read (4 warp arrivals)
    uint64_t* p_half = bars + 20;   // [2] P of keys 0..63 is there (4 warp arrivals)
    uint64_t* c_full = bars + 22;   // [2] per stage of V's codes: landed
    uint64_t* c_empty = bars + 24;  // [2] widened (4 warp arrivals)
    float* row_unit = reinterpret_cast<float*>(smem + C::kOffUnit);
    Piece* pieces = reinterpret_cast<Piece*>(smem + C::kOffPiece);
    int* run_cost = reinterpret_cast<int*>(smem + C::kOffSums);  // before each run of 32 segments
    int* run_rows = run_cost + kChunks + 1;  // ... and of results
    Meta meta;
    meta.starts = reinterpret_cast<int32_t*>(smem + C::kOffMeta);
    meta.prefix = meta.starts + p.groups + 1;
    meta.qsl = meta.prefix + p.groups;
    meta.lens = meta.qsl + p.B + 1;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    // Key tiles after which lane 0's next S has been issued: with two row tiles,
    // lane 1's product lets that S go first.
    __shared__ volatile int s_next0;
    __shared__ int s_pieces;  // listed
    __shared__ uint32_t s_odd[kPieces / 32];  // bit per piece: a value was taken out of its tiles (see below)

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        static_assert(C::kRowTiles == 2 && C::kStagesK == 2 && C::kStagesV == 2, "places of the barriers");
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], kFp8 ? 4 : 1);
            mbar_init(&q_empty[i], 1);
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], kFp8 ? 4 : 1);
            mbar_init(&v_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&p_half[i], 4);
            mbar_init(&pv_done[i], 1);
            mbar_init(&o_free[i], 4);
            mbar_init(&c_full[i], 1);
            mbar_init(&c_empty[i], 4);
        }
        fence_barrier_init();
        s_abort = 0;
        s_next0 = 0;
        tma_prefetch_desc(&maps.q);
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
    }
    // rows of a row tile that no token fills (128 / G * G < 128) stay zero
    if (p.tpt * p.G < 128)
#pragma unroll 1
        for (int i = tid; i < C::kRowTiles * C::kTileBytes / 16; i += kPxThreads)
            reinterpret_cast<uint4*>(smem + C::kOffQ)[i] = make_uint4(0, 0, 0, 0);
    if (warp == 1) tmem_alloc(&s_tmem, C::kTmemCols);
    grid_dep_wait();
    grid_dep_launch();  // (the join reads the lengths before it waits: what wrote them is done)

    // ---------------------------------------------------------------- the line
    const int runs = (p.own0 + p.B + 31) / 32;
    auto load_meta = [&] {
#pragma unroll 1
        for (int i = tid; i <= p.B; i += kPxThreads) {
            meta.qsl[i] = __ldg(p.qsl + i);
            if (i < p.B) meta.lens[i] = __ldg(p.seq_lens + i);
            if (i <= p.groups) meta.starts[i] = __ldg(p.starts + i);
            if (i < p.groups) meta.prefix[i] = __ldg(p.prefix + i);
        }
        __syncthreads();
    };
    load_meta();
    int err = 0;
    if (tid == 0 && (meta.starts[0] != 0 || meta.starts[p.groups] != p.B)) err = PKA_DEVERR_INDEX;
    if (tid == 0) s_pieces = 0;
    if (tid < kPieces / 32) s_odd[tid] = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = s_tmem;
    const uint32_t sm_base = smem_u32(smem);
    const int ncta = gridDim.x, cta = blockIdx.x;
    int lo = 0, hi = 0;  // the share

    // state of the roles across lists
    uint32_t kv_it = 0, q_it = 0;  // key tiles and row tiles so far
    uint32_t nl0 = 0, nl1 = 0;  // S products (or P . V products) of each lane
    uint32_t n_s = 0, n_p = 0;  // S tiles of this softmax lane, pieces
    uint32_t uo0 = 0, uo1 = 0;  // units in which each lane had key tiles

    // Pass 0 sums the runs of segments; pass j > 0 lists the pieces that begin in the
    // j-th stretch of the share (a piece costs cost_unit + kCostOne at least but for
    // the first, so a list holds a stretch's) and works them off. One loop body for
    // both: what runs once per launch is bound by the fetch of its instructions.
    const int stretch = (kPieces - 2) * (p.cost_unit + kCostOne);
    for (int pass = 0;; ++pass) {
        const int from = lo + (pass - 1) * stretch;
        if (pass > 1) {
            if (from >= hi) break;
            load_meta();  // (tiles were there meanwhile)
        }
#pragma unroll 1
        for (int run = warp; run < runs; run += kPxThreads / 32) {
            if (pass > 0 && (run_cost[run] >= min(hi, from + stretch) || run_cost[run + 1] <= from) &&
                (pass > 1 || run % ncta != cta))
                continue;
            const int s = run * 32 + lane;
            const Seg g = seg_of(p, meta, s, err);
            const int units = g.nrt * p.Hkv, each = unit_cost(g), cost = units * each, rows = units > 0 ? g.n * p.Hq : 0;
            if (pass == 0) {
                const int c = __reduce_add_sync(0xffffffffu, cost), r = __reduce_add_sync(0xffffffffu, rows);
                if (lane == 0) {
                    run_cost[run] = c;
                    run_rows[run] = r;
                }
                continue;
            }
            int ci = cost, ri = rows;
            warp_sums(ci, ri);
            const int cs = run_cost[run] + ci - cost, rs = run_rows[run] + ri - rows;
            if (pass == 1 && run % ncta == cta && s < p.own0 + p.B) {  // for the join
                p.seg_cost[s] = cs;
                p.seg_row[s] = rs;
            }
            if (units == 0 || cs >= hi || cs + cost <= lo) continue;
#pragma unroll 1
            for (int u = cs >= lo ? 0 : (lo - cs) / each; u < units && cs + u * each < hi; ++u) {
                const int at = cs + u * each, begin = max(at, lo);
                const int t0 = first_tile(lo, at, g), t1 = first_tile(hi, at, g);
                if (t0 >= t1 || begin < from || begin >= from + stretch) continue;
                Piece x;
                x.h = g.nrt == 1 ? u : u / g.nrt;
                const int rt = u - x.h * g.nrt;
                x.q0 = g.q0 + rt * p.upt;
                x.ntok = min(p.upt, g.n - rt * p.upt);
                const int before = rs + (x.h * g.n + rt * p.upt) * p.G;
                x.kb0 = g.base + t0 * kKeys;
                x.c0 = g.c0;
                x.c1 = g.c1;
                if (s < p.groups) {
                    int r = meta.starts[s];
                    while (r + 1 < meta.starts[s + 1] && meta.qsl[r + 1] <= g.q0) ++r;
                    x.table = r;
                    x.pos0 = INT32_MAX / 2;
                    x.nkt = t1 - t0;
                    x.row = 2 * (before + cta * p.most_pre) | INT32_MIN;
                } else {
                    x.table = s - p.own0;
                    x.pos0 = g.c1 - g.n + (x.q0 - g.q0);
                    x.nkt = seen_tiles(g, t0, t1, x.pos0 + x.ntok);
                    x.row = 2 * (before - run_rows[p.own0 / 32] + cta * p.most_own);
                }
                pieces[atomicAdd(&s_pieces, 1)] = x;  // (in any order: a piece's result does not depend on it)
                // what its first copies hang on
                prefetch_l2(p.block_table + (int64_t)x.table * p.max_blocks + (x.kb0 >> p.bs_log2));
                bulk_prefetch_l2(p.q + ((int64_t)x.q0 * p.Hq + x.h * p.G) * D, (uint32_t)(p.G * D * 2));
            }
        }
        if (pass == 0) {
            if (__syncthreads_or(err)) {  // the same for every CTA
                if (cta == 0) {
                    if (err) set_error(p.err, err);
                    if (tid == 0) p.seg_cost[p.own0 + p.B] = -1;
                }
                break;
            }
            if (warp == 0) {
                int c0 = 0, rows0 = 0;
#pragma unroll 1
                for (int r0 = 0; r0 < runs; r0 += 32) {
                    const int r = r0 + lane;
                    const int c = r < runs ? run_cost[r] : 0, n = r < runs ? run_rows[r] : 0;
                    int ci = c, ni = n;
                    warp_sums(ci, ni);
                    if (r < runs) {
                        run_cost[r] = c0 + ci - c;
                        run_rows[r] = rows0 + ni - n;
                    }
                    c0 += __shfl_sync(0xffffffffu, ci, 31);
                    rows0 += __shfl_sync(0xffffffffu, ni, 31);
                }
                if (lane == 0) {
                    run_cost[runs] = c0;
                    run_rows[runs] = rows0;
                }
            }
            __syncthreads();
            const int total = run_cost[runs];
            if (cta == 0 && tid == 0) p.seg_cost[p.own0 + p.B] = total;
            const Shares shares(total, ncta);
            lo = shares.start(cta);
            hi = shares.start(cta + 1);
            continue;
        }
        fence_proxy_async_smem();  // (what was written where tiles go)
        __syncthreads();
        const int count = s_pieces;
        if (from >= hi) break;
        // Each role first gives up or takes its registers, and none goes on before all
        // have: a warp that took its own back early would leave the softmax lanes waiting.

        if (warp < 4) {
            // (the issuing warps stay whole and one elected lane issues: from a branch of one lane 24
            // groups of 8 beams took 7 % longer)
            setmaxnreg_dec<C::kRegsIssue>();
            __syncthreads();
            if (warp == 0 || warp == 2) {
                // -------------------------------------------------------- producers: Q and K; V
                const int which = warp == 0 ? 0 : 1;
                // (keys are read once, or by the few row tiles of a group at about the same time: not kept in L2, where
                // the pieces wait for the join; kept, 24 groups of 8 beams take 102 us, not 97)
                const uint64_t pol = policy_evict_first(), pol_q = policy_evict_last();
                const bool tma = p.bs >= 8;
                // of an 8-bit cache K's codes are the product's operand, V's are widened first
                uint64_t* fulls = !which ? k_full : kFp8 ? c_full : v_full;
                uint64_t* empties = !which ? k_empty : kFp8 ? c_empty : v_empty;
                const uint32_t nst = !which ? C::kStagesK : kFp8 ? C::kStagesCode : C::kStagesV;
                uint8_t* stages = smem + (!which ? C::kOffK : kFp8 ? C::kOffCode : C::kOffV);
                constexpr int kStage = C::kStageK;
                constexpr int kBoxes = kFp8 ? 1 : C::kChunk;  // 128 bytes wide
                bool ok = true;
                // Table entries are fetched 32 at a time and a chunk (or a piece) ahead: under the
                // kernel's own traffic such a load takes up to 3 us, and one for each tile held
                // back the small units' tiles by as much.
                const int per_log2 = tma ? p.bs_log2 - 2 : 0;  // log2 of a chunk's key tiles
                int ids = 0, ids_next = tma && count > 0 ? table_entry(p, pieces[0], 0, lane) : 0;
#pragma unroll 1
                for (int i = 0; i < count && ok && !warp_flag(s_abort); ++i) {
                    const Piece U = pieces[i];
                    if (!kFp8 && which == 0) {  // (beside K: a unit's V waits for older products)
                        const int nq = U.ntok > p.tpt ? 2 : 1;
                        const bool twice = U.ntok <= p.tpt / 2;
#pragma unroll 1
                        for (int k = 0; k < nq && ok; ++k, ++q_it) {
                            const int at = q_it % C::kRowTiles;
                            const uint32_t n = q_it / C::kRowTiles;
                            if (n > 0 && !mbar_wait_warp(&q_empty[at], (n - 1) & 1, p.err)) {
                                ok = false;
                                break;
                            }
                            if (lane == 0) {
                                const int boxes = twice ? 2 : 1, tokens = twice ? p.tpt / 2 : p.tpt;
                                mbar_arrive_expect_tx(&q_full[at], (uint32_t)(C::kChunk * boxes * tokens * p.G * 128));
                                for (int c = 0; c < C::kChunk * boxes; ++c)
                                    tma_load_3d(smem + C::kOffQ + at * C::kTileBytes + c / boxes * C::kChunkBytes +
                                                    c % boxes * (C::kChunkBytes / 2),
                                                twice ? &maps.q_half : &maps.q, &q_full[at], c / boxes * 64, U.h * p.G,
                                                U.q0 + k * p.tpt, pol_q);
                            }
                        }
                        if (!ok) {
                            s_abort = 1;
                            break;
                        }
                    }
                    const int32_t* bt = p.block_table + (int64_t)U.table * p.max_blocks;
#pragma unroll 1
                    for (int t = 0; t < U.nkt; ++t, ++kv_it) {
                        const int st = (int)(kv_it % nst);
                        const uint32_t n = kv_it / nst;
                        const int kb = U.kb0 + t * kKeys;
                        if (tma && (t & ((1 << per_log2) - 1)) == 0) {
                            const int chunk = (t >> per_log2) + 1;
                            ids = ids_next;
                            if (chunk << per_log2 < U.nkt) ids_next = table_entry(p, U, chunk, lane);
                            else if (i + 1 < count) ids_next = table_entry(p, pieces[i + 1], 0, lane);
                        }
                        if (n > 0 && !mbar_wait_warp(&empties[st], (n - 1) & 1, p.err)) {
                            s_abort = 1;
                            ok = false;
                            break;
                        }
                        uint8_t* dst = stages + st * kStage;
                        if (tma) {
                            const int valid = min(kKeys >> p.bs_log2, (U.c1 - kb + p.bs - 1) >> p.bs_log2);
                            if (lane == 0) mbar_arrive_expect_tx(&fulls[st], (uint32_t)(valid * kBoxes * p.bs * 128));
                            int block = __shfl_sync(0xffffffffu, ids,
                                                    ((t & ((1 << per_log2) - 1)) << (7 - p.bs_log2)) + lane & 31);
                            if (lane < valid) {
                                if (block < 0 || block >= p.num_blocks) {
                                    set_error(p.err, PKA_DEVERR_BLOCK_ID);
                                    block = 0;
                                }
                                const int row = (block * p.Hkv + U.h) << p.bs_log2;
#pragma unroll
                                for (int c = 0; c < kBoxes; ++c)
                                    tma_load_2d(dst + c * C::kChunkBytes + lane * p.bs * 128, which ? &maps.v : &maps.k,
                                                &fulls[st], c * 64, row, pol);
                            }
                        } else {  // pages of 1, 2 or 4 tokens: 16-byte copies, zeros past the end
                            const uint32_t to = smem_u32(dst);
                            const uint8_t* from = static_cast<const uint8_t*>(which ? p.v_cache : p.k_cache);
#pragma unroll 1
                            for (int ci = lane; ci < kKeys * kBoxes * 8; ci += 32) {
                                const int row = ci / (kBoxes * 8), c = ci % (kBoxes * 8), pos = kb + row;
                                const bool valid = pos < U.c1;
                                int blk = valid ? __ldg(bt + (pos >> p.bs_log2)) : 0;
                                if (blk < 0 || blk >= p.num_blocks) {
                                    set_error(p.err, PKA_DEVERR_BLOCK_ID);
                                    blk = 0;
                                }
                                const int64_t at = (((int64_t)blk * p.Hkv + U.h) << p.bs_log2) + (valid ? pos & (p.bs - 1) : 0);
                                cp_async_16_zfill(to + (c >> 3) * C::kChunkBytes + sw128(row, c & 7), from + (at * kBoxes * 8 + c) * 16,
                                                  valid);
                            }
                            cp_async_commit();
                            cp_async_wait<0>();
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&fulls[st]);
                        }
                    }
                }
                // no copy may outlive the CTA, nor meet the next list's lengths
#pragma unroll 1
                for (uint32_t back = 1; back <= nst && back <= kv_it; ++back)
                    mbar_wait_warp(&fulls[(kv_it - back) % nst], ((kv_it - back) / nst) & 1, p.err);
#pragma unroll 1
                for (uint32_t back = 1; !kFp8 && which == 0 && back <= C::kRowTiles && back <= q_it; ++back)
                    mbar_wait_warp(&q_full[(q_it - back) % C::kRowTiles], ((q_it - back) / C::kRowTiles) & 1, p.err);
            } else if (warp == 1) {
                // -------------------------------------------------------- S_k = Q K^T
                constexpr uint32_t idesc = kFp8 ? umma_idesc_f8(128, 128) : umma_idesc_bf16(128, 128, 0, 0);
                const uint32_t q_s = sm_base + C::kOffQ, k_s = sm_base + C::kOffK;
                bool ok = true;
#pragma unroll 1
                for (int i = 0; i < count && ok && !warp_flag(s_abort); ++i) {
                    const int nkt = pieces[i].nkt;
                    const bool two = !kFp8 && pieces[i].ntok > p.tpt;
                    const uint32_t q0 = q_it, q1 = q_it + (two ? 1 : 0);
                    q_it = q1 + 1;
                    if (!mbar_wait_warp(&q_full[q0 % C::kRowTiles], (q0 / C::kRowTiles) & 1, p.err) ||
                        (two && !mbar_wait_warp(&q_full[q1 % C::kRowTiles], (q1 / C::kRowTiles) & 1, p.err))) {
                        ok = false;
                        break;
                    }
#pragma unroll 1
                    for (int t = 0; t < nkt; ++t, ++kv_it) {
                        const int st = (int)(kv_it % C::kStagesK), only = (int)(kv_it & 1);
                        if (!mbar_wait_warp(&k_full[st], (kv_it / C::kStagesK) & 1, p.err)) { ok = false; break; }
#pragma unroll 1
                        for (int k = two ? 0 : only; k < (two ? 2 : only + 1); ++k) {
                            const uint32_t done = k ? nl1 : nl0;
                            if (done > 0 && !mbar_wait_warp(&pv_done[k], (done - 1) & 1, p.err)) { ok = false; break; }
                            tc_fence_after();
                            const uint32_t qa = q_s + (k == 1 ? q1 : q0) % C::kRowTiles * C::kTileBytes;
                            const uint64_t a_desc = umma_desc_sw128(qa, 16, 1024), b_desc = umma_desc_sw128(k_s + st * C::kStageK, 16, 1024);
                            const uint32_t d = tbase + C::kColS + k * 128;
                            // (a descriptor's address counts 16 bytes)
                            if constexpr (kFp8) {  // the rows' upper and lower halves (the second tile) times the codes
#pragma unroll
                                for (int ks = 0; ks < 2 * (D / 32); ++ks)
                                    umma_f8_w(d, a_desc + ((ks >= D / 32 ? C::kCodeBytes : 0) + ks % (D / 32) * 32) / 16,
                                            b_desc + ks % (D / 32) * 32 / 16, idesc, ks > 0 ? 1u : 0u);
                            } else {
#pragma unroll
                                for (int ks = 0; ks < D / 16; ++ks) {
                                    const uint32_t off = (ks >> 2) * C::kChunkBytes + (ks & 3) * 32;
                                    umma_bf16_w(d, a_desc + off / 16, b_desc + off / 16, idesc, ks > 0 ? 1u : 0u);
                                }
                            }
                            umma_commit_w(&s_full[k]);
                            if (k) ++nl1;
                            else ++nl0;
                            if (k == 0 && t > 0) s_next0 = (int)kv_it;
                        }
                        if (!ok) break;
                        umma_commit_w(&k_empty[st]);
                        if (t == nkt - 1) {
                            umma_commit_w(&q_empty[q0 % C::kRowTiles]);
                            if (two) umma_commit_w(&q_empty[q1 % C::kRowTiles]);
                        }
                    }
                    if (ok) s_next0 = (int)kv_it;  // nothing of lane 0 follows in this unit
                }
                if (!ok) s_abort = 1;
                if (nl0 > 0) mbar_wait_warp(&s_full[0], (nl0 - 1) & 1, p.err);
                if (nl1 > 0) mbar_wait_warp(&s_full[1], (nl1 - 1) & 1, p.err);
            } else if (warp == 3) {
                // -------------------------------------------------------- O_k += P_k V
                constexpr uint32_t idesc = kFp8 ? umma_idesc_f16(128, D, 0, 1) : umma_idesc_bf16(128, D, 0, 1);
                const uint32_t v_s = sm_base + C::kOffV;
                bool ok = true;
#pragma unroll 1
                for (int i = 0; i < count && ok && !warp_flag(s_abort); ++i) {
                    const int nkt = pieces[i].nkt;
                    const bool two = !kFp8 && pieces[i].ntok > p.tpt;
#pragma unroll 1
                    for (int t = 0; t < nkt; ++t, ++kv_it) {
                        const int st = kv_it & 1;
                        if (!mbar_wait_warp(&v_full[st], (kv_it >> 1) & 1, p.err)) { ok = false; break; }
#pragma unroll 1
                        for (int k = two ? 0 : st; k < (two ? 2 : st + 1); ++k) {
                            const bool first = two ? t == 0 : t < 2;
                            const uint32_t done = k ? nl1 : nl0, units = k ? uo1 : uo0;
                            if (two && k == 1 && !__all_sync(0xffffffffu, wait_counter(s_next0, (int)kv_it + 1, p.err))) { ok = false; break; }
                            const uint64_t b_desc = umma_desc_sw128(v_s + st * C::kTileBytes, C::kChunkBytes, 1024);
#pragma unroll 1
                            for (int hh = 0; hh < 2 && ok; ++hh) {
                                if (!mbar_wait_warp((hh ? p_full : p_half) + k, done & 1, p.err)) { ok = false; break; }
                                // a unit's first product overwrites O_k: the unit before must have been read
                                if (hh == 0 && first && units > 0 && !mbar_wait_warp(&o_free[k], (units - 1) & 1, p.err)) {
                                    ok = false;
                                    break;
                                }
                                tc_fence_after();
#pragma unroll
                                for (int kq = 0; kq < kKeys / 32; ++kq) {
                                    const int at = hh * (kKeys / 32) + kq;  // the 16 keys
                                    const uint32_t a = tbase + C::kColS + k * 128 + (kFp8 ? at * 8 : at / 2 * 32 + at % 2 * 8);
                                    umma_bf16_ts_w(tbase + C::kColO + k * D, a, b_desc + at * (2048 / 16), idesc,
                                                   (!first || hh > 0 || kq > 0) ? 1u : 0u);
                                    if constexpr (!kFp8)
                                        umma_bf16_ts_w(tbase + C::kColO + k * D, a + 16, b_desc + at * (2048 / 16), idesc, 1u);
                                }
                            }
                            if (!ok) break;
                            umma_commit_w(&pv_done[k]);
                            if (k) ++nl1;
                            else ++nl0;
                        }
                        if (!ok) break;
                        umma_commit_w(&v_empty[st]);
                    }
                    const int only = two || nkt > 1 ? -1 : (int)((kv_it - 1) & 1);  // the one lane that had a key tile
                    if (only != 1) ++uo0;
                    if (only != 0) ++uo1;
                }
                if (!ok) s_abort = 1;
                if (nl0 > 0) mbar_wait_warp(&pv_done[0], (nl0 - 1) & 1, p.err);
                if (nl1 > 0) mbar_wait_warp(&pv_done[1], (nl1 - 1) & 1, p.err);
            }
            __syncwarp();
            setmaxnreg_inc<C::kRegsLaunch>();
        } else if (kFp8 && warp >= 12) {
            setmaxnreg_dec<C::kRegsWiden>();
            __syncthreads();
            // ------------------------------------------------------------ rows to 8 bits, V's codes to f16
            // S comes from the codes of K themselves: a row of q, times the power of two that
            // brings its largest magnitude to 224 .. 448, is split into two E4M3 numbers, which
            // hold its 8 significant bits exactly down to 2^-10 of the largest and 2^-18 of that
            // below. V's codes are widened to f16 (exact), P is f16 in units of 2^-7, so that it
            // keeps 11 bits down to 2^-21 and goes on to 2^-31 of the row's largest. (With V and K
            // both widened to bf16 a tile took 5300 cycles, by integer operations 7000.) Value rows
            // outside the segment's keys may hold anything: zeros.
            const int wtid = tid - 384;
            bool ok = true;
            const int part = lane & 7;
            // A thread widens 16 codes of every 16th row; of their two 16-byte pieces the threads of a
            // row's second 64 elements store the second one first: a quarter warp's stores use all banks.
            const uint32_t own_row = wtid >> 3, far = part >> 2, own_code = sw128(own_row, part);
            const uint32_t own_value[2] = {far * C::kChunkBytes + sw128(own_row, 2 * (part & 3) + far),
                                           far * C::kChunkBytes + sw128(own_row, 2 * (part & 3) + (far ^ 1))};
            // rows r0 .. r0 + 31 of a piece's row tile, 8 lanes to a row, 16 elements to a lane
            auto load_rows = [&](const Piece& U, int r0, uint4 (&x)[2][2]) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int row = min(r0 + 16 * j + (wtid >> 3), U.ntok * p.G - 1), tok = row / p.G;
                    const uint4* from = reinterpret_cast<const uint4*>(
                        p.q + ((int64_t)(U.q0 + tok) * p.Hq + U.h * p.G + (row - tok * p.G)) * D) + 2 * part;
                    x[j][0] = __ldg(from);
                    x[j][1] = __ldg(from + 1);
                }
            };
            auto split_rows = [&](const Piece& U, uint4 (&x)[2][2]) {  // (the first 32 are loaded)
                const uint32_t n = q_it / C::kRowTiles;
                if (n > 0 && !mbar_wait_warp(&q_empty[q_it % C::kRowTiles], (n - 1) & 1, p.err)) {
                    ok = false;
                    return;
                }
                const uint32_t to = sm_base + C::kOffQ + q_it % C::kRowTiles * C::kTileBytes;
                const int rows = U.ntok * p.G;
#pragma unroll 1
                for (int r0 = 0; r0 < rows; r0 += 32) {
                    if (r0 > 0) load_rows(U, r0, x);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int row = r0 + 16 * j + (wtid >> 3);
                        const uint32_t w[8] = {x[j][0].x, x[j][0].y, x[j][0].z, x[j][0].w, x[j][1].x, x[j][1].y, x[j][1].z, x[j][1].w};
                        float top = 0.f, odd = 0.f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            top = fmax3f(top, fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e])));
                            odd += bf16_lo(w[e]) * 0.f + bf16_hi(w[e]) * 0.f;  // (NaN where an element is not finite)
                        }
#pragma unroll
                        for (int o = 1; o < 8; o <<= 1) {
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                            odd += __shfl_xor_sync(0xffffffffu, odd, o);
                        }
                        // top <= 0.875 * 2^e2: 448 at most after the product
                        const int e2 = min(129, max((int)(__float_as_uint(top) >> 23) - 126 +
                                                        ((__float_as_uint(top) & 0x7fffffu) > 0x600000u), -110));
                        const float by = exp2i(9 - e2);
                        uint32_t hi[4], low[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float v0 = bf16_lo(w[2 * e]) * by, v1 = bf16_hi(w[2 * e]) * by;
                            const float v2 = bf16_lo(w[2 * e + 1]) * by, v3 = bf16_hi(w[2 * e + 1]) * by;
                            hi[e] = e4m3x4(v0, v1, v2, v3);
                            const uint32_t h01 = e4m3x2_to_f16x2(hi[e] & 0xffffu), h23 = e4m3x2_to_f16x2(hi[e] >> 16);
                            const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h01));
                            const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h23));
                            low[e] = e4m3x4(v0 - a.x, v1 - a.y, v2 - b.x, v3 - b.y);
                        }
                        if (row < rows) {
#pragma unroll
                            for (int copy = 0; copy < 2; ++copy) {
                                const int at = row + 64 * copy;
                                if (copy && U.ntok > p.tpt / 2) continue;
                                st_shared4(to + sw128(at, part), hi[0], hi[1], hi[2], hi[3]);
                                st_shared4(to + C::kCodeBytes + sw128(at, part), low[0], low[1], low[2], low[3]);
                                if (part == 0) row_unit[(q_it & 3) * 128 + at] = exp2i(e2 - 9) + odd;
                            }
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[q_it % C::kRowTiles]);
                ++q_it;
            };
            // A piece's rows are split before the values of the piece in front of it are widened: its S
            // products need not wait for those (the other way round 32 groups of 4 samples took 2 % longer).
            uint4 x[2][2];
            if (count > 0) load_rows(pieces[0], 0, x);
#pragma unroll 1
            for (int i = -1; i < count && ok && !warp_flag(s_abort); ++i) {
                if (i + 1 < count) {
                    split_rows(pieces[i + 1], x);
                    if (i + 2 < count) load_rows(pieces[i + 2], 0, x);
                }
                if (i < 0) continue;
                const Piece U = pieces[i];
#pragma unroll 1
                for (int t = 0; t < U.nkt && ok; ++t) {
                    const int st = (int)(kv_it & 1);
                    const uint32_t n = kv_it >> 1;
                    if (!mbar_wait_warp(&c_full[st], n & 1, p.err) ||
                        (n > 0 && !mbar_wait_warp(&v_empty[st], (n - 1) & 1, p.err))) {
                        ok = false;
                        break;
                    }
                    const int kb = U.kb0 + t * kKeys;
                    const uint32_t zlo = (uint32_t)max(0, U.c0 - kb), valid = (uint32_t)(min(kKeys, U.c1 - kb) - (int)zlo);
                    // (rows from `some` on are not seen by all of the piece's tokens)
                    const uint32_t some = kSeveral && U.ntok > 1 ? (uint32_t)max(0, U.pos0 + 1 - kb) : kKeys;
                    const uint32_t from = sm_base + C::kOffCode + st * C::kCodeBytes;
                    const uint32_t to = sm_base + C::kOffV + st * C::kTileBytes;
#pragma unroll 4
                    for (int j = 0; j < kKeys / 16; ++j) {  // 16 rows, whose places are 2 KB further on each
                        const uint4 x = lds128(from + own_code + j * 2048);
                        const uint32_t w[4] = {far ? x.z : x.x, far ? x.w : x.y, far ? x.x : x.z, far ? x.y : x.w};
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh)
                            st_shared4(to + own_value[hh] + j * 2048, e4m3x2_to_f16x2(w[2 * hh] & 0xffffu),
                                       e4m3x2_to_f16x2(w[2 * hh] >> 16), e4m3x2_to_f16x2(w[2 * hh + 1] & 0xffffu),
                                       e4m3x2_to_f16x2(w[2 * hh + 1] >> 16));
                    }
                    if (valid < kKeys) {  // (a thread has the same places as above)
#pragma unroll 1
                        for (int j = 0; j < kKeys / 16; ++j) {
                            if (own_row + 16 * j - zlo < valid) continue;
                            st_shared4(to + own_value[0] + j * 2048, 0, 0, 0, 0);
                            st_shared4(to + own_value[1] + j * 2048, 0, 0, 0, 0);
                        }
                    }
                    if (kSeveral && some < kKeys) {
#pragma unroll 1
                        for (int j = wtid; j < kKeys * 8; j += 128) {
                            const uint32_t row = j >> 3, c = j & 7;
                            if (row < some) continue;
#pragma unroll 1
                            for (int hh = 0; hh < 2; ++hh) {
                                const uint32_t at = to + (c >> 2) * C::kChunkBytes + sw128(row, 2 * (c & 3) + hh);
                                const uint4 x = lds128(at);
                                uint32_t w[4] = {x.x, x.y, x.z, x.w};
                                if (!take_out<0x7c00u>(w)) continue;
                                st_shared4(at, w[0], w[1], w[2], w[3]);
                                atomicOr(&s_odd[i >> 5], 1u << (i & 31));
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&v_full[st]);
                        mbar_arrive(&c_empty[st]);
                    }
                    ++kv_it;
                }
            }
            if (!ok) s_abort = 1;
            __syncwarp();
            setmaxnreg_inc<C::kRegsLaunch>();
        } else {
            setmaxnreg_inc<C::kRegsSoftmax>();
            __syncthreads();
            // ------------------------------------------------------------ softmax lanes
            const int k = warp >= 8 ? 1 : 0;
            const int row = 32 * (warp & 3) + lane;  // of the row tile = tensor memory lane
            const int row_tok0 = row / p.G, row_tok64 = (row & 63) / p.G;
            const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
            const int wg_tid = tid - 128 * (k + 1);
            const uint32_t tS = tbase + lane_off + C::kColS + k * 128;
            const uint32_t tO = tbase + lane_off + C::kColO + k * D;
            float sl2 = p.scale_log2;
            constexpr float kUnitP = kFp8 ? 7.f : 0.f;  // log2 of what P is multiplied by
#pragma unroll 1
            for (int i = 0; i < count && !warp_flag(s_abort); ++i) {
                const Piece U = pieces[i];
                const bool two = !kFp8 && U.ntok > p.tpt;
                // Up to 64 rows lie in the row tile twice, and lane 1 takes the second copy: the two
                // lanes' exponentials are then on different quarters of the SM.
                const int shift = !two && U.ntok <= p.tpt / 2 && k == 1 ? 64 : 0;
                const int row_tok = shift ? row_tok64 : row_tok0;
                const int tok = (two ? k * p.tpt : 0) + row_tok;  // of the unit
                const bool write = row >= shift && row_tok < p.tpt && tok < U.ntok;
                const bool common = U.row < 0;
                const uint32_t kv_base = kv_it, piece = n_p++;
                kv_it += U.nkt;
                const int step = two ? 1 : 2, t_first = two ? 0 : (k ^ (int)(kv_base & 1));
                if (t_first >= U.nkt) continue;  // no key tile for this lane (and the join reads no result of it)
                // a lane's half of the result: its row tile's, or that of the piece's first or second key tile on
                const int half = min(p.tpt, U.ntok) * p.G;
                const int at = (two ? k : t_first) * half + row - shift;
                const int64_t row0 = U.row & INT32_MAX;
                float* po = (common ? p.po_pre : p.po_own) + row0 * D + at * 4;
                float* pl = (common ? p.pl_pre : p.pl_own) + row0 + at;
                // warps with rows that are a token's; the others only keep the lane's step
                const int busy = (min(p.tpt, U.ntok - (two ? k * p.tpt : 0)) * p.G + 31) / 32;
                const bool idle = (uint32_t)((warp & 3) - shift / 32) >= (uint32_t)busy;
                const int c1 = min(U.c1, U.pos0 + tok + 1);  // the row's visible keys end here
                const int all1 = min(U.c1, U.pos0 + 1);      // every row sees these
                float m_used = -INFINITY, l = 0.f;
                bool ok = true;
#pragma unroll 1
                for (int t = t_first; t < U.nkt; t += step) {
                    if (!mbar_wait_warp(&s_full[k], n_s & 1, p.err)) { ok = false; break; }
                    tc_fence_after();
                    if (kFp8 && t == t_first) {
                        sl2 = p.scale_log2 * row_unit[(piece & 3) * 128 + row];
                        if (sl2 < FLT_MIN) sl2 = FLT_MIN;  // (a masked score times 0 is NaN; these scores are below 2^-99 either way)
                    }
                    const int kb = U.kb0 + t * kKeys;
                    const bool edge = kb < U.c0 || kb + kKeys > all1;
                    float ls[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                    bool rescale = false;
                    float alpha = 1.f;
                    float mx[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) mx[j] = -INFINITY;
                    float m_off = 0.f;
                    auto take_max = [&] {
                        const float top = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                                fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * sl2;
                        if (t == t_first) {
                            m_used = top;
                        } else if (top > m_used + 8.f) {  // else the older maximum stays: P is at most 2^8
                            alpha = fast_exp2(m_used - top);
                            rescale = true;
                            l *= alpha;
                            m_used = top;
                        }
                        m_off = m_used == -INFINITY ? 0.f : m_used;
                    };
                    // P of 32 keys in place of their scores: the pairs of bf16 and what these leave, in all 32
                    // columns, or pairs of f16, in 16 of columns 0 .. 63
                    auto store32 = [&](const uint32_t (&r)[32], int at) {
                        uint32_t pk[32];
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            float x0, x1;
                            fma2_bcast(x0, x1, __uint_as_float(r[j]), __uint_as_float(r[j + 1]), sl2, kUnitP - m_off);
                            const float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
                            const int q = (j >> 1) & 3;
                            add2(ls[2 * q], ls[2 * q + 1], e0, e1);
                            if constexpr (kFp8) pk[j / 2] = pack_f16(e0, e1);
                            else split_weights(e0, e1, pk[j / 2], pk[16 + j / 2]);
                        }
                        if constexpr (kFp8) tmem_st16(tS + (at >> 1), *reinterpret_cast<const uint32_t(*)[16]>(pk));
                        else tmem_st32(tS + at, pk);
                    };
                    auto max32 = [&](const uint32_t (&r)[32]) {
#pragma unroll
                        for (int j = 0; j < 32; j += 2)
                            mx[(j >> 1) & 7] = fmax3f(mx[(j >> 1) & 7], __uint_as_float(r[j]), __uint_as_float(r[j + 1]));
                    };
                    bool early = false;  // (stays so in edge tiles, whose value rows are cleared first)
                    auto signal_half = [&] {  // the product over keys 0..63 may start
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&p_half[k]);
                    };
                    if (idle) {
                        early = !edge;
                        if (early) signal_half();
                    } else if (!edge) {
                        // twice over the row, 32 scores at a time (64 at a time 24 groups of 8 beams took 3 us more, with
                        // the whole row in registers 16: the code is fetched anew at each change between full and edge tiles)
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t r[32];
                            tmem_ld32(tS + 32 * c, r);
                            tmem_wait_ld();
                            max32(r);
                        }
                        take_max();
                        early = !__any_sync(0xffffffffu, rescale);
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t r[32];
                            tmem_ld32(tS + 32 * c, r);
                            tmem_wait_ld();
                            store32(r, 32 * c);
                            if (c == 1 && early) signal_half();
                        }
                    } else {
                        // the same in one loop body, few instructions, which edge tiles wait for more than for
                        // anything else (all tiles this way cost 24 groups of 8 beams 15 us more). Chunks that no
                        // row of the warp sees are left out, and only those that not every row sees in full
                        // are masked.
                        const int vlo = U.c0 - kb, vhi = max(vlo, c1 - kb);  // visible columns [vlo, vhi)
#pragma unroll 1
                        for (int c = 0; c < 8; ++c) {
                            const int at = 32 * (c & 3), a = min(32, max(0, vlo - at)), b = min(32, max(0, vhi - at));
                            const uint32_t bits = (uint32_t)((1ull << b) - (1ull << a));  // (a <= b)
                            if (c == 4) take_max();
                            if (!__any_sync(0xffffffffu, bits != 0)) {
                                if (c >= 4) tmem_st16_zero(tS + (kFp8 ? at >> 1 : at));
                                if (!kFp8 && c >= 4) tmem_st16_zero(tS + at + 16);
                                continue;
                            }
                            uint32_t r[32];
                            tmem_ld32(tS + at, r);
                            tmem_wait_ld();
                            if (!__all_sync(0xffffffffu, bits == 0xffffffffu)) {
#pragma unroll
                                for (int j = 0; j < 32; ++j) r[j] = (bits >> j) & 1 ? r[j] : 0xff800000u;
                            }
                            if (c < 4) max32(r);
                            else store32(r, at);
                        }
                    }
                    l += ((ls[0] + ls[1]) + (ls[2] + ls[3])) + ((ls[4] + ls[5]) + (ls[6] + ls[7]));
                    // (whole warps: tcgen05.ld and .st are collective)
                    if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t r[16];
                            tmem_ld16(tO + c * 16, r);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * alpha);
                            tmem_st16(tO + c * 16, r);
                        }
                    }
                    tmem_wait_st();
                    // value rows outside the segment's keys may hold anything: zeros, by the warps
                    // without rows if there are any. With two row tiles lane 0 does it (lane 1's
                    // product of a tile follows lane 0's).
                    // Of the rows from `some` on, which not all tokens see, what is not finite is taken
                    // out too (its weight of zero would not keep it from the others) and given back
                    // at the end to those that see it.
                    const int zlo = max(0, U.c0 - kb), zhi = min(kKeys, U.c1 - kb);
                    const int some = kSeveral && U.ntok > 1 ? max(zlo, min(all1 - kb, zhi)) : zhi;
                    if (!kFp8 && edge && (zlo > 0 || some < kKeys) && (k == 0 || !two) && (idle || busy == 4)) {
                        const uint32_t vi = kv_base + t;
                        if (!mbar_wait_warp(&v_full[vi & 1], (vi >> 1) & 1, p.err)) { ok = false; break; }
                        uint8_t* vt = smem + C::kOffV + (vi & 1) * C::kTileBytes;
                        const int skip = busy == 4 ? 0 : 32 * busy;  // (threads of the lane that have rows)
                        const int first = wg_tid - ((warp & 3) >= shift / 32 ? skip : 0);
#pragma unroll 1
                        for (int ci = first; ci < (zlo + kKeys - zhi) * (D / 8); ci += 128 - skip) {
                            const int z = ci / (D / 8), c = ci % (D / 8), vr = z < zlo ? z : zhi + z - zlo;
                            *reinterpret_cast<uint4*>(vt + (c >> 3) * C::kChunkBytes + sw128(vr, c & 7)) = make_uint4(0, 0, 0, 0);
                        }
#pragma unroll 1
                        for (int ci = first; kSeveral && ci < (zhi - some) * (D / 8); ci += 128 - skip) {
                            const int c = ci % (D / 8);
                            uint4* at = reinterpret_cast<uint4*>(vt + (c >> 3) * C::kChunkBytes + sw128(some + ci / (D / 8), c & 7));
                            uint32_t w[4] = {at->x, at->y, at->z, at->w};
                            if (!take_out<0x7f80u>(w)) continue;
                            *at = make_uint4(w[0], w[1], w[2], w[3]);
                            atomicOr(&s_odd[i >> 5], 1u << (i & 31));
                        }
                        fence_proxy_async_smem();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (!early) mbar_arrive(&p_half[k]);
                        mbar_arrive(&p_full[k]);
                    }
                    ++n_s;
                }
                if (ok) ok = mbar_wait_warp(&pv_done[k], (n_s - 1) & 1, p.err);
                if (!ok) {
                    s_abort = 1;
                    break;
                }
                // -------- the piece: O / l and log2 of the sum
                tc_fence_after();
                const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
                for (int c = 0; c < (idle ? 0 : D / 32); ++c) {
                    uint32_t r[32];
                    tmem_ld32(tO + c * 32, r);
                    tmem_wait_ld();
                    if (write) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            reinterpret_cast<float4*>(po)[(int64_t)(c * 8 + j) * 2 * half] =
                                make_float4(__uint_as_float(r[4 * j]) * inv, __uint_as_float(r[4 * j + 1]) * inv,
                                            __uint_as_float(r[4 * j + 2]) * inv, __uint_as_float(r[4 * j + 3]) * inv);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&o_free[k]);
                if (write) *pl = m_used + log2f(l) - kUnitP;
                if (kSeveral && write && (*const_cast<volatile uint32_t*>(&s_odd[i >> 5]) >> (i & 31) & 1)) {
                    // what was taken out of this lane's key tiles and the row sees
                    const int end = min(c1, U.kb0 + U.nkt * kKeys);
#pragma unroll 1
                    for (int pos = max(max(U.c0, U.kb0), all1); pos < end; ++pos) {
                        if (!two && ((((pos - U.kb0) / kKeys) ^ t_first) & 1)) continue;
                        int block = __ldg(p.block_table + (int64_t)U.table * p.max_blocks + (pos >> p.bs_log2));
                        if (block < 0 || block >= p.num_blocks) block = 0;
                        const int64_t from = ((((int64_t)block * p.Hkv + U.h) << p.bs_log2) + (pos & (p.bs - 1))) * D;
#pragma unroll 1
                        for (int d = 0; d < D; ++d) {
                            float x;
                            if constexpr (kFp8) x = (static_cast<const uint8_t*>(p.v_cache)[from + d] & 0x7fu) == 0x7fu ? NAN : 0.f;
                            else x = __uint_as_float((uint32_t)static_cast<const uint16_t*>(p.v_cache)[from + d] << 16);
                            if (!(fabsf(x) < INFINITY)) po[(int64_t)(d / 4) * 8 * half + d % 4] += x;
                        }
                    }
                }
            }
            __syncwarp();
            setmaxnreg_dec<C::kRegsLaunch>();
        }
        __syncthreads();
        if (s_abort) break;
        if (tid == 0) s_pieces = 0;
        if (tid < kPieces / 32) s_odd[tid] = 0;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tbase, C::kTmemCols);
    }
}

// ---------------------------------------------------------------- the join
// One CTA per token and kv head. Its pieces are those of its rows' two units (the
// group's common keys, its request's own) in every CTA whose share has tiles of them.
struct Source {
    const float* o;  // the row's first four values of the group's first head; the next four dims' 8 * half further on
    const float* l;  // null: no piece
};

template <int D, int kThreads>
__global__ void __launch_bounds__(kThreads) prefix_join_kernel(const PrefixParams p, int ncta) {
    constexpr int kWarps = kThreads / 32;
    extern __shared__ __align__(16) uint8_t s_join[];
    __shared__ float s_inv[16];
    Source* src = reinterpret_cast<Source*>(s_join);                    // [4 * ncta]
    float* weight = reinterpret_cast<float*>(src + 4 * (size_t)ncta);  // [4 * ncta][G]
    // (no early launch of what follows: its CTAs, waiting, could take the SMs of those still to come)
    const int t = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = p.G;
    // ---- the token's segments, from the lengths (in place since before the attention started)
    const TokenPlace at = place_of(p.qsl, p.seq_lens, p.B, t);
    int g = 0, group_n = p.groups;
#pragma unroll 1
    while (group_n > 1) {  // the last group that starts at or before the request, 32 places at a time
        const int step = (group_n + 31) / 32, i = g + lane * step;
        const uint32_t before = __ballot_sync(0xffffffffu, i < g + group_n && __ldg(p.starts + i) <= max(at.r, 0));
        const int k = before ? 31 - __clz(before) : 0;
        group_n = min(step, group_n - k * step);
        g += k * step;
    }
    const int r0 = __ldg(p.starts + g), r1 = __ldg(p.starts + g + 1);
    const int common = common_keys(r0, r1, __ldg(p.prefix + g));
    const bool inside = r0 >= 0 && r1 >= r0 && r1 <= p.B;
    const int gq0 = inside ? __ldg(p.qsl + r0) : 0, gq1 = inside ? __ldg(p.qsl + r1) : 0;
    const Seg seg[2] = {make_seg(p, gq0, gq1 - gq0, 0, common), make_seg(p, at.q0, at.q1 - at.q0, common, at.len)};
    int n = 0, n_common = 0;  // pieces, in the order of their keys
    int half_common = 0, half_own = 0;  // rows of half a result
    // With few CTAs, which wait for the attention's end anyway, the steps up to the weights
    // are run through once before it, over no pieces: their instructions are then at hand.
#pragma unroll 1
    for (int pass = kThreads == 512 ? 0 : 1; pass < 2; ++pass) {
        int total = ncta, cost_at[2] = {0, 0}, row_at[2] = {0, 0};
        if (pass == 1) {
            grid_dep_wait();
            total = __ldcg(p.seg_cost + p.own0 + p.B);
            cost_at[0] = __ldcg(p.seg_cost + g);
            row_at[0] = __ldcg(p.seg_row + g);
            cost_at[1] = __ldcg(p.seg_cost + p.own0 + max(at.r, 0));
            row_at[1] = __ldcg(p.seg_row + p.own0 + max(at.r, 0)) - __ldcg(p.seg_row + p.own0);
            if (total < 0 || at.r < 0) return;  // refused lengths, or a row behind the last request's: nothing is written
        }
        const Shares shares(total, ncta);
        n = 0;
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
            const Seg s = part == 0 ? seg[0] : seg[1];
            if (part == 1) n_common = n;
            if (s.nkt == 0) continue;
            int tok = t - s.q0, rt = 0;
            if (s.nrt > 1) {
                rt = tok / p.upt;
                tok -= rt * p.upt;
            }
            const int tokens = min(p.upt, s.n - rt * p.upt), half = min(p.tpt, tokens) * G;
            const bool two = tokens > p.tpt;
            const int us = (part == 0 ? cost_at[0] : cost_at[1]) + (h * s.nrt + rt) * unit_cost(s);
            const int before = (part == 0 ? row_at[0] : row_at[1]) + (h * s.n + rt * p.upt) * G;
            const int most = part == 0 ? p.most_pre : p.most_own;
            (part == 0 ? half_common : half_own) = half;
            const int row = two && tok >= p.tpt ? half + (tok - p.tpt) * G : tok * G;
            const int first = shares.cta_of(us + s.e), last = shares.cta_of(us + s.e + (s.nkt - 1) * s.w);
            const int lanes = two ? 1 : 2, end = s.c1 - s.n + min(s.n, (rt + 1) * p.upt);  // (of own keys)
            const float* o = part == 0 ? p.po_pre : p.po_own;
            const float* l = part == 0 ? p.pl_pre : p.pl_own;
#pragma unroll 1
            for (int j = tid; j < (last - first + 1) * lanes && pass == 1; j += kThreads) {
                const int c = first + (two ? j : j >> 1), k = two ? 0 : j & 1;
                const int t0 = first_tile(shares.start(c), us, s), t1 = first_tile(shares.start(c + 1), us, s);
                const int tiles = t0 >= t1 ? 0 : part == 0 ? t1 - t0 : seen_tiles(s, t0, t1, end);
                const int64_t row0 = 2 * (before + c * most);
                Source x;
                x.o = o + row0 * D + (k * half + row) * 4;
                x.l = tiles > k ? l + row0 + k * half + row : nullptr;
                src[n + j] = x;
            }
            n += (last - first + 1) * lanes;
        }
        if (pass == 0) n = n_common = 0;
        __syncthreads();
        // ---- weights: a warp per head
#pragma unroll 1
        for (int hh = warp; hh < G; hh += kWarps) {
            float top = -INFINITY, nan = 0.f;
#pragma unroll 1
            for (int i = lane; i < n; i += 32) {
                const float* from = src[i].l;
                const float l = from ? __ldcg(from + hh) : -INFINITY;
                weight[i * G + hh] = l;
                top = fmaxf(top, l);
                nan += l == l ? 0.f : l;
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                nan += __shfl_xor_sync(0xffffffffu, nan, o);
            }
            float sum = nan;
#pragma unroll 1
            for (int i = lane; i < n; i += 32) {
                const float l = weight[i * G + hh];
                const float w = l == -INFINITY ? 0.f : l == top ? 1.f : exp2f(l - top);
                weight[i * G + hh] = w;
                sum += w;
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0 && pass == 1) {
                s_inv[hh] = sum == 0.f ? 0.f : p.v_scale / sum;
                if (p.lse) p.lse[(int64_t)t * p.Hq + h * G + hh] = (top + log2f(sum)) * 0.69314718055994531f;
            }
        }
        __syncthreads();
    }
    // ---- the weighted sums: four dims of a head per thread, the pieces dealt out where threads are left over
    const int flats = D / 4 * G, deal = max(1, kThreads / flats);
    float4* parts = reinterpret_cast<float4*>(weight + (size_t)4 * ncta * G);  // [deal][flats], where deal > 1
#pragma unroll 1
    for (int f0 = tid; f0 < flats * deal; f0 += kThreads) {
        const int f = f0 % flats, part = f0 / flats, hh = f % G, d4 = f / G;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        const int at_common = d4 * 2 * half_common + hh, at_own = d4 * 2 * half_own + hh;
#pragma unroll 4
        for (int i = part; i < n; i += deal) {
            const float w = weight[i * G + hh];
            const float4 o = __ldcg(reinterpret_cast<const float4*>(src[i].o) + (i < n_common ? at_common : at_own));
            if (w != 0.f) {  // (the place of a piece that is none may hold anything)
                acc.x += w * o.x;
                acc.y += w * o.y;
                acc.z += w * o.z;
                acc.w += w * o.w;
            }
        }
        if (deal > 1) parts[f0] = acc;
        if (deal == 1) {
            const float inv = s_inv[hh];
            *reinterpret_cast<uint2*>(p.out + ((int64_t)t * p.Hq + h * G + hh) * D + d4 * 4) =
                make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
        }
    }
    if (deal == 1) return;
    __syncthreads();
#pragma unroll 1
    for (int f = tid; f < flats; f += kThreads) {
        const int hh = f % G, d4 = f / G;
        float4 acc = parts[f];
#pragma unroll 1
        for (int k = 1; k < deal; ++k) {
            const float4 o = parts[k * flats + f];
            acc.x += o.x;
            acc.y += o.y;
            acc.z += o.z;
            acc.w += o.w;
        }
        const float inv = s_inv[hh];
        *reinterpret_cast<uint2*>(p.out + ((int64_t)t * p.Hq + h * G + hh) * D + d4 * 4) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    }
}

template <int D, bool kFp8, bool kSeveral>
cudaError_t go_attn(const PrefixMaps& maps, const PrefixParams& p, int ncta, cudaStream_t stream) {
    using C = PxCfg<D, kFp8>;
    auto kern = prefix_attn_kernel<D, kFp8, kSeveral>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(ncta), dim3(C::kThreads), C::kSmem, stream, maps, p);
}

template <int D, int kThreads>
cudaError_t go_join(const PrefixParams& p, int ncta, cudaStream_t stream) {
    auto kern = prefix_join_kernel<D, kThreads>;
    const size_t head = sizeof(Source) + sizeof(float) * p.G;
    const int flats = D / 4 * p.G;
    const size_t smem = 4 * (size_t)ncta * head + (kThreads / flats > 1 ? sizeof(float4) * kThreads : 0);
    if (smem > 47 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
            (int)(4 * (size_t)ncta * (sizeof(Source) + sizeof(float) * 16) + sizeof(float4) * kThreads));
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(kern, dim3(p.T, p.Hkv), dim3(kThreads), smem, stream, p, ncta);
}

template <int D>
cudaError_t go_join_by_size(const PrefixParams& p, int ncta, cudaStream_t stream) {
    // few tokens: their units are cut into many pieces, and SMs are idle
    return (int64_t)p.T * p.Hkv <= 2 * ncta ? go_join<D, 512>(p, ncta, stream) : go_join<D, 128>(p, ncta, stream);
}

}  // namespace

cudaError_t launch_prefix_attn(const PrefixMaps& maps, const PrefixParams& p, int head_dim, bool fp8, int ncta,
                               cudaStream_t stream) {
    if (p.max_query > 1) {
        if (fp8) return go_attn<128, true, true>(maps, p, ncta, stream);
        return head_dim == 128 ? go_attn<128, false, true>(maps, p, ncta, stream)
                               : go_attn<64, false, true>(maps, p, ncta, stream);
    }
    if (fp8) return go_attn<128, true, false>(maps, p, ncta, stream);
    return head_dim == 128 ? go_attn<128, false, false>(maps, p, ncta, stream)
                           : go_attn<64, false, false>(maps, p, ncta, stream);
}

cudaError_t launch_prefix_join(const PrefixParams& p, int head_dim, int ncta, cudaStream_t stream) {
    return head_dim == 128 ? go_join_by_size<128>(p, ncta, stream) : go_join_by_size<64>(p, ncta, stream);
}

}  // namespace pka
