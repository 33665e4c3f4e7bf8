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
// table), two MMA-issuing threads, two softmax warpgroups ("lanes" 0 and 1, one
// thread per row). With two row tiles in a unit, lane k has row tile k and every
// key tile serves both; with one, the lanes take alternate key tiles of the same
// rows, so that one's exponentials overlap the other's products, and leave two
// pieces. Tensor memory: S_k (128 columns, P_k written over it in bf16) and O_k.
// P is rounded to bf16 for the product (the type of V, which the tensor cores ask
// for); its sum is kept from the unrounded values in 32 bits.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "params.cuh"
#include "plan.cuh"
#include "tcgen05.cuh"

namespace pka {

namespace {

constexpr int kKeys = 128;  // keys of a key tile
constexpr int kPieces = 256;  // pieces of a CTA's share that are listed at a time
constexpr int kMaxSegs = 2 * kMaxRequests;
constexpr int kChunks = kMaxSegs / 32;  // warp-sized runs of segments
// Cost of a key tile for one row tile and for two.
constexpr int kCostOne = 1, kCostTwo = 1;

using i64 = long long;

struct Seg {
    int q0, n;      // its tokens
    int c0, c1;     // its keys
    int base;       // the first key tile's first key
    int nkt, nrt;   // key tiles; units per kv head
    int w;          // cost of a key tile
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
    s.nrt = s.nkt > 0 ? (n + p.upt - 1) / p.upt : 0;
    s.w = n > p.tpt ? kCostTwo : kCostOne;
    return s;
}

// A group of one request has no common keys: they are its own.
PKA_DEVICE int common_keys(int r0, int r1, int prefix) { return r1 - r0 > 1 ? prefix : 0; }

// The last i in [0, n) with a[i] <= x (a[0] <= x).
PKA_DEVICE int last_at_most(const int32_t* a, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The CTA whose share holds position x of a line of length total.
PKA_DEVICE int cta_of(i64 x, i64 total, int ncta) { return (int)(((x + 1) * ncta - 1) / total); }
PKA_DEVICE i64 share_start(int cta, i64 total, int ncta) { return total * cta / ncta; }
// Key tiles [t0, t1) of a unit that starts at `us` lie in [lo, hi).
PKA_DEVICE int first_tile(i64 lo, i64 us, int w, int nkt) {
    const i64 d = lo - us;
    return d <= 0 ? 0 : (int)min((i64)nkt, (d + w - 1) / w);
}

struct Piece {
    int table;      // the request whose block table row is read
    int h;          // kv head
    int q0, ntok;   // the unit's tokens
    int kb0, nkt;   // first key of the first tile, key tiles
    int c0, c1;     // visible keys of the segment
    int pos0;       // position of token q0 (past everything for common keys)
    int slot;       // where its result goes; common keys: bit 31
};

template <int D, bool kFp8>
struct PxCfg {
    // Registers by role: the launch gives every thread the same.
    static constexpr int kThreads = kFp8 ? 512 : 384;
    static constexpr int kRegsLaunch = kFp8 ? 128 : 168, kRegsIssue = kFp8 ? 64 : 80;
    static constexpr int kRegsSoftmax = kFp8 ? 176 : 208, kRegsWiden = 96;
    static_assert(128 * kRegsIssue + 256 * kRegsSoftmax + (kFp8 ? 128 * kRegsWiden : 0) <= kThreads * kRegsLaunch,
                  "register split");
    static constexpr int kRowTiles = kFp8 ? 1 : 2;   // of a unit, at most
    static constexpr int kChunk = D / 64;            // 64-wide swizzle chunks per row
    static constexpr int kChunkBytes = 128 * 128;    // 128 rows x 128 B
    static constexpr int kTileBytes = kChunk * kChunkBytes;
    static constexpr int kCodeBytes = kFp8 ? kKeys * D : 0;  // a key tile's codes
    static constexpr int kCodeK = 2, kCodeV = 1;             // stages of codes
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kRowTiles * kTileBytes;  // two stages
    static constexpr int kOffV = kOffK + 2 * kTileBytes;  // two stages
    static constexpr int kOffCode = kOffV + 2 * kTileBytes;
    static constexpr int kOffPiece = kOffCode + (kCodeK + kCodeV) * kCodeBytes;
    static constexpr int kOffSums = kOffPiece + kPieces * (int)sizeof(Piece);
    static constexpr int kOffBar = kOffSums + (kChunks + 1) * 16;
    static constexpr int kSmem = kOffBar + 256 + 1024;
    static constexpr uint32_t kColS = 0, kColO = 256, kTmemCols = 512;
    static_assert(kSmem <= 232448, "shared memory");
    static_assert(4 * kTileBytes >= (int)sizeof(int32_t) * (2 * kMaxRequests + 1), "the groups pass through the K and V stages");
};

// The block of lane `b` of the key tile at kb (lanes past its valid blocks get 0).
PKA_DEVICE int tile_block(const PrefixParams& p, const int32_t* bt, int kb, int c1, int lane) {
    const int pos = kb + (lane << p.bs_log2);
    if (lane >= (kKeys >> p.bs_log2) || pos >= c1) return 0;
    int blk = __ldg(bt + (pos >> p.bs_log2));
    if (blk < 0 || blk >= p.num_blocks) {
        set_error(p.err, PKA_DEVERR_BLOCK_ID);
        blk = 0;
    }
    return blk;
}

// The line of all units: sums of costs and units before each run of 32 segments.
struct Plan {
    i64* cost;   // [runs + 1]
    int* units;  // [runs + 1]
    int runs;
    i64 total;
};

// Segment s from the lengths: the groups, then, from own0 on, the requests (own0
// is the number of groups, up to whole runs of 32). The groups' starts and prefixes
// lie in shared memory.
PKA_DEVICE Seg seg_of(const PrefixParams& p, const int32_t* starts, const int32_t* prefix, int s, int& err) {
    if (s < p.groups) {
        const int r0 = starts[s], r1 = starts[s + 1], len = prefix[s];
        if (r0 > r1 || r0 < 0 || r1 > p.B) {
            err |= PKA_DEVERR_INDEX;
            return make_seg(p, 0, 0, 0, 0);
        }
        if (len < 0) err |= PKA_DEVERR_SEQ_LEN;
        const int q0 = __ldg(p.qsl + r0), q1 = __ldg(p.qsl + r1);
        return make_seg(p, q0, q1 - q0, 0, common_keys(r0, r1, len));
    }
    if (s < p.own0) return make_seg(p, 0, 0, 0, 0);
    const int r = s - p.own0;
    const int q0 = __ldg(p.qsl + r), q1 = __ldg(p.qsl + r + 1), len = __ldg(p.seq_lens + r);
    if (q0 < 0 || q1 < q0 || q1 > p.T || (r == 0 && q0 != 0)) err |= PKA_DEVERR_QUERY_START_LOC;
    const int n = q1 - q0;
    if (n <= 0) return make_seg(p, q0, 0, 0, 0);
    if (n > p.max_query) err |= PKA_DEVERR_QUERY_LEN;
    if (len < n || len > p.max_seq) err |= PKA_DEVERR_SEQ_LEN;
    const int g = last_at_most(starts, p.groups, r);
    const int have = prefix[g];
    if (have < 0 || have > len - n) err |= PKA_DEVERR_SEQ_LEN;
    return make_seg(p, q0, n, common_keys(starts[g], starts[g + 1], have), len);
}

template <int D, bool kFp8>
__global__ void __launch_bounds__((PxCfg<D, kFp8>::kThreads), 1)
    prefix_attn_kernel(const __grid_constant__ PrefixMaps maps, const PrefixParams p) {
    using C = PxCfg<D, kFp8>;
    constexpr int kPxThreads = C::kThreads;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint64_t* q_full = bars + 0;    // the unit's row tiles landed
    uint64_t* q_empty = bars + 1;   // its last S product is done
    uint64_t* k_full = bars + 2;    // [2] per K stage
    uint64_t* k_empty = bars + 4;
    uint64_t* v_full = bars + 6;    // [2] per V stage
    uint64_t* v_empty = bars + 8;
    uint64_t* s_full = bars + 10;   // [2] per lane: its S tile is in tensor memory
    uint64_t* p_full = bars + 12;   // [2] its P is (4 warp arrivals)
    uint64_t* pv_done = bars + 14;  // [2] the product that read its P is done
    uint64_t* o_free = bars + 16;   // [2] its O has been read (4 warp arrivals)
    uint64_t* p_half = bars + 18;   // [2] P of keys 0..63 is there (4 warp arrivals)
    uint64_t* ck_full = bars + 20;  // [2] per stage of key codes: landed
    uint64_t* ck_empty = bars + 22;  // [2] widened (4 warp arrivals)
    uint64_t* cv_full = bars + 24;  // the same for value codes
    uint64_t* cv_empty = bars + 26;
    Piece* pieces = reinterpret_cast<Piece*>(smem + C::kOffPiece);
    i64* run_cost = reinterpret_cast<i64*>(smem + C::kOffSums);
    int* run_units = reinterpret_cast<int*>(run_cost + kChunks + 1);
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    // Key tiles after which lane 0's next S has been issued: with two row tiles,
    // lane 1's product lets that S go first.
    __shared__ volatile int s_next0;
    __shared__ int s_pieces;  // of the share, all

    grid_dep_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], kFp8 ? 4 : 1);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], kFp8 ? 4 : 1);
            mbar_init(&v_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&p_half[i], 4);
            mbar_init(&pv_done[i], 1);
            mbar_init(&o_free[i], 4);
            mbar_init(&ck_full[i], 1);
            mbar_init(&ck_empty[i], 4);
            mbar_init(&cv_full[i], 1);
            mbar_init(&cv_empty[i], 4);
        }
        fence_barrier_init();
        s_abort = 0;
        s_next0 = 0;
        tma_prefetch_desc(&maps.q);
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
    }
    // rows of a row tile that no token fills (128 / G * G < 128) stay zero
    for (int i = tid; i < C::kRowTiles * C::kTileBytes / 16; i += kPxThreads)
        reinterpret_cast<uint4*>(smem + C::kOffQ)[i] = make_uint4(0, 0, 0, 0);
    if (warp == 1) tmem_alloc(&s_tmem, C::kTmemCols);
    grid_dep_wait();

    // ---------------------------------------------------------------- the line
    const int segs = p.own0 + p.B, runs = (segs + 31) / 32;
    int32_t* starts = reinterpret_cast<int32_t*>(smem + C::kOffK);
    int32_t* prefix = starts + p.groups + 1;
    for (int i = tid; i <= p.groups; i += kPxThreads) starts[i] = p.starts[i];
    for (int i = tid; i < p.groups; i += kPxThreads) prefix[i] = p.prefix[i];
    __syncthreads();
    int err = 0;
    if (tid == 0 && (starts[0] != 0 || starts[p.groups] != p.B)) err = PKA_DEVERR_INDEX;
    for (int run = warp; run < runs; run += kPxThreads / 32) {
        const int s = run * 32 + lane;
        i64 cost = 0;
        int units = 0;
        if (s < segs) {
            const Seg g = seg_of(p, starts, prefix, s, err);
            units = g.nrt * p.Hkv;
            cost = (i64)units * g.nkt * g.w;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            cost += __shfl_xor_sync(0xffffffffu, cost, o);
            units += __shfl_xor_sync(0xffffffffu, units, o);
        }
        if (lane == 0) {
            run_cost[run] = cost;
            run_units[run] = units;
        }
    }
    const int bad = __syncthreads_or(err);
    if (bad) {  // the same for every CTA
        if (blockIdx.x == 0) {
            if (err) set_error(p.err, err);
            if (tid == 0) p.seg_cost[segs] = -1;
        }
    } else if (warp == 0) {
        i64 c0 = 0;
        int u0 = 0;
        for (int r0 = 0; r0 < runs; r0 += 32) {
            const int r = r0 + lane;
            const i64 c = r < runs ? run_cost[r] : 0;
            const int u = r < runs ? run_units[r] : 0;
            i64 ci = c;
            int ui = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const i64 a = __shfl_up_sync(0xffffffffu, ci, o);
                const int b = __shfl_up_sync(0xffffffffu, ui, o);
                if (lane >= o) {
                    ci += a;
                    ui += b;
                }
            }
            if (r < runs) {
                run_cost[r] = c0 + ci - c;
                run_units[r] = u0 + ui - u;
            }
            c0 += __shfl_sync(0xffffffffu, ci, 31);
            u0 += __shfl_sync(0xffffffffu, ui, 31);
        }
        if (lane == 0) {
            run_cost[runs] = c0;
            run_units[runs] = u0;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = s_tmem;
    const uint32_t sm_base = smem_u32(smem);
    const int ncta = gridDim.x, cta = blockIdx.x;
    const i64 total = bad ? 0 : run_cost[runs];
    const i64 lo = share_start(cta, total, ncta), hi = share_start(cta + 1, total, ncta);

    // state of the roles across lists
    uint32_t kv_it = 0, q_it = 0;
    uint32_t last[2] = {0, 0};  // phase + 1 of the last copy per stage (0 = none)
    uint32_t nl[2] = {0, 0};    // S products (or P . V products) of each lane
    uint32_t n_s = 0;           // S tiles of this softmax lane
    uint32_t uo[2] = {0, 0};    // units in which each lane had key tiles

    for (int listed = 0;; listed += kPieces) {
        // ------------------------------------------------------------ a list of the share's pieces
        if (listed > 0) {  // (the groups were overwritten by tiles)
            for (int i = tid; i <= p.groups; i += kPxThreads) starts[i] = p.starts[i];
            for (int i = tid; i < p.groups; i += kPxThreads) prefix[i] = p.prefix[i];
            __syncthreads();
        }
        if (warp == 0) {
            int found = 0;
            if (hi > lo) {
                int run = 0;
                for (int r0 = 0; r0 < runs; r0 += 32) {  // the last run that starts at or before lo
                    const uint32_t before = __ballot_sync(0xffffffffu, r0 + lane < runs && run_cost[r0 + lane] <= lo);
                    if (before) run = r0 + 31 - __clz(before);
                    if (before != 0xffffffffu) break;
                }
                for (; run < runs && run_cost[run] < hi; ++run) {
                    const int s = run * 32 + lane;
                    int none = 0;
                    const Seg g = s < segs ? seg_of(p, starts, prefix, s, none) : make_seg(p, 0, 0, 0, 0);
                    const int units = g.nrt * p.Hkv;
                    const i64 unit_cost = (i64)g.nkt * g.w, cost = units * unit_cost;
                    i64 ci = cost;
                    int ui = units;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const i64 a = __shfl_up_sync(0xffffffffu, ci, o);
                        const int b = __shfl_up_sync(0xffffffffu, ui, o);
                        if (lane >= o) {
                            ci += a;
                            ui += b;
                        }
                    }
                    const i64 cs = run_cost[run] + ci - cost;
                    const int us0 = run_units[run] + ui - units;
                    int first = 0, end = 0;  // units that may have tiles in the share
                    if (units > 0 && cs < hi && cs + cost > lo) {
                        first = cs >= lo ? 0 : (int)((lo - cs) / unit_cost);
                        end = (int)min((i64)units, (hi - cs + unit_cost - 1) / unit_cost);
                    }
                    int mine = 0;
                    for (int u = first; u < end; ++u) {
                        const i64 at = cs + u * unit_cost;
                        mine += first_tile(lo, at, g.w, g.nkt) < first_tile(hi, at, g.w, g.nkt);
                    }
                    int before = mine;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int a = __shfl_up_sync(0xffffffffu, before, o);
                        if (lane >= o) before += a;
                    }
                    const int sum = __shfl_sync(0xffffffffu, before, 31);
                    int to = found + before - mine - listed;
                    found += sum;
                    for (int u = first; u < end && to < kPieces; ++u) {
                        const i64 at = cs + u * unit_cost;
                        const int t0 = first_tile(lo, at, g.w, g.nkt), t1 = first_tile(hi, at, g.w, g.nkt);
                        if (t0 >= t1) continue;
                        if (to >= 0) {
                            Piece x;
                            const int rt = u % g.nrt;
                            x.h = u / g.nrt;
                            x.q0 = g.q0 + rt * p.upt;
                            x.ntok = min(p.upt, g.n - rt * p.upt);
                            x.kb0 = g.base + t0 * kKeys;
                            x.c0 = g.c0;
                            x.c1 = g.c1;
                            x.nkt = t1 - t0;
                            if (s < p.groups) {
                                int r = starts[s];
                                while (r + 1 < starts[s + 1] && __ldg(p.qsl + r + 1) <= g.q0) ++r;
                                x.table = r;
                                x.pos0 = INT32_MAX / 2;
                                x.slot = (us0 + u + cta) | INT32_MIN;
                            } else {
                                x.table = s - p.own0;
                                x.pos0 = g.c1 - g.n + (x.q0 - g.q0);
                                // key tiles behind the last token's position have nothing to see; one is kept
                                const int seen = (min(g.c1, x.pos0 + x.ntok) - x.kb0 + kKeys - 1) / kKeys;
                                x.nkt = max(1, min(x.nkt, seen));
                                x.slot = us0 + u + cta - run_units[p.own0 / 32];
                            }
                            pieces[to] = x;
                        }
                        ++to;
                    }
                }
            }
            if (lane == 0) s_pieces = found;
        } else if (warp == 11 && listed == 0 && !bad) {
            // the segments' places on the line, for the join
            for (int run = cta; run < runs; run += ncta) {
                const int s = run * 32 + lane;
                int none = 0;
                const Seg g = s < segs ? seg_of(p, starts, prefix, s, none) : make_seg(p, 0, 0, 0, 0);
                const int units = g.nrt * p.Hkv;
                const i64 cost = (i64)units * g.nkt * g.w;
                i64 ci = cost;
                int ui = units;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const i64 a = __shfl_up_sync(0xffffffffu, ci, o);
                    const int b = __shfl_up_sync(0xffffffffu, ui, o);
                    if (lane >= o) {
                        ci += a;
                        ui += b;
                    }
                }
                if (s < segs) {
                    p.seg_cost[s] = run_cost[run] + ci - cost;
                    p.seg_unit[s] = run_units[run] + ui - units;
                }
            }
            if (cta == 0 && lane == 0) p.seg_cost[segs] = total;
        }
        fence_proxy_async_smem();  // (what was written where tiles go)
        __syncthreads();
        const int count = min(kPieces, s_pieces - listed);
        if (count <= 0) break;

        if (warp < 4) {
            setmaxnreg_dec<C::kRegsIssue>();
            if (warp == 0 || warp == 2) {
                // -------------------------------------------------------- producers: K; V and Q
                const int which = warp == 0 ? 0 : 1;
                const uint64_t pol = policy_evict_normal(), pol_q = policy_evict_last();
                const bool tma = p.bs >= 8;
                // over an 8-bit cache the codes' stages, else the tiles'
                uint64_t* fulls = kFp8 ? (which ? cv_full : ck_full) : which ? v_full : k_full;
                uint64_t* empties = kFp8 ? (which ? cv_empty : ck_empty) : which ? v_empty : k_empty;
                const uint32_t nst = !kFp8 ? 2 : which ? C::kCodeV : C::kCodeK;
                uint8_t* stages = smem + (kFp8 ? C::kOffCode + (which ? C::kCodeK * C::kCodeBytes : 0)
                                               : which ? C::kOffV : C::kOffK);
                constexpr int kStage = kFp8 ? C::kCodeBytes : C::kTileBytes;
                constexpr int kBoxes = kFp8 ? 1 : C::kChunk;  // 128 bytes wide
                bool ok = true;
                for (int i = 0; i < count && ok && !warp_flag(s_abort); ++i, ++q_it) {
                    const Piece U = pieces[i];
                    if (which == 1) {
                        if (q_it > 0 && !mbar_wait_warp(q_empty, (q_it - 1) & 1, p.err)) {
                            s_abort = 1;
                            break;
                        }
                        if (lane == 0) {
                            const int nq = !kFp8 && U.ntok > p.tpt ? 2 : 1, bytes = p.tpt * p.G * 128;
                            mbar_arrive_expect_tx(q_full, (uint32_t)(nq * C::kChunk * bytes));
                            for (int k = 0; k < nq; ++k)
                                for (int c = 0; c < C::kChunk; ++c)
                                    tma_load_3d(smem + C::kOffQ + k * C::kTileBytes + c * C::kChunkBytes, &maps.q, q_full,
                                                c * 64, U.h * p.G, U.q0 + k * p.tpt, pol_q);
                        }
                    }
                    const int32_t* bt = p.block_table + (int64_t)U.table * p.max_blocks;
                    int next = tma ? tile_block(p, bt, U.kb0, U.c1, lane) : 0;
                    for (int t = 0; t < U.nkt; ++t, ++kv_it) {
                        const int st = (int)(kv_it % nst);
                        const uint32_t n = kv_it / nst;
                        const int kb = U.kb0 + t * kKeys;
                        const int block = next;
                        if (tma && t + 1 < U.nkt) next = tile_block(p, bt, kb + kKeys, U.c1, lane);
                        if (n > 0 && !mbar_wait_warp(&empties[st], (n - 1) & 1, p.err)) {
                            s_abort = 1;
                            ok = false;
                            break;
                        }
                        uint8_t* dst = stages + st * kStage;
                        if (tma) {
                            const int valid = min(kKeys >> p.bs_log2, (U.c1 - kb + p.bs - 1) >> p.bs_log2);
                            if (lane == 0) mbar_arrive_expect_tx(&fulls[st], (uint32_t)(valid * kBoxes * p.bs * 128));
                            __syncwarp();
                            if (lane < valid) {
                                const int row = (block * p.Hkv + U.h) << p.bs_log2;
#pragma unroll
                                for (int c = 0; c < kBoxes; ++c)
                                    tma_load_2d(dst + c * C::kChunkBytes + lane * p.bs * 128, which ? &maps.v : &maps.k,
                                                &fulls[st], c * 64, row, pol);
                            }
                        } else {  // pages of 1, 2 or 4 tokens: 16-byte copies, zeros past the end
                            const uint32_t to = smem_u32(dst);
                            const uint8_t* from = static_cast<const uint8_t*>(which ? p.v_cache : p.k_cache);
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
                        if (st == 0) last[0] = n + 1;
                        else last[1] = n + 1;
                    }
                }
                // no copy may outlive the CTA, nor meet the next list's groups
#pragma unroll
                for (int st = 0; st < 2; ++st)
                    if (last[st]) mbar_wait_warp(&fulls[st], (last[st] - 1) & 1, p.err);
                if (which == 1 && q_it > 0) mbar_wait_warp(q_full, (q_it - 1) & 1, p.err);
            } else if (lane == 0 && warp == 1) {
                // -------------------------------------------------------- S_k = Q K^T
                constexpr uint32_t idesc = umma_idesc_bf16(128, 128, 0, 0);
                const uint32_t q_s = sm_base + C::kOffQ, k_s = sm_base + C::kOffK;
                bool ok = true;
                for (int i = 0; i < count && ok && !s_abort; ++i, ++q_it) {
                    const int nkt = pieces[i].nkt;
                    const bool two = !kFp8 && pieces[i].ntok > p.tpt;
                    if (!mbar_wait(q_full, q_it & 1, p.err)) {
                        ok = false;
                        break;
                    }
                    for (int t = 0; t < nkt; ++t, ++kv_it) {
                        const int st = kv_it & 1;
                        if (!mbar_wait(&k_full[st], (kv_it >> 1) & 1, p.err)) { ok = false; break; }
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            if (!ok || (!two && k != (t & 1))) continue;
                            if (nl[k] > 0 && !mbar_wait(&pv_done[k], (nl[k] - 1) & 1, p.err)) { ok = false; continue; }
                            tc_fence_after();
#pragma unroll
                            for (int ks = 0; ks < D / 16; ++ks) {
                                const uint32_t off = (ks >> 2) * C::kChunkBytes + (ks & 3) * 32;
                                umma_bf16(tbase + C::kColS + k * 128,
                                          umma_desc_sw128(q_s + (two ? k * C::kTileBytes : 0) + off, 16, 1024),
                                          umma_desc_sw128(k_s + st * C::kTileBytes + off, 16, 1024), idesc, ks > 0 ? 1u : 0u);
                            }
                            umma_commit(&s_full[k]);
                            ++nl[k];
                            if (k == 0 && t > 0) s_next0 = (int)kv_it;
                        }
                        if (!ok) break;
                        umma_commit(&k_empty[st]);
                        if (t == nkt - 1) umma_commit(q_empty);
                    }
                    if (ok) s_next0 = (int)kv_it;  // nothing of lane 0 follows in this unit
                }
                if (!ok) s_abort = 1;
                #pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (nl[k] > 0) mbar_wait(&s_full[k], (nl[k] - 1) & 1, p.err);
            } else if (lane == 0 && warp == 3) {
                // -------------------------------------------------------- O_k += P_k V
                constexpr uint32_t idesc = umma_idesc_bf16(128, D, 0, 1);
                const uint32_t v_s = sm_base + C::kOffV;
                bool ok = true;
                for (int i = 0; i < count && ok && !s_abort; ++i) {
                    const int nkt = pieces[i].nkt;
                    const bool two = !kFp8 && pieces[i].ntok > p.tpt;
                    for (int t = 0; t < nkt; ++t, ++kv_it) {
                        const int st = kv_it & 1;
                        if (!mbar_wait(&v_full[st], (kv_it >> 1) & 1, p.err)) { ok = false; break; }
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            if (!ok || (!two && k != (t & 1))) continue;
                            const bool first = two ? t == 0 : t < 2;
                            if (two && k == 1 && !wait_counter(s_next0, (int)kv_it + 1, p.err)) { ok = false; continue; }
                            for (int hh = 0; hh < 2 && ok; ++hh) {
                                if (!mbar_wait(hh ? &p_full[k] : &p_half[k], nl[k] & 1, p.err)) { ok = false; break; }
                                // a unit's first product overwrites O_k: the unit before must have been read
                                if (hh == 0 && first && uo[k] > 0 && !mbar_wait(&o_free[k], (uo[k] - 1) & 1, p.err)) {
                                    ok = false;
                                    break;
                                }
                                tc_fence_after();
#pragma unroll
                                for (int kq = 0; kq < kKeys / 32; ++kq) {
                                    const int kk = hh * (kKeys / 32) + kq;
                                    umma_bf16_ts(tbase + C::kColO + k * D, tbase + C::kColS + k * 128 + kk * 8,
                                                 umma_desc_sw128(v_s + st * C::kTileBytes + kk * 2048, C::kChunkBytes, 1024),
                                                 idesc, (!first || kk > 0) ? 1u : 0u);
                                }
                            }
                            if (!ok) continue;
                            umma_commit(&pv_done[k]);
                            ++nl[k];
                        }
                        if (!ok) break;
                        umma_commit(&v_empty[st]);
                    }
                    ++uo[0];
                    if (two || nkt > 1) ++uo[1];
                }
                if (!ok) s_abort = 1;
                #pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (nl[k] > 0) mbar_wait(&pv_done[k], (nl[k] - 1) & 1, p.err);
            }
            __syncwarp();
            setmaxnreg_inc<C::kRegsLaunch>();
        } else if (kFp8 && warp >= 12) {
            setmaxnreg_dec<C::kRegsWiden>();
            // ------------------------------------------------------------ codes to bf16 tiles
            // (E4M3 -> f16 -> f32 -> bf16, each exact.) A thread takes 16 codes of a row at a
            // time; of its two 16-byte pieces the threads of a row's second 64 elements
            // store the second one first, so that a quarter warp's stores use all banks.
            bool ok = true;
            const int wtid = tid - 384;
            for (int i = 0; i < count && ok && !warp_flag(s_abort); ++i) {
                const int nkt = pieces[i].nkt;
                for (int t = 0; t < nkt && ok; ++t, ++kv_it) {
                    const int st = (int)(kv_it & 1);
                    const uint32_t n = kv_it >> 1;
#pragma unroll
                    for (int which = 0; which < 2; ++which) {
                        const uint32_t ncode = which ? C::kCodeV : C::kCodeK;
                        const int cst = (int)(kv_it % ncode);
                        const uint32_t cn = kv_it / ncode;
                        uint64_t* cfull = (which ? cv_full : ck_full) + cst;
                        uint64_t* empty = (which ? v_empty : k_empty) + st;
                        if (!ok || !mbar_wait_warp(cfull, cn & 1, p.err) ||
                            (n > 0 && !mbar_wait_warp(empty, (n - 1) & 1, p.err))) {
                            ok = false;
                            continue;
                        }
                        const uint32_t from = sm_base + C::kOffCode + (which ? C::kCodeK * C::kCodeBytes : 0) + cst * C::kCodeBytes;
                        uint8_t* to = smem + (which ? C::kOffV : C::kOffK) + st * C::kTileBytes;
#pragma unroll 4
                        for (int j = wtid; j < kKeys * 8; j += 128) {
                            const uint32_t row = j >> 3, c = j & 7;
                            const uint4 x = lds128(from + sw128(row, c));
                            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                            uint32_t y[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const uint32_t h = e4m3x2_to_f16x2((w[e >> 1] >> ((e & 1) * 16)) & 0xffffu);
                                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
                                y[e] = pack_bf16(f.x, f.y);
                            }
                            uint8_t* base = to + (c >> 2) * C::kChunkBytes;
                            const uint32_t p0 = 2 * (c & 3);
                            const uint4 a = make_uint4(y[0], y[1], y[2], y[3]), b = make_uint4(y[4], y[5], y[6], y[7]);
                            const bool second = c >= 4;
                            *reinterpret_cast<uint4*>(base + sw128(row, p0 + second)) = second ? b : a;
                            *reinterpret_cast<uint4*>(base + sw128(row, p0 + !second)) = second ? a : b;
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive((which ? v_full : k_full) + st);
                            mbar_arrive((which ? cv_empty : ck_empty) + cst);
                        }
                    }
                }
            }
            if (!ok) s_abort = 1;
            __syncwarp();
            setmaxnreg_inc<C::kRegsLaunch>();
        } else {
            setmaxnreg_inc<C::kRegsSoftmax>();
            // ------------------------------------------------------------ softmax lanes
            const int k = warp >= 8 ? 1 : 0;
            const int row = 32 * (warp & 3) + lane;  // of the row tile = tensor memory lane
            const int row_tok = row / p.G;
            const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
            const int wg_tid = tid - 128 * (k + 1);
            const uint32_t tS = tbase + lane_off + C::kColS + k * 128;
            const uint32_t tO = tbase + lane_off + C::kColO + k * D;
            const float sl2 = p.scale_log2;
            for (int i = 0; i < count && !warp_flag(s_abort); ++i) {
                const Piece U = pieces[i];
                const bool two = !kFp8 && U.ntok > p.tpt;
                const int tok = (two ? k * p.tpt : 0) + row_tok;  // of the unit
                const bool write = row_tok < p.tpt && tok < U.ntok;
                const bool common = U.slot < 0;
                const int half = common ? p.rows_pre : p.rows_own;  // rows of a lane's half of a slot
                const int64_t slot = U.slot & INT32_MAX;
                float* po = (common ? p.po_pre : p.po_own) + slot * 2 * half * D + (k * half + row) * 4;
                float* pl = (common ? p.pl_pre : p.pl_own) + slot * 2 * half + k * half + row;
                const uint32_t kv_base = kv_it;
                kv_it += U.nkt;
                const int step = two ? 1 : 2, t_first = two ? 0 : k;
                if (t_first >= U.nkt) {  // no key tile for this lane (the join reads no result of it)
                    if (write) *pl = -INFINITY;
                    continue;
                }
                const int c1 = min(U.c1, U.pos0 + tok + 1);  // the row's visible keys end here
                const int all1 = min(U.c1, U.pos0 + 1);      // every row sees these
                float m_used = -INFINITY, l = 0.f;
                bool ok = true;
                for (int t = t_first; t < U.nkt; t += step) {
                    if (!mbar_wait_warp(&s_full[k], n_s & 1, p.err)) { ok = false; break; }
                    tc_fence_after();
                    const int kb = U.kb0 + t * kKeys;
                    const bool edge = kb < U.c0 || kb + kKeys > all1;
                    const int vlo = U.c0 - kb;  // visible columns [vlo, vlo + seen)
                    const uint32_t seen = (uint32_t)max(0, c1 - U.c0);
                    float ls[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                    bool rescale = false;
                    float alpha = 1.f;
                    float mx[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) mx[j] = -INFINITY;
                    auto load_half = [&](uint32_t (&r)[64], int h) {  // scores of keys 64 h ...
                        tmem_ld32(tS + 64 * h, *reinterpret_cast<uint32_t(*)[32]>(r));
                        tmem_ld32(tS + 64 * h + 32, *reinterpret_cast<uint32_t(*)[32]>(r + 32));
                    };
                    auto mask_half = [&](uint32_t (&r)[64], int h) {
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            if ((uint32_t)(64 * h + j - vlo) >= seen) r[j] = 0xff800000u;
                    };
                    auto max_half = [&](const uint32_t (&r)[64]) {
#pragma unroll
                        for (int j = 0; j < 64; j += 2)
                            mx[(j >> 1) & 7] = fmax3f(mx[(j >> 1) & 7], __uint_as_float(r[j]), __uint_as_float(r[j + 1]));
                    };
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
                    // P of 64 keys, in bf16 pairs over columns 32 h of S (which have been read)
                    auto store_half = [&](const uint32_t (&r)[64], int h) {
                        uint32_t pk[32];
#pragma unroll
                        for (int j = 0; j < 64; j += 2) {
                            float x0, x1;
                            fma2_bcast(x0, x1, __uint_as_float(r[j]), __uint_as_float(r[j + 1]), sl2, -m_off);
                            const float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
                            const int a = (j >> 1) & 3;
                            add2(ls[2 * a], ls[2 * a + 1], e0, e1);
                            pk[j / 2] = pack_bf16(e0, e1);
                        }
                        tmem_st32(tS + 32 * h, pk);
                    };
                    bool early;
                    auto signal_half = [&] {  // the product over keys 0..63 may start
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&p_half[k]);
                    };
                    if constexpr (!kFp8) {  // the whole row in registers
                        uint32_t r0[64], r1[64];
                        load_half(r0, 0);
                        load_half(r1, 1);
                        tmem_wait_ld();
                        if (edge) {
                            mask_half(r0, 0);
                            mask_half(r1, 1);
                        }
                        max_half(r0);
                        max_half(r1);
                        take_max();
                        early = !edge && !__any_sync(0xffffffffu, rescale);
                        store_half(r0, 0);
                        if (early) signal_half();
                        store_half(r1, 1);
                    } else {  // twice in halves: these lanes have fewer registers
                        uint32_t r[64], r1[64];
                        load_half(r, 0);
                        tmem_wait_ld();
                        if (edge) mask_half(r, 0);
                        max_half(r);
                        load_half(r1, 1);
                        tmem_wait_ld();
                        if (edge) mask_half(r1, 1);
                        max_half(r1);
                        take_max();
                        early = !edge && !__any_sync(0xffffffffu, rescale);
                        load_half(r, 0);
                        tmem_wait_ld();
                        if (edge) mask_half(r, 0);
                        store_half(r, 0);
                        if (early) signal_half();
                        load_half(r1, 1);
                        tmem_wait_ld();
                        if (edge) mask_half(r1, 1);
                        store_half(r1, 1);
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
                    // value rows outside the segment's keys may hold anything: zero. With two
                    // row tiles lane 0 does it (lane 1's product of a tile follows lane 0's).
                    const int zlo = max(0, U.c0 - kb), zhi = min(kKeys, U.c1 - kb);
                    if ((zlo > 0 || zhi < kKeys) && (k == 0 || !two)) {
                        const uint32_t vi = kv_base + t;
                        if (!mbar_wait_warp(&v_full[vi & 1], (vi >> 1) & 1, p.err)) { ok = false; break; }
                        uint8_t* vt = smem + C::kOffV + (vi & 1) * C::kTileBytes;
                        for (int ci = wg_tid; ci < kKeys * (D / 8); ci += 128) {
                            const int vr = ci / (D / 8), c = ci % (D / 8);
                            if (vr >= zlo && vr < zhi) continue;
                            *reinterpret_cast<uint4*>(vt + (c >> 3) * C::kChunkBytes + sw128(vr, c & 7)) = make_uint4(0, 0, 0, 0);
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
                for (int c = 0; c < D / 32; ++c) {
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
                if (write) *pl = m_used + log2f(l);
            }
            __syncwarp();
            setmaxnreg_dec<C::kRegsLaunch>();
        }
        __syncthreads();
        if (s_abort) break;
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
constexpr int kJoinThreads = 128;

struct Source {
    const float* o;  // the rows' first four values; those of the next four dims 4 * rows further on
    const float* l;
    int rows;
};

template <int D>
__global__ void __launch_bounds__(kJoinThreads) prefix_join_kernel(const PrefixParams p, int ncta) {
    extern __shared__ __align__(16) uint8_t s_join[];
    __shared__ float s_top[16], s_sum[16];
    Source* src = reinterpret_cast<Source*>(s_join);                    // [4 * ncta]
    float* weight = reinterpret_cast<float*>(src + 4 * (size_t)ncta);  // [4 * ncta][G]
    grid_dep_launch();
    grid_dep_wait();
    const int t = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
    const i64 total = p.seg_cost[p.own0 + p.B];
    if (total < 0) return;  // refused lengths: nothing is written
    const TokenPlace at = place_of(p.qsl, p.seq_lens, p.B, t);
    if (at.r < 0) return;
    const int g = last_at_most(p.starts, p.groups, at.r);
    const int r0 = __ldg(p.starts + g), r1 = __ldg(p.starts + g + 1);
    const int common = common_keys(r0, r1, __ldg(p.prefix + g));
    int n = 0;  // pieces, in the order of their keys
    for (int part = 0; part < 2; ++part) {
        const int gq0 = __ldg(p.qsl + r0);
        const Seg s = part == 0 ? make_seg(p, gq0, __ldg(p.qsl + r1) - gq0, 0, common)
                                : make_seg(p, at.q0, at.q1 - at.q0, common, at.len);
        if (s.nkt == 0) continue;
        const int index = part == 0 ? g : p.own0 + at.r;
        const int rt = (t - s.q0) / p.upt, tok = (t - s.q0) % p.upt;
        const bool two = min(p.upt, s.n - rt * p.upt) > p.tpt;
        const int local = h * s.nrt + rt;
        const i64 us = p.seg_cost[index] + (i64)local * s.nkt * s.w;
        const int unit = p.seg_unit[index] + local - (part == 0 ? 0 : p.seg_unit[p.own0]);
        const int half = part == 0 ? p.rows_pre : p.rows_own;
        const int row = two ? tok / p.tpt * half + tok % p.tpt * p.G : tok * p.G;
        const int first = cta_of(us, total, ncta), last = cta_of(us + (i64)(s.nkt - 1) * s.w, total, ncta);
        const int lanes = two ? 1 : 2;
        for (int j = tid; j < (last - first + 1) * lanes; j += kJoinThreads) {
            const int c = first + j / lanes, k = j % lanes;
            const int t0 = first_tile(share_start(c, total, ncta), us, s.w, s.nkt);
            const int t1 = first_tile(share_start(c + 1, total, ncta), us, s.w, s.nkt);
            const i64 slot = (i64)(unit + c) * 2 * half;
            Source x;
            x.rows = 2 * half;
            x.o = (part == 0 ? p.po_pre : p.po_own) + slot * D + (k * half + row) * 4;
            x.l = t1 - t0 > k ? (part == 0 ? p.pl_pre : p.pl_own) + slot + k * half + row : nullptr;  // (no tile for that lane)
            src[n + j] = x;
        }
        n += (last - first + 1) * lanes;
    }
    __syncthreads();
    const int G = p.G;
    for (int j = tid; j < n * G; j += kJoinThreads) {
        const float* l = src[j / G].l;
        weight[j] = l ? __ldcg(l + j % G) : -INFINITY;
    }
    __syncthreads();
    // ---- weights: a thread per head
    if (tid < G) {
        float top = -INFINITY;
        for (int i = 0; i < n; ++i) top = fmaxf(top, weight[i * G + tid]);
        s_top[tid] = top;
    }
    __syncthreads();
    for (int j = tid; j < n * G; j += kJoinThreads) {
        const float l = weight[j], top = s_top[j % G];
        weight[j] = l == -INFINITY ? 0.f : l == top ? 1.f : exp2f(l - top);  // (equal infinities are NaN anyway)
    }
    __syncthreads();
    if (tid < G) {
        float sum = 0.f;
        for (int i = 0; i < n; ++i) sum += weight[i * G + tid];
        s_sum[tid] = sum;
        if (p.lse) p.lse[(int64_t)t * p.Hq + h * G + tid] = (s_top[tid] + log2f(sum)) * 0.69314718055994531f;
    }
    __syncthreads();
    for (int f = tid; f < D / 4 * G; f += kJoinThreads) {
        const int hh = f % G, d4 = f / G;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const float w = weight[i * G + hh];
            const float4 o = __ldcg(reinterpret_cast<const float4*>(src[i].o) + (i64)d4 * src[i].rows + hh);
            if (w != 0.f) {  // (the place of a piece that is none may hold anything)
                acc.x += w * o.x;
                acc.y += w * o.y;
                acc.z += w * o.z;
                acc.w += w * o.w;
            }
        }
        const float inv = p.v_scale / s_sum[hh];
        *reinterpret_cast<uint2*>(p.out + ((int64_t)t * p.Hq + h * G + hh) * D + d4 * 4) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    }
}

template <int D, bool kFp8>
cudaError_t go_attn(const PrefixMaps& maps, const PrefixParams& p, int ncta, cudaStream_t stream) {
    using C = PxCfg<D, kFp8>;
    auto kern = prefix_attn_kernel<D, kFp8>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(ncta), dim3(C::kThreads), C::kSmem, stream, maps, p);
}

template <int D>
cudaError_t go_join(const PrefixParams& p, int ncta, cudaStream_t stream) {
    auto kern = prefix_join_kernel<D>;
    const size_t smem = 4 * (size_t)ncta * (sizeof(Source) + sizeof(float) * p.G);
    if (smem > 47 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)(4 * (size_t)ncta * (sizeof(Source) + sizeof(float) * 16)));
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(kern, dim3(p.T, p.Hkv), dim3(kJoinThreads), smem, stream, p, ncta);
}

}  // namespace

cudaError_t launch_prefix_attn(const PrefixMaps& maps, const PrefixParams& p, int head_dim, bool fp8, int ncta,
                               cudaStream_t stream) {
    if (fp8) return go_attn<128, true>(maps, p, ncta, stream);
    return head_dim == 128 ? go_attn<128, false>(maps, p, ncta, stream) : go_attn<64, false>(maps, p, ncta, stream);
}

cudaError_t launch_prefix_join(const PrefixParams& p, int head_dim, int ncta, cudaStream_t stream) {
    return head_dim == 128 ? go_join<128>(p, ncta, stream) : go_join<64>(p, ncta, stream);
}

}  // namespace pka
