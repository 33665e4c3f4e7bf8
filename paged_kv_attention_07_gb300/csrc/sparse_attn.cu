// sparse_attn.cu -- attention of each new token over the pages listed for it.
//
// Token t at position p of request r, kv head g with its G query heads, the
// ascending list of pages e_0 < e_1 < ... <= p / bs:
//     s_j = scale * <q, K_j>,  out = sum_j softmax(s)_j V_j,  lse = log sum_j exp(s_j)
// over the keys j <= p of the listed pages. Only the token's own page can be
// partly filled and it comes last, so the listed keys are one run of
// (count - 1) * bs + tail keys: tile i of 16 keys lies in page e[16 i / bs].
//
// HBM-bound: every listed page is read once, 16 keys of one (page, kv head) are
// one contiguous tile that 16-byte asynchronous copies bring into a warp's own
// ring of stages (swizzled by the row, so that the fragments' reads meet no bank
// twice). Tile copies by TMA boxes read a full batch as fast, but one lane's
// TMA instructions take 390 to 750 cycles of the warp's time per tile, more than
// the products; 32 lanes' copies some 80. A warp owns a contiguous run of tiles
// and never waits for another: its lanes hold the cache rows of its next 32
// pages (list entry -> block table -> row), a tile's row is one shuffle away. The work of one (token, kv head) is split over the
// 4 warps of a CTA and the CTAs of a cluster; the warps' (m, l, O) join in
// shared memory and the CTAs' over distributed shared memory, so there is one
// launch and nothing partial goes to memory.
//
// Several tokens of one request (a prompt's chunk, drafted tokens) are taken in
// groups: their lists, mostly the same pages, are united in shared memory (a
// bit map per token, then one prefix sum), each page of the union is read and
// widened once, and the tokens' heads lie side by side in the MMA's columns;
// columns whose token does not list the page, or stands before the key, get
// weight zero. A zero weight does not hide an infinite or NaN value, so a group
// whose result is not finite throughout is done again token by token.
//
// Math per tile as in the split-KV decode (bf16 operands, fp32 accumulation):
//   S^T[16 keys x 8 columns] = K Q^T;  online softmax per column;  O^T += V^T P^T
// P is rounded to bf16 for the product (its sum l is not): the error is that of
// the operands' own type. Over an 8-bit cache the codes are widened to f16
// (exact), q and P are f16, and the scales come out of the sums.
#include "common.cuh"
#include "params.cuh"

namespace pka {

namespace {

constexpr int kSaWarps = 4;
constexpr int kSaThreads = kSaWarps * 32;
constexpr int kSaTile = 16;  // keys per tile
constexpr int kSaJoin = 8;   // CTAs' results read together
constexpr int kSaGroup = 8;  // tokens of a group, at most

template <int D, int NT, bool kFp8>
struct SaCfg {
    static constexpr int kRowBytes = D * (kFp8 ? 1 : 2);
    static constexpr int kTileBytes = kSaTile * kRowBytes;
    static constexpr int kStageBytes = 2 * kTileBytes;  // K + V
    static constexpr int kStages = 3;
    static constexpr int kRing = kSaWarps * kStages * kStageBytes;
    static constexpr int kCols = NT * 8;
    // q's fragments: in registers up to two column blocks, beyond in shared memory
    static constexpr bool kQShared = NT > 2;
    static constexpr int kQ = kQShared ? NT * (D / 16) * 32 * 8 : 0;
    // the join: each warp's m, l and O (over the ring), and the CTA's own
    static constexpr int kWarpFloats = kCols * (D + 2);
    static constexpr int kJoin = kSaWarps * kWarpFloats * 4;
    static constexpr int kBody = kRing > kJoin ? kRing : kJoin;
    static constexpr int kSmem = 1024 /*align*/ + kBody + kWarpFloats * 4 + kQ;
};

// A tile's keys in a group, eight at a time: the position of the first, and the
// tokens (bits) that list their page.
struct SaHalf {
    int base;
    uint32_t who;
};

// Where group w of kGroupTokens tokens stands: groups of request r are w =
// qsl[r] / R + r and the following (some of them empty). With whole warps.
struct GroupPlace {
    int r, t0, n, q1, len;  // n tokens from t0 on; 0: none
};
PKA_DEVICE GroupPlace group_of(const int32_t* qsl, const int32_t* seq_lens, int nreq, int w, int R) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = nreq;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5;
        const int i = lo + lane * step;
        const uint32_t at_most = __ballot_sync(0xffffffffu, i < hi && __ldg(qsl + i) / R + i <= w);
        const int k = at_most ? 31 - __clz(at_most) : 0;
        lo += k * step;
        hi = min(hi, lo + step);
    }
    GroupPlace g;
    g.r = lo;
    const int q0 = __ldg(qsl + lo);
    g.q1 = __ldg(qsl + lo + 1);
    g.len = __ldg(seq_lens + lo);
    const long long t0 = (long long)q0 + (long long)(w - (q0 / R + lo)) * R;
    g.t0 = (int)t0;
    g.n = t0 < q0 || t0 >= g.q1 ? 0 : min(R, g.q1 - g.t0);
    return g;
}

PKA_DEVICE uint32_t e4m3_lo(uint32_t w) { return e4m3x2_to_f16x2(w & 0xffffu); }
PKA_DEVICE uint32_t e4m3_hi(uint32_t w) { return e4m3x2_to_f16x2(w >> 16); }

// Row `tr`, 16-byte chunk c of a bf16 tile: 128-byte column segments of 16
// rows one after another, each in the 128-byte swizzle.
PKA_DEVICE uint32_t seg_off(int tr, int c) { return sw128((uint32_t)((c >> 3) * kSaTile + tr), (uint32_t)(c & 7)); }

template <int D, int NT, bool kFp8, bool kGroup>
__global__ void __launch_bounds__(kSaThreads, kFp8 && NT == 1 ? 4 : 2)
    sparse_attn_kernel(const SparseAttnParams p) {
    using C = SaCfg<D, NT, kFp8>;
    constexpr int kKSteps = D / 16;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int s_stop[kSaGroup];
    __shared__ uint32_t s_scan[kSaWarps], s_bad;
    __shared__ SaHalf s_half[kGroup ? kSaWarps : 1][C::kStages][2];
    grid_dep_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c4 = lane & 3, r8 = lane >> 2;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* own = reinterpret_cast<float*>(smem + C::kBody);  // this CTA's O [kCols][D], m, l
    uint4* s_q = reinterpret_cast<uint4*>(smem + C::kBody + C::kWarpFloats * 4);
    // a group's united list: page | tokens << 24
    uint32_t* s_list = reinterpret_cast<uint32_t*>(smem + C::kSmem - 1024);
    if (tid < kSaGroup) s_stop[tid] = p.num_pages;
    if (tid == 0) s_bad = 0;
    __syncthreads();
    grid_dep_wait();

    // ---- the tokens [t0, t0 + ntok), consecutive ones of one request
    const int ncta = (int)cluster_size(), cta = (int)cluster_rank();
    const int g = blockIdx.y, unit = (int)(blockIdx.x / (unsigned)ncta);
    int r, t0, ntok, q1, len;
    if constexpr (kGroup) {
        const GroupPlace at = group_of(p.qsl, p.seq_lens, p.num_reqs, unit, p.group);
        r = at.r, t0 = at.t0, ntok = at.n, q1 = at.q1, len = at.len;
        if (ntok <= 0 || t0 < 0 || t0 > p.num_tokens - ntok) return;  // no such group
    } else {
        const TokenPlace at = place_of(p.qsl, p.seq_lens, p.num_reqs, unit);
        r = at.r, t0 = unit, ntok = 1, q1 = at.q1, len = at.len;
        if (r < 0) return;  // a row behind the last sequence
        if (t0 < at.q0) len = -1;
    }
    const long long pos = (long long)len - q1 + t0;  // the first token's position
    if (pos < 0 || pos + ntok > len || len > p.max_seq_len) {
        if (tid == 0 && cta == 0 && g == 0) set_error(p.err, PKA_DEVERR_SEQ_LEN);
        return;
    }
    const int pos0 = (int)pos, pos1 = pos0 + ntok - 1;
    const int64_t row0 = (int64_t)t0 * p.Hq + g * p.G;  // first output row of the first token
    const int cols = ntok * p.G;
    auto row_of = [&](int col) { return kGroup ? row0 + (int64_t)(col / p.G) * p.Hq + col % p.G : row0 + col; };

    // ---- the lists: each ends at its first negative entry; entries ascend and none is past the token's page
    const int32_t* sel = p.sel + ((int64_t)t0 * p.Hkv + g) * p.num_pages;
    const int64_t sel_step = (int64_t)p.Hkv * p.num_pages;  // from a token's list to the next one's
    if constexpr (!kGroup) {
        const int own_page = pos0 >> p.bs_log2;
        for (int i = tid; i < p.num_pages; i += kSaThreads) {
            const int e = __ldg(sel + i), before = i ? __ldg(sel + i - 1) : -1;
            if (e <= before || e > own_page) {  // e < 0 among them
                atomicMin(&s_stop[0], i);
                break;
            }
        }
    } else {
        for (int i0 = tid; i0 < p.num_pages; i0 += kSaThreads) {
            int e[kSaGroup], before[kSaGroup];
#pragma unroll
            for (int k = 0; k < kSaGroup; ++k) {
                e[k] = k < ntok ? __ldg(sel + k * sel_step + i0) : 0;
                before[k] = k < ntok && i0 ? __ldg(sel + k * sel_step + i0 - 1) : -1;
            }
#pragma unroll
            for (int k = 0; k < kSaGroup; ++k)
                if (k < ntok && (e[k] <= before[k] || e[k] > (pos0 + k) >> p.bs_log2)) atomicMin(&s_stop[k], i0);
        }
    }
    const int last_page = pos1 >> p.bs_log2;
    const int words = last_page / 32 + 1;
    uint32_t* s_map = reinterpret_cast<uint32_t*>(smem);  // (the ring is idle still) a bit map per token
    if constexpr (kGroup)
        for (int i = tid; i < ntok * words; i += kSaThreads) s_map[i] = 0;
    __syncthreads();
    if (cta == 0 && tid < ntok && s_stop[tid] < p.num_pages && __ldg(sel + tid * sel_step + s_stop[tid]) >= 0)
        set_error(p.err, PKA_DEVERR_INDEX);
    int count = s_stop[0], last = -1;  // pages to read, and the last of them
    if constexpr (kGroup) {
        for (int i = tid; i < p.num_pages; i += kSaThreads) {
            int e[kSaGroup];
#pragma unroll
            for (int k = 0; k < kSaGroup; ++k) e[k] = k < ntok && i < s_stop[k] ? __ldg(sel + k * sel_step + i) : -1;
#pragma unroll
            for (int k = 0; k < kSaGroup; ++k)
                if (e[k] >= 0) atomicOr(&s_map[k * words + (e[k] >> 5)], 1u << (e[k] & 31));
        }
        __syncthreads();
        const int per = (words + kSaThreads - 1) / kSaThreads;
        const int w0 = min(words, tid * per), w1 = min(words, w0 + per);
        uint32_t mine = 0;
        for (int w = w0; w < w1; ++w) {
            uint32_t any = 0;
            for (int k = 0; k < ntok; ++k) any |= s_map[k * words + w];
            mine += __popc(any);
        }
        uint32_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) s_scan[warp] = incl;
        __syncthreads();
        uint32_t at = incl - mine;
        count = 0;
#pragma unroll
        for (int w = 0; w < kSaWarps; ++w) {
            at += w < warp ? s_scan[w] : 0u;
            count += (int)s_scan[w];
        }
        for (int w = w0; w < w1; ++w) {
            uint32_t any = 0, map[kSaGroup];
#pragma unroll
            for (int k = 0; k < kSaGroup; ++k) {
                map[k] = k < ntok ? s_map[k * words + w] : 0u;
                any |= map[k];
            }
            for (; any; any &= any - 1) {
                const int bit = __ffs(any) - 1;
                uint32_t who = 0;
#pragma unroll
                for (int k = 0; k < kSaGroup; ++k) who |= (map[k] >> bit & 1u) << k;
                s_list[at++] = (uint32_t)(w * 32 + bit) | who << 24;
            }
        }
        __syncthreads();  // (the ring is written by copies from here on)
        if (count > 0) last = (int)(s_list[count - 1] & 0xffffffu);
    } else {
        if (count > 0) last = __ldg(sel + count - 1);
    }
    const int keys = count * p.bs - (last == last_page ? p.bs - 1 - (pos1 & (p.bs - 1)) : 0);
    // tokens without a page: nothing to read
    if (cta == 0)
        for (int k = 0; k < ntok; ++k) {
            if (s_stop[k] > 0) continue;
            for (int i = tid; i < p.G * D / 8; i += kSaThreads)
                reinterpret_cast<uint4*>(p.out + (row0 + (int64_t)k * p.Hq) * D)[i] = make_uint4(0, 0, 0, 0);
            if (p.lse && tid < p.G) p.lse[row0 + (int64_t)k * p.Hq + tid] = -INFINITY;
        }
    if (keys == 0) return;
    const int ntiles = (keys + kSaTile - 1) / kSaTile;
    const int part = cta * kSaWarps + warp, parts = ncta * kSaWarps;
    // (parts is a power of two up to 64, ntiles below 2^31 / kSaTile)
    const int parts_log2 = 31 - __clz(parts);
    const int i0 = (int)((uint32_t)ntiles >> parts_log2) * part + (((ntiles & (parts - 1)) * part) >> parts_log2);
    const int i1 = (int)((uint32_t)ntiles >> parts_log2) * (part + 1) + (((ntiles & (parts - 1)) * (part + 1)) >> parts_log2);

    // ---- this warp's loads: step j of a tile copies 32 pieces of 16 bytes, kRows rows
    constexpr int kPieces = C::kRowBytes / 16, kRows = 32 / kPieces, kSteps = kSaTile / kRows;
    const uint64_t pol = policy_evict_first();
    const uint8_t* kc = static_cast<const uint8_t*>(p.k_cache) + lane * 16;
    const uint8_t* vc = static_cast<const uint8_t*>(p.v_cache) + lane * 16;
    uint32_t place[8 / kRows];  // of step j in a tile; 8 rows on, the same swizzle
#pragma unroll
    for (int j = 0; j < 8 / kRows; ++j) {
        const int row = j * kRows + lane / kPieces, piece = lane % kPieces;
        place[j] = kFp8 ? sw128(row, piece) : seg_off(row, piece);
    }
    uint8_t* ring = smem + warp * C::kStages * C::kStageBytes;
    const int boxr = min(p.bs, kSaTile);
    int page0 = -32, rows = 0;  // lane l holds the first cache row of listed page page0 + l
    uint32_t entry = 0;         // and, of a group, its entry
    uint32_t it = 0;  // tiles taken
    auto issue = [&](int i, int stage) {
        const int first = (i * kSaTile) >> p.bs_log2;
        if (first < page0 || first + kSaTile / boxr > page0 + 32) {
            page0 = first;
            const int j = page0 + lane;
            int blk = 0;
            entry = 0;
            if (j < count) {
                int e;
                if constexpr (kGroup) {
                    entry = s_list[j];
                    e = (int)(entry & 0xffffffu);
                } else {
                    e = __ldg(sel + j);
                }
                blk = __ldg(p.block_table + (int64_t)r * p.max_blocks + e);
                if (blk < 0 || blk >= p.num_blocks) {
                    set_error(p.err, PKA_DEVERR_BLOCK_ID);
                    blk = 0;
                }
            }
            rows = (blk * p.Hkv + g) * p.bs;
        }
        const int off = (i * kSaTile) & (p.bs - 1);
        const int ra = __shfl_sync(0xffffffffu, rows, first - page0) + off;
        const int rb = __shfl_sync(0xffffffffu, rows, (first + 1 - page0) & 31);  // bs == 8: the tile's second page
        const bool two = boxr < kSaTile && i * kSaTile + boxr < keys;
        if constexpr (kGroup) {
            const uint32_t ea = __shfl_sync(0xffffffffu, entry, first - page0);
            const uint32_t eb = boxr < kSaTile ? __shfl_sync(0xffffffffu, entry, (first + 1 - page0) & 31) : ea;
            if (lane < 2) {
                const uint32_t e = lane ? eb : ea;
                SaHalf h;
                h.base = (int)(e & 0xffffffu) * p.bs + (boxr < kSaTile ? 0 : off + 8 * lane);
                h.who = lane && boxr < kSaTile && !two ? 0u : e >> 24;
                s_half[warp][stage][lane] = h;
            }
        }
        const uint32_t kdst = smem_u32(ring + stage * C::kStageBytes), vdst = kdst + C::kTileBytes;
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // eight rows each
            if (h && boxr < kSaTile && !two) break;
            const int64_t src = (int64_t)(h && boxr < kSaTile ? rb - 8 : ra) * C::kRowBytes;
#pragma unroll
            for (int j = 0; j < kSteps / 2; ++j) {
                const int step = h * (kSteps / 2) + j;
                cp_async_16_hint(kdst + place[j] + h * 1024, kc + src + step * 512, pol);
                cp_async_16_hint(vdst + place[j] + h * 1024, vc + src + step * 512, pol);
            }
        }
    };
    auto first_tiles = [&] {
#pragma unroll
        for (int s = 0; s < C::kStages; ++s) {
            if (i0 + s < i1) issue(i0 + s, s);
            cp_async_commit();  // (a group per tile, empty behind the last)
        }
        it = 0;
    };
    first_tiles();

    // ---- Q^T fragments: column n, zero behind the last
    uint32_t qf[C::kQShared ? 1 : NT][kKSteps][2];
    auto load_q = [&](uint32_t (&f)[kKSteps][2], int nt) {
        const int n = nt * 8 + r8;
        const bool ok = n < cols;
        const __nv_bfloat16* qrow = p.q + row_of(ok ? n : 0) * D;
        if constexpr (kFp8) {  // k-step ks holds dims 32 c4 + 4 ks .. + 3, as the codes are read
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint4 v = ok ? __ldg(reinterpret_cast<const uint4*>(qrow + 32 * c4) + j) : make_uint4(0, 0, 0, 0);
                f[2 * j][0] = bf16x2_to_f16x2(v.x);
                f[2 * j][1] = bf16x2_to_f16x2(v.y);
                f[2 * j + 1][0] = bf16x2_to_f16x2(v.z);
                f[2 * j + 1][1] = bf16x2_to_f16x2(v.w);
            }
        } else {
#pragma unroll
            for (int ks = 0; ks < kKSteps; ++ks) {
                f[ks][0] = ok ? __ldg(reinterpret_cast<const uint32_t*>(qrow) + ks * 8 + c4) : 0u;
                f[ks][1] = ok ? __ldg(reinterpret_cast<const uint32_t*>(qrow) + ks * 8 + 4 + c4) : 0u;
            }
        }
    };
    if constexpr (C::kQShared) {  // one column block per warp, two k-steps per 16 bytes
        for (int nt = warp; nt < NT; nt += kSaWarps) {
            load_q(qf[0], nt);
#pragma unroll
            for (int ks = 0; ks < kKSteps; ks += 2)
                s_q[(nt * kKSteps / 2 + ks / 2) * 32 + lane] = make_uint4(qf[0][ks][0], qf[0][ks][1], qf[0][ks + 1][0], qf[0][ks + 1][1]);
        }
        __syncthreads();
    } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) load_q(qf[nt], nt);
    }
    // q's fragments of k-steps ks and ks + 1
    auto q_pair = [&](int nt, int ks) {
        if constexpr (C::kQShared) return s_q[(nt * kKSteps / 2 + ks / 2) * 32 + lane];
        else return make_uint4(qf[nt][ks][0], qf[nt][ks][1], qf[nt][ks + 1][0], qf[nt][ks + 1][1]);
    };
    // this lane's columns of S^T: their token's bit and position (a column behind the last: none)
    uint32_t bit[kGroup ? NT : 1][2];
    int limit[kGroup ? NT : 1][2];
    if constexpr (kGroup) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int hc = 0; hc < 2; ++hc) {
                const int n = nt * 8 + c4 * 2 + hc, k = n / p.G;
                bit[nt][hc] = n < cols ? 1u << k : 0u;
                limit[nt][hc] = pos0 + k;
            }
    }

    // ---- one pass over the tiles; a group with values that are not finite takes one more per token
    for (int pass = 0;; ++pass) {
    const uint32_t who = pass == 0 ? (1u << ntok) - 1 : 1u << (pass - 1);  // the tokens of this pass
    const int end = pass == 0 ? pos1 : pos0 + pass - 1;                    // the last one's position
    if (pass > 0) first_tiles();
    float o[kKSteps][NT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int mt = 0; mt < kKSteps; ++mt) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
    }

    for (int i = i0; i < i1; ++i) {
        const int stage = it % C::kStages;
        ++it;
        cp_async_wait<C::kStages - 1>();
        __syncwarp();
        uint8_t* kt = ring + stage * C::kStageBytes;
        uint8_t* vt = kt + C::kTileBytes;
        // valid keys of the tile's two halves; the rest's values may be anything: zeros instead
        int valid0, valid1;
        SaHalf h0, h1;
        if constexpr (kGroup) {
            h0 = s_half[warp][stage][0], h1 = s_half[warp][stage][1];
            valid0 = h0.who & who ? min(8, max(0, end + 1 - h0.base)) : 0;
            valid1 = h1.who & who ? min(8, max(0, end + 1 - h1.base)) : 0;
        } else {
            valid0 = min(8, keys - i * kSaTile);
            valid1 = min(8, max(0, keys - i * kSaTile - 8));
        }
        if (valid0 + valid1 < kSaTile) {
            for (int ci = lane; ci < kSaTile * (C::kRowBytes / 16); ci += 32) {
                const int tr = ci / (C::kRowBytes / 16), c = ci % (C::kRowBytes / 16);
                if (tr < 8 ? tr >= valid0 : tr - 8 >= valid1)
                    *reinterpret_cast<uint4*>(vt + (kFp8 ? sw128(tr, c) : seg_off(tr, c))) = make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
        }
        const uint32_t kb = smem_u32(kt), vb = smem_u32(vt);

        // ---- S^T = K Q^T
        float sc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
        if constexpr (kFp8) {
#pragma unroll
            for (int jc = 0; jc < 2; ++jc) {
                const uint4 lo = lds128(kb + sw128(r8, 2 * c4 + jc)), hi = lds128(kb + sw128(r8 + 8, 2 * c4 + jc));
                const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    const uint32_t a0 = e4m3_lo(wl[k]), a1 = e4m3_lo(wh[k]), a2 = e4m3_hi(wl[k]), a3 = e4m3_hi(wh[k]);
                    const uint32_t b0 = e4m3_lo(wl[k + 1]), b1 = e4m3_lo(wh[k + 1]), b2 = e4m3_hi(wl[k + 1]), b3 = e4m3_hi(wh[k + 1]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint4 q = q_pair(nt, 4 * jc + k);
                        mma_f16(sc[nt], a0, a1, a2, a3, q.x, q.y);
                        mma_f16(sc[nt], b0, b1, b2, b3, q.z, q.w);
                    }
                }
            }
        } else {
            const int mi = lane >> 3, tr = (mi & 1) * 8 + (lane & 7);
#pragma unroll
            for (int ks = 0; ks < kKSteps; ks += 2) {
                uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
                ldsm_x4(kb + seg_off(tr, ks * 2 + (mi >> 1)), a0, a1, a2, a3);
                ldsm_x4(kb + seg_off(tr, ks * 2 + 2 + (mi >> 1)), b0, b1, b2, b3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint4 q = q_pair(nt, ks);
                    mma_bf16(sc[nt], a0, a1, a2, a3, q.x, q.y);
                    mma_bf16(sc[nt], b0, b1, b2, b3, q.z, q.w);
                }
            }
        }
        // ---- online softmax in the log2 domain; other keys weigh nothing
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float x[4];
#pragma unroll
            for (int hc = 0; hc < 2; ++hc) {
                bool v0 = r8 < valid0, v1 = r8 < valid1;
                if constexpr (kGroup) {
                    const uint32_t mine = bit[nt][hc] & who;
                    v0 = (h0.who & mine) && h0.base + r8 <= limit[nt][hc];
                    v1 = (h1.who & mine) && h1.base + r8 <= limit[nt][hc];
                }
                x[hc] = v0 ? sc[nt][hc] * p.scale_log2 : -INFINITY;
                x[hc + 2] = v1 ? sc[nt][hc + 2] * p.scale_log2 : -INFINITY;
            }
            float alpha[2], pr[4];
#pragma unroll
            for (int hc = 0; hc < 2; ++hc) {
                float mx = fmaxf(x[hc], x[hc + 2]);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                const float mn = fmaxf(m[nt][hc], mx);
                const float sub = mn == -INFINITY ? 0.f : mn;  // scores of -inf alone so far: weights 0
                alpha[hc] = fast_exp2(m[nt][hc] - sub);
                m[nt][hc] = mn;
                pr[hc] = fast_exp2(x[hc] - sub);
                pr[hc + 2] = fast_exp2(x[hc + 2] - sub);
                l[nt][hc] = l[nt][hc] * alpha[hc] + pr[hc] + pr[hc + 2];
            }
            if (alpha[0] != 1.f || alpha[1] != 1.f) {
#pragma unroll
                for (int mt = 0; mt < kKSteps; ++mt) {
                    o[mt][nt][0] *= alpha[0];
                    o[mt][nt][1] *= alpha[1];
                    o[mt][nt][2] *= alpha[0];
                    o[mt][nt][3] *= alpha[1];
                }
            }
            pb[nt][0] = movmatrix_t(kFp8 ? pack_f16(pr[0], pr[1]) : pack_bf16(pr[0], pr[1]));  // keys 0-7
            pb[nt][1] = movmatrix_t(kFp8 ? pack_f16(pr[2], pr[3]) : pack_bf16(pr[2], pr[3]));  // keys 8-15
        }
        // ---- O^T += V^T P^T
        if constexpr (kFp8) {
            // keys 2c, 2c+1, 8+2c, 9+2c; dims [16 r8, 16 r8 + 16): 4 x 4 byte blocks transposed
            const uint4 w0 = lds128(vb + sw128(2 * c4, r8)), w1 = lds128(vb + sw128(2 * c4 + 1, r8));
            const uint4 w2 = lds128(vb + sw128(8 + 2 * c4, r8)), w3 = lds128(vb + sw128(9 + 2 * c4, r8));
            const uint32_t k0w[4] = {w0.x, w0.y, w0.z, w0.w}, k1w[4] = {w1.x, w1.y, w1.z, w1.w};
            const uint32_t k2w[4] = {w2.x, w2.y, w2.z, w2.w}, k3w[4] = {w3.x, w3.y, w3.z, w3.w};
#pragma unroll
            for (int pp = 0; pp < 4; ++pp) {
                const uint32_t x01 = __byte_perm(k0w[pp], k1w[pp], 0x5140), x23 = __byte_perm(k2w[pp], k3w[pp], 0x5140);
                const uint32_t y01 = __byte_perm(k0w[pp], k1w[pp], 0x7362), y23 = __byte_perm(k2w[pp], k3w[pp], 0x7362);
                const uint32_t a0 = e4m3_lo(x01), a1 = e4m3_hi(x01), a2 = e4m3_lo(x23), a3 = e4m3_hi(x23);
                const uint32_t b0 = e4m3_lo(y01), b1 = e4m3_hi(y01), b2 = e4m3_lo(y23), b3 = e4m3_hi(y23);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_f16(o[2 * pp][nt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                    mma_f16(o[2 * pp + 1][nt], b0, b1, b2, b3, pb[nt][0], pb[nt][1]);
                }
            }
        } else {
            const int mi = lane >> 3, tr = (mi >> 1) * 8 + (lane & 7);
#pragma unroll
            for (int mt = 0; mt < kKSteps; ++mt) {
                uint32_t a0, a1, a2, a3;
                ldsm_x4_t(vb + seg_off(tr, mt * 2 + (mi & 1)), a0, a1, a2, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_bf16(o[mt][nt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
            }
        }
        __syncwarp();
        if (i + C::kStages < i1) issue(i + C::kStages, stage);
        cp_async_commit();
    }
    // ---- the warps' results, then the CTAs', join by their maxima
    __syncthreads();  // the ring is idle
    float* mine = reinterpret_cast<float*>(smem) + warp * C::kWarpFloats;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int hc = 0; hc < 2; ++hc) {
            float lt = l[nt][hc];
            lt += __shfl_xor_sync(0xffffffffu, lt, 4);
            lt += __shfl_xor_sync(0xffffffffu, lt, 8);
            lt += __shfl_xor_sync(0xffffffffu, lt, 16);
            const int hh = nt * 8 + c4 * 2 + hc;
            if (lane < 4) {
                mine[C::kCols * D + hh] = m[nt][hc];
                mine[C::kCols * (D + 1) + hh] = lt;
            }
#pragma unroll
            for (int mt = 0; mt < kKSteps; ++mt) {
                // rows of O^T: dims 16 mt + r8 and + 8; over 8-bit tiles 16 r8 + 2 mt and + 1
                const int d0 = kFp8 ? 16 * r8 + 2 * mt : 16 * mt + r8;
                mine[hh * D + d0] = o[mt][nt][hc];
                mine[hh * D + d0 + (kFp8 ? 1 : 8)] = o[mt][nt][hc + 2];
            }
        }
    __syncthreads();
    auto weight = [](float mw, float M) { return mw == -INFINITY ? 0.f : fast_exp2(mw - M); };
    const float* all = reinterpret_cast<const float*>(smem);
    for (int it = tid; it < cols * (D / 4); it += kSaThreads) {
        const int hh = it / (D / 4), c = it % (D / 4) * 4;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < kSaWarps; ++w) M = fmaxf(M, all[w * C::kWarpFloats + C::kCols * D + hh]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kSaWarps; ++w) {
            const float* x = all + w * C::kWarpFloats;
            const float wt = weight(x[C::kCols * D + hh], M);
            const float4 v = *reinterpret_cast<const float4*>(x + hh * D + c);
            L += wt * x[C::kCols * (D + 1) + hh];
            acc.x += wt * v.x, acc.y += wt * v.y, acc.z += wt * v.z, acc.w += wt * v.w;
        }
        *reinterpret_cast<float4*>(own + hh * D + c) = acc;
        if (c == 0) {
            own[C::kCols * D + hh] = M;
            own[C::kCols * (D + 1) + hh] = L;
        }
    }
    if (ncta == 1) __syncthreads();
    else cluster_barrier();
    bool bad = false;
    for (int it = cta * kSaThreads + tid; it < cols * (D / 4); it += ncta * kSaThreads) {
        const int hh = it / (D / 4), c = it % (D / 4) * 4;
        if (kGroup && !(who >> (hh / p.G) & 1 && s_stop[hh / p.G] > 0)) continue;
        // up to kSaJoin CTAs' parts in flight together
        float M = -INFINITY, L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = 0; k0 < ncta; k0 += kSaJoin) {
            float mk[kSaJoin], lk[kSaJoin];
            float4 vk[kSaJoin];
#pragma unroll
            for (int j = 0; j < kSaJoin; ++j) {
                if (k0 + j >= ncta) continue;
                mk[j] = load_cluster(own + C::kCols * D + hh, k0 + j);
                lk[j] = load_cluster(own + C::kCols * (D + 1) + hh, k0 + j);
                vk[j] = load_cluster4(own + hh * D + c, k0 + j);
            }
            float Mn = M;
#pragma unroll
            for (int j = 0; j < kSaJoin; ++j)
                if (k0 + j < ncta) Mn = fmaxf(Mn, mk[j]);
            const float keep = weight(M, Mn);
            M = Mn;
            L *= keep, acc.x *= keep, acc.y *= keep, acc.z *= keep, acc.w *= keep;
#pragma unroll
            for (int j = 0; j < kSaJoin; ++j) {
                if (k0 + j >= ncta) continue;
                const float wt = weight(mk[j], M);
                L += wt * lk[j];
                acc.x += wt * vk[j].x, acc.y += wt * vk[j].y, acc.z += wt * vk[j].z, acc.w += wt * vk[j].w;
            }
        }
        const float inv = p.v_scale / L;
        const int64_t row = row_of(hh);
        if (kGroup) bad |= !(fabsf(acc.x) + fabsf(acc.y) + fabsf(acc.z) + fabsf(acc.w) <= 3.4e38f);
        *reinterpret_cast<uint2*>(p.out + row * D + c) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
        if (p.lse && c == 0) p.lse[row] = (M + __log2f(L)) * 0.69314718055994531f;
    }
    if (kGroup && pass == 0 && bad)
        for (int k = 0; k < ncta; ++k) store_cluster(&s_bad, k, 1u);
    // no CTA goes on (or leaves) while another reads its shared memory
    if (ncta == 1) {
        if (!kGroup) return;
        __syncthreads();
    } else {
        cluster_barrier();
    }
    if (!kGroup || ntok == 1 || s_bad == 0 || pass == ntok) return;
    }
}

template <int D, int NT, bool kFp8, bool kGroup>
cudaError_t go(const SparseAttnParams& p, int num_sms, cudaStream_t stream) {
    auto kern = sparse_attn_kernel<D, NT, kFp8, kGroup>;
    const int smem = SaCfg<D, NT, kFp8>::kSmem + (kGroup ? 4 * p.list_cap : 0);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t groups = kGroup ? (int64_t)p.num_tokens / p.group + p.num_reqs : p.num_tokens;
    const int64_t units = groups * p.Hkv;
    const int tiles = (int)std::min<int64_t>(((int64_t)p.num_pages * p.bs + kSaTile - 1) / kSaTile, 1 << 30);
    int n = 1;
    while (n < 8 && units * n < (int64_t)num_sms * 4 && tiles >= n * kSaWarps * 4) n *= 2;

    return launch_cluster(kern, dim3((unsigned)(n * groups), p.Hkv), dim3(kSaThreads), smem, n, stream, p);
}

template <int D, bool kFp8>
cudaError_t by_columns(const SparseAttnParams& p, int num_sms, cudaStream_t stream) {
    const int cols = p.group * p.G;
    if (p.group == 1)
        return cols > 8 ? go<D, 2, kFp8, false>(p, num_sms, stream) : go<D, 1, kFp8, false>(p, num_sms, stream);
    return cols > 16  ? go<D, 4, kFp8, true>(p, num_sms, stream)
           : cols > 8 ? go<D, 2, kFp8, true>(p, num_sms, stream)
                      : go<D, 1, kFp8, true>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_sparse_attn(SparseAttnParams p, int head_dim, bool fp8, int num_sms, cudaStream_t stream) {
    // Tokens of one request taken together: about as many as a request has on
    // average, at most kSaGroup and 32 columns; where that leaves fewer groups
    // than tokens (some groups are empty), and the bit maps and lists fit.
    int group = 1;
    while (group < kSaGroup && group * p.num_reqs < p.num_tokens && 2 * group * p.G <= 32) group *= 2;
    const int64_t pages = ((int64_t)p.max_seq_len + p.bs - 1) / p.bs;
    const int64_t cap = std::min<int64_t>((int64_t)group * p.num_pages, pages);
    if (p.num_tokens / group + p.num_reqs >= p.num_tokens || pages > 32 * 1024 || cap > 4096) group = 1;
    p.group = group;
    p.list_cap = (int)cap;
    if (fp8) return by_columns<128, true>(p, num_sms, stream);
    return head_dim == 128 ? by_columns<128, false>(p, num_sms, stream)
                           : by_columns<64, false>(p, num_sms, stream);
}

}  // namespace pka
