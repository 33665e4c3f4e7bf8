// sparse_attn.cu -- attention of each new token over the pages listed for it.
//
// Token t at position p of request r, kv head g with its G query heads, the
// ascending list of pages e_0 < e_1 < ... <= p / bs:
//     s_j = scale * <q, K_j>,  out = sum_j softmax(s)_j V_j,  lse = log sum_j exp(s_j)
// over the keys j <= p of the listed pages. Only the token's own page can be
// partly filled and it comes last, so the listed keys are one run of
// (count - 1) * bs + tail keys: key i of the run lies in page e[i / bs].
//
// HBM-bound: every listed page is read once, 8 keys of one (page, kv head) are
// contiguous, and 16-byte asynchronous copies bring a tile of 16 (bf16) or 32
// (8-bit) keys into a warp's own ring of stages (swizzled by the row, so that the
// fragments' reads meet no bank twice). Tile copies by TMA boxes read a full
// batch as fast, but one lane's TMA instructions take 390 to 750 cycles of the
// warp's time per tile, more than the products; 32 lanes' copies some 80. A warp
// owns a contiguous run of tiles and never waits for another: its lanes hold the
// cache rows of its next 32 pages (list entry -> block table -> row), a tile's
// rows are a shuffle away. The work of one (token, kv head) is split over the
// 4 or 8 warps of a CTA and the CTAs of a cluster; the warps' (m, l, O) join in
// shared memory and the CTAs' over distributed shared memory, so there is one
// launch and nothing partial goes to memory.
//
// Each token reads its own pages, tokens of one request mostly the same ones
// through L2. (Taking such tokens together over their united lists was measured:
// 96 x 4 tokens 238 -> 216 us, but 24 x 4 tokens 46 -> 52 us and 8-bit caches
// 143 -> 201 us, with P as one bf16 number: the lists' union and the registers of
// more columns cost what the shared reads save.)
//
// Math per tile (tensor cores, fp32 accumulation):
//   S^T[keys x 8 columns] = K Q^T;  online softmax per column;  O^T += V^T P^T
// bf16: P is two bf16 numbers, the largest one below it and the rest, off by 2^-15
// of each weight: the result's error is that of its own rounding. (Rounded to one:
// 0.0021 against 64 bits instead of 0.0017; 96 x 4 tokens 225 us instead of 247, 96
// requests 120.2 and 121.2, one 8.5 and 8.7.) Both are positive, so that an infinite
// value is not taken off itself.
// 8-bit: the codes are widened to f16 (exact) in registers, q is f16 in units of a
// power of two per query head (its largest element is 128 to 256 units: bf16's
// bits are kept down to 2^-22 of it), and P is f16, 2^-11 of each weight or 2^-40 of
// the largest: weights are in units of 2^-15, the largest 2^15 of them, so that
// the sum of many small ones is not lost below f16's least number. (The codes as e4m3 operands,
// with q and P as two e4m3 numbers each, need no conversions but twice the
// products: 24 x 4 tokens 36 us, 27 us this way.)
//
// Measured: 96 requests, 4 kv heads, 64 pages of 64 tokens each, bf16: 121 us, 6.6
// TB/s; 8-bit: 68 us, 5.9 TB/s. One request of 8 kv heads, bf16: 8.7 us: 3 until
// the first tiles are there (launch, request, block table, tile), 3 of tiles, 2 of joins.
#include "common.cuh"
#include "params.cuh"

namespace pka {

namespace {

constexpr int kSaJoin = 8;   // CTAs' results read together

template <int D, int NT, bool kFp8, int kWarps>
struct SaCfg {
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kTile = kFp8 ? 32 : 16;  // keys of a tile
    static constexpr int kOctets = kTile / 8;     // eight keys each, of one page
    static constexpr int kRowBytes = D * (kFp8 ? 1 : 2);
    static constexpr int kTileBytes = kTile * kRowBytes;
    static constexpr int kStageBytes = 2 * kTileBytes;  // K + V
    // Heads of 64 elements have tiles of half the bytes: more of them in flight (96
    // requests 65 us, 68 us with 3 stages and 2 CTAs per SM; 16 requests 15.2 and 16.6).
    static constexpr int kStages = kFp8 ? 2 : D == 64 ? 4 : 3;
    static constexpr int kMinBlocks = kWarps == 8 ? 1 : (kFp8 || D == 64) && NT == 1 ? 3 : 2;  // CTAs per SM
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    static constexpr int kCols = NT * 8;
    static constexpr float kWeightPower = kFp8 ? 15.f : 0.f;  // weights (and l, O) in units of 2^-15: P fills f16's range
    // the join: each warp's m, l and O (over the ring), and the CTA's own
    static constexpr int kWarpFloats = kCols * (D + 2);
    static constexpr int kJoin = kWarps * kWarpFloats * 4;
    static constexpr int kBody = kRing > kJoin ? kRing : kJoin;
    static constexpr int kSmem = 1024 /*align*/ + kBody + kWarpFloats * 4;
};

// Row `row`, 16-byte chunk c of a tile of `tile` rows: 128-byte column segments of
// all its rows one after another, each in the 128-byte swizzle.
template <int kTile>
PKA_DEVICE uint32_t seg_off(int row, int c) {
    return sw128((uint32_t)((c >> 3) * kTile + row), (uint32_t)(c & 7));
}

// Four E4M3 codes to two f16 pairs (exact).
PKA_DEVICE void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// The float of the largest bf16 number below p > 0 (in its high half; zero for zero).
PKA_DEVICE uint32_t below(float p) { return max(__float_as_uint(p), 1u) - 1; }

template <int D, int NT, bool kFp8, int kWarps>
__global__ void __launch_bounds__(kWarps * 32, SaCfg<D, NT, kFp8, kWarps>::kMinBlocks)
    sparse_attn_kernel(const SparseAttnParams p) {
    using C = SaCfg<D, NT, kFp8, kWarps>;
    constexpr int kThreads = C::kThreads;
    constexpr int kTile = C::kTile, kOctets = C::kOctets;
    constexpr int kMTiles = kTile / 16;  // of S^T: 16 keys each
    constexpr int kKSteps = D / 16;      // m-tiles of O^T (and k-steps of S^T over bf16)
    extern __shared__ uint8_t smem_raw[];
    __shared__ int s_stop;
    grid_dep_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c4 = lane & 3, r8 = lane >> 2;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* own = reinterpret_cast<float*>(smem + C::kBody);  // this CTA's O [kCols][D], m, l
    if (tid == 0) s_stop = p.num_pages;
    __syncthreads();
    grid_dep_wait();

    // ---- the token's request and position (the same for the whole cluster)
    const int ncta = (int)cluster_size(), cta = (int)cluster_rank();
    const int g = blockIdx.y, t0 = (int)(blockIdx.x / (unsigned)ncta);
    const int32_t* sel = p.sel + ((int64_t)t0 * p.Hkv + g) * p.num_pages;
    int entry = -1, before = -1;  // this thread's first of the list, on its way meanwhile
    if (tid < p.num_pages) {
        entry = __ldg(sel + tid);
        if (tid) before = __ldg(sel + tid - 1);
    }
    const TokenPlace at = place_of(p.qsl, p.seq_lens, p.num_reqs, t0);
    if (at.r < 0) return;  // a row behind the last sequence
    const long long pos = (long long)at.len - at.q1 + t0;
    if (t0 < at.q0 || pos < 0 || pos >= at.len || at.len > p.max_seq_len) {
        if (tid == 0 && cta == 0 && g == 0) set_error(p.err, PKA_DEVERR_SEQ_LEN);
        return;
    }
    const int own_page = (int)pos >> p.bs_log2;
    const int64_t row0 = (int64_t)t0 * p.Hq + g * p.G;  // first output row

    // ---- the list: it ends at its first negative entry; entries ascend and none is past the own page
    for (int i = tid; i < p.num_pages;) {
        if (entry <= before || entry > own_page) {  // negative ones among them
            atomicMin(&s_stop, i);
            break;
        }
        if ((i += kThreads) >= p.num_pages) break;
        entry = __ldg(sel + i);
        before = __ldg(sel + i - 1);
    }
    __syncthreads();
    const int count = s_stop;
    if (cta == 0 && tid == 0 && count < p.num_pages && __ldg(sel + count) >= 0) set_error(p.err, PKA_DEVERR_INDEX);
    if (count == 0) {  // nothing to read
        if (cta == 0) {
            for (int i = tid; i < p.G * D / 8; i += kThreads)
                reinterpret_cast<uint4*>(p.out + row0 * D)[i] = make_uint4(0, 0, 0, 0);
            if (p.lse && tid < p.G) p.lse[row0 + tid] = -INFINITY;
        }
        return;
    }
    const bool tail = __ldg(sel + count - 1) == own_page;
    const int keys = count * p.bs - (tail ? p.bs - 1 - ((int)pos & (p.bs - 1)) : 0);
    const int ntiles = (keys + kTile - 1) / kTile;
    const int part = cta * kWarps + warp, parts = ncta * kWarps;
    // (parts is a power of two up to 64, ntiles below 2^31 / kTile)
    const int parts_log2 = 31 - __clz(parts);
    const int i0 = (ntiles >> parts_log2) * part + (((ntiles & (parts - 1)) * part) >> parts_log2);
    const int i1 = (ntiles >> parts_log2) * (part + 1) + (((ntiles & (parts - 1)) * (part + 1)) >> parts_log2);

    // ---- this warp's loads: a step copies 32 pieces of 16 bytes, kRows rows
    constexpr int kPieces = C::kRowBytes / 16, kRows = 32 / kPieces, kSteps = 8 / kRows;  // steps of an octet
    const uint64_t pol = policy_evict_first();
    const uint8_t* kc = static_cast<const uint8_t*>(p.k_cache) + lane * 16;
    const uint8_t* vc = static_cast<const uint8_t*>(p.v_cache) + lane * 16;
    uint32_t place[kSteps];  // of a step in an octet; 1024 bytes on, the next octet
#pragma unroll
    for (int j = 0; j < kSteps; ++j) place[j] = seg_off<kTile>(j * kRows + lane / kPieces, lane % kPieces);
    uint8_t* ring = smem + warp * C::kStages * C::kStageBytes;
    int page0 = -32, rows = 0;  // lane l holds the first cache row of listed page page0 + l
    auto issue = [&](int i, int stage) {
        const int first = (i * kTile) >> p.bs_log2;
        if ((i * kTile + kTile - 1) >> p.bs_log2 >= page0 + 32) {
            page0 = first;
            const int j = page0 + lane;
            int blk = 0;
            if (j < count) {
                blk = __ldg(p.block_table + (int64_t)at.r * p.max_blocks + __ldg(sel + j));
                if (blk < 0 || blk >= p.num_blocks) {
                    set_error(p.err, PKA_DEVERR_BLOCK_ID);
                    blk = 0;
                }
            }
            rows = (blk * p.Hkv + g) * p.bs;
        }
        const uint32_t kdst = smem_u32(ring + stage * C::kStageBytes), vdst = kdst + C::kTileBytes;
#pragma unroll
        for (int o = 0; o < kOctets; ++o) {
            const int key = i * kTile + 8 * o, off = key & (p.bs - 1);
            const int from = ((key >> p.bs_log2) - page0) & 31;
            const int64_t src = (int64_t)(__shfl_sync(0xffffffffu, rows, from) + off) * C::kRowBytes;
            if (key >= keys) continue;
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
                cp_async_16_hint(kdst + place[j] + o * 1024, kc + src + j * 512, pol);
                cp_async_16_hint(vdst + place[j] + o * 1024, vc + src + j * 512, pol);
            }
        }
    };
#pragma unroll
    for (int s = 0; s < C::kStages; ++s) {
        if (i0 + s < i1) issue(i0 + s, s);
        cp_async_commit();  // (a group per tile, empty behind the last)
    }

    // ---- Q^T fragments: column n, zero behind the last; [k-step of 16 elements][2]
    uint32_t qf[NT][kKSteps][2];
    float factor[NT][2];  // 8-bit: this lane's columns of S^T, from their units to the log2 domain
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int n = nt * 8 + r8;
        const bool ok = n < p.G;
        const __nv_bfloat16* qrow = p.q + (row0 + (ok ? n : 0)) * D;
        if constexpr (kFp8) {  // k-step s of this lane: elements 32 c4 + 8 s .. + 7, as the codes are read
            float x[32];
            float a = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint4 v = ok ? __ldg(reinterpret_cast<const uint4*>(qrow + 32 * c4) + j) : make_uint4(0, 0, 0, 0);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[8 * j + 2 * i] = bf16_lo(w[i]);
                    x[8 * j + 2 * i + 1] = bf16_hi(w[i]);
                }
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) a = fmaxf(a, fabsf(x[j]));
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
            int e = 0;
            if (a <= 3.4e38f) frexpf(a, &e);  // a < 2^e
            e = max(e - 8, -100);
            const float unit = exp2i(-e);
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = fabsf(x[j]) <= 3.4e38f ? x[j] * unit : __int_as_float(0x7fffffff);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                qf[nt][ks][0] = pack_f16(x[4 * ks], x[4 * ks + 1]);
                qf[nt][ks][1] = pack_f16(x[4 * ks + 2], x[4 * ks + 3]);
            }
            const float f = p.scale_log2 * exp2i(e);
#pragma unroll
            for (int hc = 0; hc < 2; ++hc) factor[nt][hc] = __shfl_sync(0xffffffffu, f, (c4 * 2 + hc) * 4);
        } else {
#pragma unroll
            for (int ks = 0; ks < kKSteps; ++ks) {
                qf[nt][ks][0] = ok ? __ldg(reinterpret_cast<const uint32_t*>(qrow) + ks * 8 + c4) : 0u;
                qf[nt][ks][1] = ok ? __ldg(reinterpret_cast<const uint32_t*>(qrow) + ks * 8 + 4 + c4) : 0u;
            }
            factor[nt][0] = factor[nt][1] = p.scale_log2;
        }
    }
    float o[kKSteps][NT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int mt = 0; mt < kKSteps; ++mt) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
    }
    int stage = 0;
    for (int i = i0; i < i1; ++i) {
        cp_async_wait<C::kStages - 1>();
        __syncwarp();
        uint8_t* kt = ring + stage * C::kStageBytes;
        uint8_t* vt = kt + C::kTileBytes;
        // valid keys of each octet; the others' values may be anything: zeros instead
        int valid[kOctets];
#pragma unroll
        for (int q = 0; q < kOctets; ++q) valid[q] = min(8, max(0, keys - i * kTile - 8 * q));
        if (valid[kOctets - 1] < 8) {
#pragma unroll
            for (int q = 0; q < kOctets; ++q)
                for (int ci = valid[q] * kPieces + lane; ci < 8 * kPieces; ci += 32)
                    *reinterpret_cast<uint4*>(vt + q * 1024 + seg_off<kTile>(ci / kPieces, ci % kPieces)) =
                        make_uint4(0, 0, 0, 0);
            __syncwarp();
        }
        const uint32_t kb = smem_u32(kt), vb = smem_u32(vt);

        // ---- S^T = K Q^T: rows r8 (octet 2 t) and r8 + 8 (octet 2 t + 1) of m-tile t
        float sc[kMTiles][NT][4];
#pragma unroll
        for (int t = 0; t < kMTiles; ++t)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) sc[t][nt][0] = sc[t][nt][1] = sc[t][nt][2] = sc[t][nt][3] = 0.f;
        if constexpr (kFp8) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int jc = 0; jc < 2; ++jc) {
                    const uint4 a = lds128(kb + t * 2048 + sw128(r8, 2 * c4 + jc));
                    const uint4 b = lds128(kb + t * 2048 + sw128(r8 + 8, 2 * c4 + jc));
                    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t a0, a1, a2, a3;
                        widen4(aw[k], a0, a2);
                        widen4(bw[k], a1, a3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_f16(sc[t][nt], a0, a1, a2, a3, qf[nt][4 * jc + k][0], qf[nt][4 * jc + k][1]);
                    }
                }
        } else {
            // two sums side by side: half the length of the chain of products
            float sd[NT][4] = {};
            const int mi = lane >> 3, tr = (mi & 1) * 8 + (lane & 7);
#pragma unroll
            for (int ks = 0; ks < kKSteps; ++ks) {
                uint32_t a0, a1, a2, a3;
                ldsm_x4(kb + seg_off<kTile>(tr, ks * 2 + (mi >> 1)), a0, a1, a2, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_bf16(ks % 2 ? sd[nt] : sc[0][nt], a0, a1, a2, a3, qf[nt][ks][0], qf[nt][ks][1]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[0][nt][e] += sd[nt][e];
        }
        // ---- online softmax in the log2 domain; other keys weigh nothing
        uint32_t pb[kOctets][NT];             // P^T fragments
        uint32_t pl[kFp8 ? 1 : kOctets][NT];  // bf16: what these leave of P^T
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float pr[kOctets][2];
            float alpha[2];
#pragma unroll
            for (int hc = 0; hc < 2; ++hc) {
                float mx = -INFINITY;
#pragma unroll
                for (int q = 0; q < kOctets; ++q) {
                    pr[q][hc] = r8 < valid[q] ? sc[q / 2][nt][q % 2 * 2 + hc] * factor[nt][hc] : -INFINITY;
                    mx = fmaxf(mx, pr[q][hc]);
                }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                const float mn = fmaxf(m[nt][hc], mx);
                const float sub = mn == -INFINITY ? 0.f : mn;  // scores of -inf alone so far: weights 0
                alpha[hc] = fast_exp2(m[nt][hc] - sub);
                m[nt][hc] = mn;
                float sum = 0.f;
#pragma unroll
                for (int q = 0; q < kOctets; ++q) {
                    pr[q][hc] = fast_exp2(pr[q][hc] - sub + C::kWeightPower);
                    sum += pr[q][hc];
                }
                l[nt][hc] = l[nt][hc] * alpha[hc] + sum;
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
#pragma unroll
            for (int q = 0; q < kOctets; ++q) {
                if constexpr (kFp8) {
                    pb[q][nt] = movmatrix_t(pack_f16(pr[q][0], pr[q][1]));
                } else {
                    const uint32_t w = __byte_perm(below(pr[q][0]), below(pr[q][1]), 0x7632);
                    pb[q][nt] = movmatrix_t(w);
                    pl[q][nt] = movmatrix_t(pack_bf16(pr[q][0] - bf16_lo(w), pr[q][1] - bf16_hi(w)));
                }
            }
        }
        // ---- O^T += V^T P^T
        if constexpr (kFp8) {
            // keys 16 t + 2c, + 1, + 8, + 9; elements 16 r8 .. + 15 of each, pairs of keys per element:
            // rows of m-tile 2 pp + j are elements 16 r8 + 4 pp + 2 j and + 1
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint32_t row = t * 16 + 2 * c4;
                const uint4 w0 = lds128(vb + sw128(row, r8)), w1 = lds128(vb + sw128(row + 1, r8));
                const uint4 w2 = lds128(vb + sw128(row + 8, r8)), w3 = lds128(vb + sw128(row + 9, r8));
                const uint32_t k0[4] = {w0.x, w0.y, w0.z, w0.w}, k1[4] = {w1.x, w1.y, w1.z, w1.w};
                const uint32_t k2[4] = {w2.x, w2.y, w2.z, w2.w}, k3[4] = {w3.x, w3.y, w3.z, w3.w};
#pragma unroll
                for (int pp = 0; pp < 4; ++pp) {
                    const uint32_t x01 = __byte_perm(k0[pp], k1[pp], 0x5140), x23 = __byte_perm(k2[pp], k3[pp], 0x5140);
                    const uint32_t y01 = __byte_perm(k0[pp], k1[pp], 0x7362), y23 = __byte_perm(k2[pp], k3[pp], 0x7362);
                    uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
                    widen4(x01, a0, a1);
                    widen4(x23, a2, a3);
                    widen4(y01, b0, b1);
                    widen4(y23, b2, b3);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_f16(o[2 * pp][nt], a0, a1, a2, a3, pb[2 * t][nt], pb[2 * t + 1][nt]);
                        mma_f16(o[2 * pp + 1][nt], b0, b1, b2, b3, pb[2 * t][nt], pb[2 * t + 1][nt]);
                    }
                }
            }
        } else {
            const int mi = lane >> 3, tr = (mi >> 1) * 8 + (lane & 7);
#pragma unroll
            for (int mt = 0; mt < kKSteps; ++mt) {
                uint32_t a0, a1, a2, a3;
                ldsm_x4_t(vb + seg_off<kTile>(tr, mt * 2 + (mi & 1)), a0, a1, a2, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_bf16(o[mt][nt], a0, a1, a2, a3, pb[0][nt], pb[1][nt]);
                    mma_bf16(o[mt][nt], a0, a1, a2, a3, pl[0][nt], pl[1][nt]);
                }
            }
        }
        __syncwarp();
        if (i + C::kStages < i1) issue(i + C::kStages, stage);
        cp_async_commit();
        stage = stage + 1 == C::kStages ? 0 : stage + 1;
    }
    cp_async_wait<0>();

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
                // rows of O^T: elements 16 mt + r8 and + 8; over 8-bit tiles 16 r8 + 2 mt and + 1
                const int d0 = kFp8 ? 16 * r8 + 2 * mt : 16 * mt + r8;
                mine[hh * D + d0] = o[mt][nt][hc];
                mine[hh * D + d0 + (kFp8 ? 1 : 8)] = o[mt][nt][hc + 2];
            }
        }
    __syncthreads();
    auto weight = [](float mw, float M) { return mw == -INFINITY ? 0.f : fast_exp2(mw - M); };
    const float* all = reinterpret_cast<const float*>(smem);
    for (int it = tid; it < p.G * (D / 4); it += kThreads) {
        const int hh = it / (D / 4), c = it % (D / 4) * 4;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, all[w * C::kWarpFloats + C::kCols * D + hh]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
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
    for (int it = cta * kThreads + tid; it < p.G * (D / 4); it += ncta * kThreads) {
        const int hh = it / (D / 4), c = it % (D / 4) * 4;
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
        const int64_t row = row0 + hh;
        *reinterpret_cast<uint2*>(p.out + row * D + c) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
        if (p.lse && c == 0) p.lse[row] = (M + __log2f(L * exp2i(-(int)C::kWeightPower))) * 0.69314718055994531f;
    }
    if (ncta > 1) cluster_barrier();  // no CTA leaves while another reads its shared memory
}

template <int D, int NT, bool kFp8, int kWarps>
cudaError_t go(const SparseAttnParams& p, int num_sms, cudaStream_t stream) {
    using C = SaCfg<D, NT, kFp8, kWarps>;
    auto kern = sparse_attn_kernel<D, NT, kFp8, kWarps>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)p.num_tokens * p.Hkv, listed = (int64_t)p.num_pages * p.bs;
    int n = 1;  // CTAs per (token, kv head)
    if (kWarps == 8) {
        // One CTA per SM, all at once, a tile per warp at least. (Clusters of 8
        // such CTAs find room on half of the SMs only: 16 units in clusters of 4 / 8
        // 10.6 / 17.0 us.)
        while (n < 8 && units * n * (n == 4 ? 4 : 2) <= num_sms && listed >= 2 * n * kWarps * C::kTile) n *= 2;
    } else {
        // More CTAs shorten each one's run of tiles but each costs a start of about
        // kStart tiles, and beyond the resident CTAs they run in turns. Measured with
        // 1 / 2 / 4 CTAs: bf16 (P as one number), 64 tiles per warp, 156 units 56 / 66 / 63
        // us, 308 units 117 / 107 / 107, 384 units 125 / 120 / 131; 8-bit, 32 tiles per warp,
        // 156 units 43 / 32 / 37, 280 units 52 / 61 / 57, 612 units 109 / 102 / 111.
        constexpr int64_t kStart = 8;
        const int64_t slots = (int64_t)num_sms * C::kMinBlocks;
        const int64_t tiles = (listed + C::kTile * kWarps - 1) / (C::kTile * kWarps);
        int64_t best = 0;
        for (int c = 1; c <= 8; c *= 2) {
            const int64_t turns = (units * c + slots - 1) / slots;
            const int64_t cost = turns * (kStart + (tiles + c - 1) / c);
            if (c == 1 || cost < best) {
                best = cost;
                n = c;
            }
        }
    }
    return launch_cluster(kern, dim3((unsigned)n * (unsigned)p.num_tokens, p.Hkv), dim3(C::kThreads), C::kSmem, n, stream,
                          p);
}

}  // namespace

cudaError_t launch_sparse_attn(const SparseAttnParams& p, int head_dim, bool fp8, int num_sms, cudaStream_t stream) {
    // CTAs of 8 warps while there is an SM for each (token, kv head), and a tile for each
    // warp, else of 4, several to an SM. Measured, 4096 listed keys each, best cluster of either, 4 / 8 warps:
    // 8 units bf16 9.6 / 8.3 us, 8-bit 8.8 / 7.5; 32 units 15.9 / 15.8, 12.9 / 10.9;
    // 64 units 25.0 / 25.2, 17.7 / 16.4; 128 units 43.8 / 43.2, 27.8 / 25.1 us.
    const bool two = p.G > 8;
    const bool wide = (int64_t)p.num_tokens * p.Hkv <= num_sms && (int64_t)p.num_pages * p.bs >= 256;
    auto by_warps = [&](auto d, auto nt, auto codes) {
        constexpr int D = decltype(d)::value, NT = decltype(nt)::value;
        constexpr bool kFp8 = decltype(codes)::value;
        return wide ? go<D, NT, kFp8, 8>(p, num_sms, stream) : go<D, NT, kFp8, 4>(p, num_sms, stream);
    };
    auto by_columns = [&](auto d, auto codes) {
        return two ? by_warps(d, std::integral_constant<int, 2>{}, codes)
                   : by_warps(d, std::integral_constant<int, 1>{}, codes);
    };
    if (fp8) return by_columns(std::integral_constant<int, 128>{}, std::true_type{});
    if (head_dim == 128) return by_columns(std::integral_constant<int, 128>{}, std::false_type{});
    return by_columns(std::integral_constant<int, 64>{}, std::false_type{});
}

}  // namespace pka
