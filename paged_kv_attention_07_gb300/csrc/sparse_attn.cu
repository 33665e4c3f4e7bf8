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
// one contiguous tile that a TMA box brings into a warp's own ring of stages
// (all 128-byte column segments of the rows with one copy). A warp owns a
// contiguous run of tiles and never waits for another: its lanes hold the
// cache rows of its next 32 pages (list entry -> block table -> row), a tile's
// row is one shuffle away. The work of one (token, kv head) is split over the
// 4 warps of a CTA and the CTAs of a cluster; the warps' (m, l, O) join in
// shared memory and the CTAs' over distributed shared memory, so there is one
// launch and nothing partial goes to memory.
//
// Math per tile as in the split-KV decode (bf16 operands, fp32 accumulation):
//   S^T[16 keys x 8 heads] = K Q^T;  online softmax per head;  O^T += V^T P^T
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

template <int D, int NT, bool kFp8>
struct SaCfg {
    static constexpr int kRowBytes = D * (kFp8 ? 1 : 2);
    static constexpr int kTileBytes = kSaTile * kRowBytes;
    static constexpr int kStageBytes = 2 * kTileBytes;  // K + V
    static constexpr int kStages = 3;
    static constexpr int kRing = kSaWarps * kStages * kStageBytes;
    static constexpr int kHeads = NT * 8;
    // the join: each warp's m, l and O (over the ring), and the CTA's own
    static constexpr int kWarpFloats = kHeads * (D + 2);
    static constexpr int kJoin = kSaWarps * kWarpFloats * 4;
    static constexpr int kBody = kRing > kJoin ? kRing : kJoin;
    static constexpr int kSmem = 1024 /*align*/ + kBody + kWarpFloats * 4 + kSaWarps * kStages * 8;
};

PKA_DEVICE uint32_t e4m3_lo(uint32_t w) { return e4m3x2_to_f16x2(w & 0xffffu); }
PKA_DEVICE uint32_t e4m3_hi(uint32_t w) { return e4m3x2_to_f16x2(w >> 16); }

// Row `tr`, 16-byte chunk c of a bf16 tile: 128-byte column segments of 16
// rows one after another, each in the 128-byte swizzle.
PKA_DEVICE uint32_t seg_off(int tr, int c) { return sw128((uint32_t)((c >> 3) * kSaTile + tr), (uint32_t)(c & 7)); }

template <int D, int NT, bool kFp8>
__global__ void __launch_bounds__(kSaThreads, kFp8 && NT == 1 ? 4 : 2)
    sparse_attn_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       const SparseAttnParams p) {
    using C = SaCfg<D, NT, kFp8>;
    constexpr int kKSteps = D / 16;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int s_stop;
    grid_dep_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c4 = lane & 3, r8 = lane >> 2;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* own = reinterpret_cast<float*>(smem + C::kBody);  // this CTA's O [kHeads][D], m, l
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBody + C::kWarpFloats * 4) + warp * C::kStages;
    if (lane == 0) {
        for (int s = 0; s < C::kStages; ++s) mbar_init(&full[s], 1);
        fence_barrier_init();
        if (warp == 0) {
            tma_prefetch_desc(&kmap);
            tma_prefetch_desc(&vmap);
        }
    }
    if (tid == 0) s_stop = p.num_pages;
    __syncthreads();
    grid_dep_wait();

    const int ncta = (int)cluster_size(), cta = (int)cluster_rank();
    const int g = blockIdx.y, t = (int)(blockIdx.x / (unsigned)ncta);
    const TokenPlace at = place_of(p.qsl, p.seq_lens, p.num_reqs, t);
    const int r = at.r;
    if (r < 0) return;  // a row behind the last sequence
    const long long pos = (long long)at.len - at.q1 + t;
    const bool bad = t < at.q0 || pos < 0 || pos >= at.len || at.len > p.max_seq_len;
    if (bad) {
        if (tid == 0 && cta == 0 && g == 0) set_error(p.err, PKA_DEVERR_SEQ_LEN);
        return;
    }
    // ---- the list: it ends at its first negative entry; entries ascend and none is past the own page
    const int own_page = (int)pos / p.bs;
    const int32_t* sel = p.sel + ((int64_t)t * p.Hkv + g) * p.num_pages;
    for (int i = tid; i < p.num_pages; i += kSaThreads) {
        const int e = __ldg(sel + i), before = i ? __ldg(sel + i - 1) : -1;
        if (e <= before || e > own_page) {  // e < 0 among them, before its first occurrence is kept
            atomicMin(&s_stop, i);
            break;
        }
    }
    __syncthreads();
    const int count = s_stop;
    if (cta == 0 && tid == 0 && count < p.num_pages && __ldg(sel + count) >= 0) set_error(p.err, PKA_DEVERR_INDEX);
    int keys = count * p.bs;
    if (count > 0 && __ldg(sel + count - 1) == own_page) keys += (int)pos % p.bs + 1 - p.bs;
    const int64_t row0 = (int64_t)t * p.Hq + g * p.G;  // first output row
    if (keys == 0) {
        if (cta == 0) {
            for (int i = tid; i < p.G * D / 8; i += kSaThreads)
                reinterpret_cast<uint4*>(p.out + row0 * D)[i] = make_uint4(0, 0, 0, 0);
            if (p.lse && tid < p.G) p.lse[row0 + tid] = -INFINITY;
        }
        return;
    }
    const int ntiles = (keys + kSaTile - 1) / kSaTile;
    const int part = cta * kSaWarps + warp, parts = ncta * kSaWarps;
    const int i0 = (int)((int64_t)ntiles * part / parts), i1 = (int)((int64_t)ntiles * (part + 1) / parts);

    // ---- this warp's loads
    const uint64_t pol = policy_evict_first();
    uint8_t* ring = smem + warp * C::kStages * C::kStageBytes;
    const int boxr = min(p.bs, kSaTile);
    int page0 = -32, rows = 0;  // lane l holds the first cache row of listed page page0 + l
    uint32_t ld_it = 0, cs_it = 0;
    auto issue = [&](int i) {
        const int first = i * kSaTile / p.bs;
        if (first + kSaTile / boxr > page0 + 32) {
            page0 = first;
            const int j = page0 + lane;
            int blk = 0;
            if (j < count) {
                blk = __ldg(p.block_table + (int64_t)r * p.max_blocks + __ldg(sel + j));
                if (blk < 0 || blk >= p.num_blocks) {
                    set_error(p.err, PKA_DEVERR_BLOCK_ID);
                    blk = 0;
                }
            }
            rows = (blk * p.Hkv + g) * p.bs;
        }
        const int ra = __shfl_sync(0xffffffffu, rows, first - page0) + i * kSaTile % p.bs;
        const int rb = __shfl_sync(0xffffffffu, rows, (first + 1 - page0) & 31);  // bs == 8: the tile's second page
        if (lane == 0) {
            const int stage = ld_it % C::kStages;
            uint8_t* kdst = ring + stage * C::kStageBytes;
            uint8_t* vdst = kdst + C::kTileBytes;
            const int nbox = boxr < kSaTile && i * kSaTile + boxr < keys ? 2 : 1;
            fence_proxy_async_smem();
            mbar_arrive_expect_tx(&full[stage], (uint32_t)(2 * nbox * boxr * C::kRowBytes));
            for (int b = 0; b < nbox; ++b) {
                const int row = b ? rb : ra;
                if constexpr (kFp8) {
                    tma_load_2d(kdst + b * boxr * 128, &kmap, &full[stage], 0, row, pol);
                    tma_load_2d(vdst + b * boxr * 128, &vmap, &full[stage], 0, row, pol);
                } else if (nbox == 1 && boxr == kSaTile) {
                    tma_load_3d(kdst, &kmap, &full[stage], 0, row, 0, pol);
                    tma_load_3d(vdst, &vmap, &full[stage], 0, row, 0, pol);
                } else {  // boxes of 8 rows and one segment
#pragma unroll
                    for (int sg = 0; sg < D / 64; ++sg) {
                        const int off = (sg * kSaTile + b * boxr) * 128;
                        tma_load_3d(kdst + off, &kmap, &full[stage], 0, row, sg, pol);
                        tma_load_3d(vdst + off, &vmap, &full[stage], 0, row, sg, pol);
                    }
                }
            }
        }
        ++ld_it;
        __syncwarp();
    };
    for (int i = i0; i < i1 && i < i0 + C::kStages; ++i) issue(i);

    // ---- Q^T fragments: head n of the group, zero beyond G
    uint32_t qf[NT][kKSteps][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int hh = nt * 8 + r8;
        const bool ok = hh < p.G;
        const __nv_bfloat16* qrow = p.q + (row0 + (ok ? hh : 0)) * D;
        if constexpr (kFp8) {  // k-step ks holds dims 32 c4 + 4 ks .. + 3, as the codes are read
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint4 v = ok ? __ldg(reinterpret_cast<const uint4*>(qrow + 32 * c4) + j) : make_uint4(0, 0, 0, 0);
                qf[nt][2 * j][0] = bf16x2_to_f16x2(v.x);
                qf[nt][2 * j][1] = bf16x2_to_f16x2(v.y);
                qf[nt][2 * j + 1][0] = bf16x2_to_f16x2(v.z);
                qf[nt][2 * j + 1][1] = bf16x2_to_f16x2(v.w);
            }
        } else {
#pragma unroll
            for (int ks = 0; ks < kKSteps; ++ks) {
                qf[nt][ks][0] = ok ? __ldg(reinterpret_cast<const uint32_t*>(qrow) + ks * 8 + c4) : 0u;
                qf[nt][ks][1] = ok ? __ldg(reinterpret_cast<const uint32_t*>(qrow) + ks * 8 + 4 + c4) : 0u;
            }
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

    for (int i = i0; i < i1; ++i) {
        const int stage = cs_it % C::kStages;
        if (!mbar_wait_warp(&full[stage], (cs_it / C::kStages) & 1, p.err)) break;
        ++cs_it;
        uint8_t* kt = ring + stage * C::kStageBytes;
        uint8_t* vt = kt + C::kTileBytes;
        const int valid = min(kSaTile, keys - i * kSaTile);
        if (valid < kSaTile) {  // V rows past the end may hold anything: zeros instead
            for (int ci = lane; ci < (kSaTile - valid) * (C::kRowBytes / 16); ci += 32) {
                const int tr = valid + ci / (C::kRowBytes / 16), c = ci % (C::kRowBytes / 16);
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
                for (int k = 0; k < 4; ++k) {
                    const uint32_t a0 = e4m3_lo(wl[k]), a1 = e4m3_lo(wh[k]), a2 = e4m3_hi(wl[k]), a3 = e4m3_hi(wh[k]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_f16(sc[nt], a0, a1, a2, a3, qf[nt][4 * jc + k][0], qf[nt][4 * jc + k][1]);
                }
            }
        } else {
            const int mi = lane >> 3, tr = (mi & 1) * 8 + (lane & 7);
#pragma unroll
            for (int ks = 0; ks < kKSteps; ++ks) {
                uint32_t a0, a1, a2, a3;
                ldsm_x4(kb + seg_off(tr, ks * 2 + (mi >> 1)), a0, a1, a2, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_bf16(sc[nt], a0, a1, a2, a3, qf[nt][ks][0], qf[nt][ks][1]);
            }
        }
        // ---- online softmax in the log2 domain; keys past the end weigh nothing
        const bool v0 = r8 < valid, v1 = r8 + 8 < valid;
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float x[4] = {v0 ? sc[nt][0] * p.scale_log2 : -INFINITY, v0 ? sc[nt][1] * p.scale_log2 : -INFINITY,
                                v1 ? sc[nt][2] * p.scale_log2 : -INFINITY, v1 ? sc[nt][3] * p.scale_log2 : -INFINITY};
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
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_f16(o[2 * pp][nt], e4m3_lo(x01), e4m3_hi(x01), e4m3_lo(x23), e4m3_hi(x23), pb[nt][0], pb[nt][1]);
                    mma_f16(o[2 * pp + 1][nt], e4m3_lo(y01), e4m3_hi(y01), e4m3_lo(y23), e4m3_hi(y23), pb[nt][0],
                            pb[nt][1]);
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
        if (i + C::kStages < i1) issue(i + C::kStages);
    }
    // after a wait that gave up: no copy may outlive the CTA
    while (cs_it < ld_it) {
        mbar_wait_warp(&full[cs_it % C::kStages], (cs_it / C::kStages) & 1, p.err);
        ++cs_it;
    }

    // ---- the warps' results, then the CTA's, join by their maxima
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
                mine[C::kHeads * D + hh] = m[nt][hc];
                mine[C::kHeads * (D + 1) + hh] = lt;
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
    for (int it = tid; it < p.G * (D / 4); it += kSaThreads) {
        const int hh = it / (D / 4), c = it % (D / 4) * 4;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < kSaWarps; ++w) M = fmaxf(M, all[w * C::kWarpFloats + C::kHeads * D + hh]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kSaWarps; ++w) {
            const float* x = all + w * C::kWarpFloats;
            const float wt = weight(x[C::kHeads * D + hh], M);
            const float4 v = *reinterpret_cast<const float4*>(x + hh * D + c);
            L += wt * x[C::kHeads * (D + 1) + hh];
            acc.x += wt * v.x, acc.y += wt * v.y, acc.z += wt * v.z, acc.w += wt * v.w;
        }
        *reinterpret_cast<float4*>(own + hh * D + c) = acc;
        if (c == 0) {
            own[C::kHeads * D + hh] = M;
            own[C::kHeads * (D + 1) + hh] = L;
        }
    }
    cluster_barrier();
    for (int it = cta * kSaThreads + tid; it < p.G * (D / 4); it += ncta * kSaThreads) {
        const int hh = it / (D / 4), c = it % (D / 4) * 4;
        float M = -INFINITY, L = 0.f;
        for (int k = 0; k < ncta; ++k) M = fmaxf(M, load_cluster(own + C::kHeads * D + hh, k));
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < ncta; ++k) {
            const float wt = weight(load_cluster(own + C::kHeads * D + hh, k), M);
            const float4 v = load_cluster4(own + hh * D + c, k);
            L += wt * load_cluster(own + C::kHeads * (D + 1) + hh, k);
            acc.x += wt * v.x, acc.y += wt * v.y, acc.z += wt * v.z, acc.w += wt * v.w;
        }
        const float inv = p.v_scale / L;
        *reinterpret_cast<uint2*>(p.out + (row0 + hh) * D + c) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
        if (p.lse && c == 0) p.lse[row0 + hh] = (M + __log2f(L)) * 0.69314718055994531f;
    }
    cluster_barrier();  // no CTA leaves while another reads its shared memory
}

template <int D, int NT, bool kFp8>
cudaError_t go(const CUtensorMap& km, const CUtensorMap& vm, const SparseAttnParams& p, int num_sms,
               cudaStream_t stream) {
    using C = SaCfg<D, NT, kFp8>;
    auto kern = sparse_attn_kernel<D, NT, kFp8>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)p.num_tokens * p.Hkv;
    const int tiles = (int)std::min<int64_t>(((int64_t)p.num_pages * p.bs + kSaTile - 1) / kSaTile, 1 << 30);
    int n = 1;
    while (n < 8 && units * n < (int64_t)num_sms * 8 && tiles >= n * kSaWarps * 4) n *= 2;
    return launch_cluster(kern, dim3((unsigned)n * (unsigned)p.num_tokens, p.Hkv), dim3(kSaThreads), C::kSmem, n, stream,
                          km, vm, p);
}

}  // namespace

cudaError_t launch_sparse_attn(const CUtensorMap& km, const CUtensorMap& vm, const SparseAttnParams& p, int head_dim,
                               bool fp8, int num_sms, cudaStream_t stream) {
    const bool two = p.G > 8;
    if (fp8)
        return two ? go<128, 2, true>(km, vm, p, num_sms, stream) : go<128, 1, true>(km, vm, p, num_sms, stream);
    if (head_dim == 128)
        return two ? go<128, 2, false>(km, vm, p, num_sms, stream) : go<128, 1, false>(km, vm, p, num_sms, stream);
    return two ? go<64, 2, false>(km, vm, p, num_sms, stream) : go<64, 1, false>(km, vm, p, num_sms, stream);
}

}  // namespace pka
