// beam_select.cu -- the best continuations of each group of beams:
//   score(b, v) = scores[b] + x_b[v] - log sum_u exp(x_b[u])
// and of a group's num_beams * vocab candidates the num_out best.
//
// Within a row the order is that of the logits, so a row's candidates are its
// num_out largest logits (of equal ones the lower tokens), found in the same pass
// that sums the exponentials. A row is cut into slices of one length for all
// rows, a CTA takes (row, slice) parts in turn, and the CTAs of a group are a
// cluster whose first CTA joins the parts' sums and lists through distributed
// shared memory: no workspace, no second launch.
//
// A part goes in tiles of kTile elements held in registers. The first tile gives
// a threshold that at least num_out of its elements reach (the num_out-th of the
// threads' largest), elements above the threshold are collected in shared memory
// and cut back to the best num_out now and then. A key is the logit's order in the
// upper and the token's complement in the lower 32 bits: keys are distinct, the
// larger one is the better, and the collected order does not matter. Where too
// many elements reach the threshold at once (a tile of equal logits), the tile is
// gone through one element per thread at a time.
//
// The sum runs over x - m, m the thread's largest so far, which no scale of the
// logits overflows; threads, warps and slices are joined in a fixed order that
// depends on nothing but the element's index, so that equal rows have equal sums.
// Candidates of different rows are compared by their 64-bit scores.
#include <algorithm>

#include "common.cuh"
#include "params.cuh"

namespace pka {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPer = 32;  // elements of a thread per tile
constexpr int kTile = kThreads * kPer;
constexpr int kCap = 1024;    // collected keys
constexpr int kCutAt = 128;   // keys that are cut back at a tile's end
constexpr int kMaxEntries = 4096;  // of all parts' lists of a group
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kMinusInf = 0x007fffffu;  // order_of(-infinity)
constexpr unsigned long long kNone = ((unsigned long long)kMinusInf << 32) | 0xffffffffu;  // below every candidate

using u64 = unsigned long long;

// Larger floats have larger orders; -0 has that of +0.
PKA_DEVICE uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
PKA_DEVICE float of_order(uint32_t o) { return __uint_as_float((o >> 31) ? o ^ 0x80000000u : ~o); }
PKA_DEVICE u64 key_of(float x, int token) { return ((u64)order_of(x) << 32) | (0xffffffffu - (uint32_t)token); }

PKA_DEVICE u64 order_of(double x) {
    const u64 b = (u64)__double_as_longlong(x + 0.0);
    return b ^ ((b >> 63) ? ~0ull : 1ull << 63);
}
PKA_DEVICE double of_order(u64 o) { return __longlong_as_double((long long)((o >> 63) ? o ^ (1ull << 63) : ~o)); }

PKA_DEVICE u64 load_cluster64(const u64* p, uint32_t rank) {
    u64 v;
    asm volatile("{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.u64 %0, [a];\n\t}"
                 : "=l"(v)
                 : "r"(smem_u32(p)), "r"(rank)
                 : "memory");
    return v;
}

template <bool kBf16>
PKA_DEVICE float element(const void* row, int64_t i) {
    if constexpr (kBf16) return __bfloat162float(static_cast<const __nv_bfloat16*>(row)[i]);
    else return static_cast<const float*>(row)[i];
}

// Element e of a thread's kPer of a tile: with 16-byte loads runs of 8 (4)
// elements, else neighbours in neighbouring threads.
template <bool kBf16, bool kVec>
PKA_DEVICE int place_of(int e) {
    constexpr int kRun = !kVec ? 1 : kBf16 ? 8 : 4;
    return (e / kRun * kThreads + (int)threadIdx.x) * kRun + e % kRun;
}

// A tile's elements of this thread; -infinity from element n of the tile on.
template <bool kBf16, bool kVec>
PKA_DEVICE void load_tile(float (&x)[kPer], const void* row, int64_t at, int n) {
    if constexpr (kVec) {
        constexpr int kRun = kBf16 ? 8 : 4;
        uint4 raw[kPer / kRun];
#pragma unroll
        for (int j = 0; j < kPer / kRun; ++j) {
            const int i = place_of<kBf16, kVec>(j * kRun);
            if (i + kRun <= n) raw[j] = __ldcs(reinterpret_cast<const uint4*>(row) + (at + i) / kRun);
        }
#pragma unroll
        for (int j = 0; j < kPer / kRun; ++j) {
            const int i = place_of<kBf16, kVec>(j * kRun);
            const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
            if (i + kRun <= n) {
#pragma unroll
                for (int e = 0; e < kRun; ++e)
                    x[j * kRun + e] = !kBf16 ? __uint_as_float(w[e % 4]) : e % 2 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
            } else {
#pragma unroll
                for (int e = 0; e < kRun; ++e) x[j * kRun + e] = i + e < n ? element<kBf16>(row, at + i + e) : -INFINITY;
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int i = place_of<kBf16, kVec>(e);
            x[e] = i < n ? element<kBf16>(row, at + i) : -INFINITY;
        }
    }
}

struct Shared {
    u64 keys[kCap];
    uint32_t tops[kThreads];
    float m[kWarps], s[kWarps];
    u64 limit;
    int count;
};

// Cuts the collected keys back to the best `keep`, sorted, and raises the limit
// to the last of them. All threads.
PKA_DEVICE void cut(Shared& sh, int keep) {
    const int n = sh.count;
    u64 mine[kCap / kThreads];
    int rank[kCap / kThreads];
#pragma unroll
    for (int j = 0; j < kCap / kThreads; ++j) {
        const int i = (int)threadIdx.x + j * kThreads;
        rank[j] = keep;
        if (i >= n) continue;
        mine[j] = sh.keys[i];
        rank[j] = 0;
        for (int o = 0; o < n; ++o) rank[j] += sh.keys[o] > mine[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kCap / kThreads; ++j) {
        if (rank[j] >= keep) continue;
        sh.keys[rank[j]] = mine[j];
        if (rank[j] == keep - 1) sh.limit = mine[j];
    }
    if (threadIdx.x == 0) sh.count = min(n, keep);
    __syncthreads();
}

// What a CTA leaves of a part: the largest logit, the sum of exp(x - largest) and
// the best keys (0 behind the last).
struct Part {
    float m, s;
};

template <bool kBf16, bool kVec>
__global__ void __launch_bounds__(kThreads) beam_select_kernel(const BeamSelectParams p) {
    extern __shared__ __align__(16) uint8_t s_dyn[];
    __shared__ Shared sh;
    __shared__ double s_lse[kMaxBeams];
    __shared__ int s_state[kMaxBeams];
    grid_dep_launch();
    grid_dep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ncta = (int)cluster_size(), rank = (int)cluster_rank(), group = blockIdx.x / ncta;
    const int keep = p.keep, parts = p.beams * p.slices;
    const int per = (parts + ncta - 1) / ncta;
    u64* lists = reinterpret_cast<u64*>(s_dyn);                      // [per][keep]
    Part* part = reinterpret_cast<Part*>(lists + (size_t)per * keep);  // [per]

    for (int i = rank, li = 0; i < parts; i += ncta, ++li) {
        const int beam = i / p.slices, slice = i % p.slices;
        const int64_t row = (int64_t)group * p.beams + beam;
        const float score = p.scores[row];
        const bool done = p.finished && p.finished[row] != 0;
        const int from = slice * p.slice_len;
        const int n = done || !(fabsf(score) < INFINITY) ? 0 : min(p.slice_len, p.vocab - from);
        const void* logits = kBf16 ? (const void*)(static_cast<const __nv_bfloat16*>(p.logits) + row * p.row_stride)
                                   : (const void*)(static_cast<const float*>(p.logits) + row * p.row_stride);
        if (tid == 0) {
            sh.limit = kNone;
            sh.count = 0;
        }
        float m = -INFINITY, s = 0.f;
        for (int t = 0; t < n; t += kTile) {
            float x[kPer];
            load_tile<kBf16, kVec>(x, logits, from + t, n - t);
            float top = -INFINITY;
#pragma unroll
            for (int e = 0; e < kPer; ++e) top = fmaxf(top, x[e]);
            if (top > m) {
                s *= fast_exp2((m - top) * kLog2e);
                m = top;
            }
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
            if (m > -INFINITY) {
#pragma unroll
                for (int e = 0; e < kPer; ++e) sum[e % 4] += fast_exp2((x[e] - m) * kLog2e);
            } else {
#pragma unroll
                for (int e = 0; e < kPer; ++e) sum[e % 4] += x[e] == x[e] ? 0.f : x[e];  // a NaN among -infinities
            }
            s += (sum[0] + sum[1]) + (sum[2] + sum[3]);

            // ---- candidates
            const uint32_t high = order_of(top);
            if (t == 0) {
                sh.tops[tid] = high;
                __syncthreads();
                int above = 0;
#pragma unroll 8
                for (int o = 0; o < kThreads; ++o) above += sh.tops[o] > high || (sh.tops[o] == high && o < tid);
                if (above == keep - 1 && high > kMinusInf) sh.limit = ((u64)high << 32) - 1;
            }
            __syncthreads();
            const int had = sh.count;
            const u64 limit = sh.limit;
            __syncthreads();
            if ((((u64)high << 32) | 0xffffffffu) > limit) {
#pragma unroll
                for (int e = 0; e < kPer; ++e) {
                    const u64 key = key_of(x[e], from + t + place_of<kBf16, kVec>(e));
                    if (key <= limit) continue;
                    const int at = atomicAdd(&sh.count, 1);
                    if (at < kCap) sh.keys[at] = key;
                }
            }
            __syncthreads();
            if (sh.count > kCap) {
                __syncthreads();
                if (tid == 0) sh.count = had;
                for (int e = 0; e < kPer; ++e) {
                    __syncthreads();
                    if (sh.count > kCap - kThreads) cut(sh, keep);
                    const u64 now = sh.limit;
                    const int at_row = t + place_of<kBf16, kVec>(e);
                    const u64 key = at_row < n ? key_of(element<kBf16>(logits, from + at_row), from + at_row) : 0;
                    __syncthreads();
                    if (key > now) sh.keys[atomicAdd(&sh.count, 1)] = key;
                }
                __syncthreads();
            }
            if (sh.count > kCutAt) cut(sh, keep);
        }
        __syncthreads();
        if (n > 0) cut(sh, keep);
        const int have = sh.count;
        for (int k = tid; k < keep; k += kThreads) lists[(size_t)li * keep + k] = k < have ? sh.keys[k] : 0;
        // ---- the part's sum, in a fixed order
        float wm = m;
#pragma unroll
        for (int o = 16; o; o >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, o));
        if (lane == 0) sh.m[warp] = wm;
        __syncthreads();
        float all = sh.m[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) all = fmaxf(all, sh.m[w]);
        float ws = m == all ? s : s * fast_exp2((m - all) * kLog2e);  // (of -infinities: 0, or NaN)
#pragma unroll
        for (int o = 16; o; o >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, o);
        if (lane == 0) sh.s[warp] = ws;
        __syncthreads();
        if (tid == 0) {
            float total = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) total += sh.s[w];
            part[li] = Part{all, total};
        }
        __syncthreads();
    }

    cluster_barrier();
    if (rank == 0) {
        // ---- log-sums of the rows
        for (int b = tid; b < p.beams; b += kThreads) {
            const int64_t row = (int64_t)group * p.beams + b;
            const float score = p.scores[row];
            const bool done = p.finished && p.finished[row] != 0;
            float m = -INFINITY, s = 0.f;
            for (int k = 0; k < p.slices; ++k) {
                const int i = b * p.slices + k;
                const float pm = load_cluster(&part[i / ncta].m, i % ncta), ps = load_cluster(&part[i / ncta].s, i % ncta);
                if (pm > m) {
                    s *= fast_exp2((m - pm) * kLog2e);
                    m = pm;
                }
                s += pm == m ? ps : ps * fast_exp2((pm - m) * kLog2e);
            }
            int state = 0;  // no candidates
            double lse = 0;
            if (!(score < INFINITY)) {
                set_error(p.err, PKA_DEVERR_LOGITS);
            } else if (score > -INFINITY && done) {
                state = 2;
            } else if (score > -INFINITY) {
                if (!(s < INFINITY) || m == INFINITY) {
                    set_error(p.err, PKA_DEVERR_LOGITS);
                } else if (m > -INFINITY) {
                    state = 1;
                    lse = (double)m + log((double)s);
                }
            }
            s_lse[b] = lse;
            s_state[b] = state;
        }
        // the joined lists: 64-bit scores, and what decides between equal ones
        u64* hi = reinterpret_cast<u64*>(part + per);  // [parts][keep]
        u64* lo = hi + (size_t)parts * keep;
        int32_t* picked = reinterpret_cast<int32_t*>(lo + (size_t)parts * keep);
        if (tid == 0) sh.count = 0;
        __syncthreads();
        const int entries = parts * keep;
        for (int j = tid; j < entries; j += kThreads) {
            const int i = j / keep, k = j % keep, b = i / p.slices;
            const int64_t row = (int64_t)group * p.beams + b;
            const u64 key = load_cluster64(&lists[(size_t)(i / ncta) * keep + k], i % ncta);
            u64 h = 0, l = 0;
            uint32_t order = 0;
            int token = -1;
            if (s_state[b] == 1 && key) {
                order = (uint32_t)(key >> 32);
                token = (int)(0xffffffffu - (uint32_t)key);
                h = order_of((double)p.scores[row] + ((double)of_order(order) - s_lse[b]));
            } else if (s_state[b] == 2 && i % p.slices == 0 && k == 0) {
                token = p.end_token;
                h = order_of((double)p.scores[row]);
            }
            if (token >= 0)
                l = ((u64)(kMaxBeams - 1 - b) << 58) | ((u64)order << 26) | (u64)(kMaxVocab - 1 - token);
            hi[j] = h;
            lo[j] = l;
        }
        __syncthreads();
        // a threshold that at least `keep` entries reach: the keep-th of the lists' first `deep`
        const int deep = (keep + parts - 1) / parts, heads = parts * deep;
        u64 th = 0, tl = 0;
        if (entries > kThreads) {
            for (int j = tid; j < heads; j += kThreads) {
                const int at = j / deep * keep + j % deep;
                const u64 h = hi[at], l = lo[at];
                int above = 0;
                for (int o = 0; o < heads; ++o) {
                    const int a = o / deep * keep + o % deep;
                    above += hi[a] > h || (hi[a] == h && (lo[a] > l || (lo[a] == l && o < j)));
                }
                if (above == keep - 1) {
                    sh.keys[0] = h;
                    sh.keys[1] = l;
                }
            }
            __syncthreads();
            th = sh.keys[0];
            tl = sh.keys[1];
        }
        for (int j = tid; j < entries; j += kThreads)
            if (hi[j] && (hi[j] > th || (hi[j] == th && lo[j] >= tl))) picked[atomicAdd(&sh.count, 1)] = j;
        __syncthreads();
        const int found = sh.count;
        const int64_t base = (int64_t)group * keep;
        for (int j = tid; j < found; j += kThreads) {
            const u64 h = hi[picked[j]], l = lo[picked[j]];
            int above = 0;
            for (int o = 0; o < found; ++o) {
                const u64 a = hi[picked[o]];
                above += a > h || (a == h && lo[picked[o]] > l);
            }
            if (above >= keep) continue;
            const int b = kMaxBeams - 1 - (int)(l >> 58), token = kMaxVocab - 1 - (int)(l & (kMaxVocab - 1));
            p.out_scores[base + above] = (float)of_order(h);
            p.parents[base + above] = group * p.beams + b;
            p.tokens[base + above] = token;
            if (p.out_finished) p.out_finished[base + above] = s_state[b] == 2 || token == p.end_token;
        }
        for (int k = found + tid; k < keep; k += kThreads) {
            p.out_scores[base + k] = -INFINITY;
            p.parents[base + k] = -1;
            p.tokens[base + k] = -1;
            if (p.out_finished) p.out_finished[base + k] = 0;
        }
    }
    cluster_barrier();  // no CTA's lists go before they are read
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

template <bool kBf16, bool kVec>
cudaError_t go(BeamSelectParams p, int num_sms, cudaStream_t stream) {
    // CTAs of a group: until there is one for each tile, or two for each SM; up to the parts' lists that one CTA joins
    int ncta = 1, slices = 1;
    while (ncta < 8) {
        const int more = 2 * ncta, s = more / gcd(p.beams, more);
        if ((int64_t)ncta * kTile >= (int64_t)p.beams * p.vocab || (int64_t)p.groups * ncta >= 2 * num_sms ||
            p.beams * s * p.keep > kMaxEntries)
            break;
        ncta = more;
        slices = s;
    }
    p.slices = slices;
    p.slice_len = ((p.vocab + slices - 1) / slices + 7) & ~7;  // (16-byte pieces stay whole)
    const int parts = p.beams * slices, per = (parts + ncta - 1) / ncta;
    const size_t smem = (size_t)per * (p.keep * sizeof(u64) + sizeof(Part)) +
                        (size_t)parts * p.keep * (2 * sizeof(u64) + sizeof(int32_t));
    auto kern = beam_select_kernel<kBf16, kVec>;
    if (smem > 32 * 1024) {  // (the most that any call takes)
        const cudaError_t e = cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
            (int)((size_t)kMaxEntries * (3 * sizeof(u64) + sizeof(int32_t)) + kMaxEntries * sizeof(Part)));
        if (e != cudaSuccess) return e;
    }
    return launch_cluster(kern, dim3(p.groups * ncta), dim3(kThreads), smem, ncta, stream, p);
}

}  // namespace

cudaError_t launch_beam_select(const BeamSelectParams& p, bool bf16, int num_sms, cudaStream_t stream) {
    const size_t size = bf16 ? 2 : 4;
    const bool vec = reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 && (size_t)p.row_stride * size % 16 == 0;
    if (bf16) return vec ? go<true, true>(p, num_sms, stream) : go<true, false>(p, num_sms, stream);
    return vec ? go<false, true>(p, num_sms, stream) : go<false, false>(p, num_sms, stream);
}

}  // namespace pka
