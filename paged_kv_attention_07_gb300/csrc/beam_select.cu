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
// A part is gone through twice. First every warp streams its share, four 16-byte loads
// per lane at a time with the next four on their way: the sum, and the lane's largest
// logit of each of up to kEpochs stretches. num_out lanes reach the num_out-th of the
// lanes' largest, so nothing below that limit counts, and few stretches reach it: only
// those are loaded again, and their elements past the limit collected. (With the search in
// the stream each tile that passed a limit cost a microsecond: 64 x 4 beams took 34 us, not 30.) A
// warp's buffer of keys is cut back to the best num_out when it is full (a part of equal
// logits), and the limit rises to the last of them. A key is the logit's order in the upper
// and the token's complement in the lower 32 bits: keys are distinct, the larger one is the
// better, and the order of their arrival does not matter.
//
// The sum runs over x - m, m the lane's largest so far, which no scale of the
// logits overflows; lanes, warps and slices are joined in a fixed order that
// depends on nothing but the element's index, so that equal rows have equal sums.
// Candidates of different rows are compared by their 64-bit scores.
//
// Measured: 4 rows of 32000 bf16 logits 8.7 us; 64 groups of 4 rows of 131072 23.6 us (2.8 TB/s; at the
// rate of a copy the 67 MB take 9.9); 17 groups of 5 rows of 50001 float32 logits 11.4 us. A
// launch and the phases behind the stream (limit, second reading, lists, ranks: each a
// few hundred instructions fetched for the first time) take about 7 us of each; the stream
// of 256 rows is bound by the busiest SMs, which have two rows where the mean is 1.7.
#include <float.h>

#include <algorithm>

#include "common.cuh"
#include "params.cuh"

namespace pka {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kLoads = 4;     // 16-byte loads of a lane in flight
constexpr int kBuffer = 128;  // keys that a warp collects
constexpr int kEpochs = 16;   // stretches of a lane's share
constexpr int kResident = 2;  // CTAs of an SM (of 4, with half the registers, 64 x 4 beams took 29 us, not 23)
constexpr int kMaxCluster = 16;
constexpr int kMaxEntries = 4096;  // of all parts' lists of a group
constexpr int kDirect = 96;        // of them that are compared with each other as they are
static_assert(kThreads == 256, "a bin per thread");
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

// Stores v where `p` lies in the shared memory of the cluster's first CTA (which must have started).
PKA_DEVICE void store_first64(u64* p, u64 v) {
    asm volatile("{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\tst.shared::cluster.u64 [a], %1;\n\t}" ::"r"(
                     smem_u32(p)),
                 "l"(v)
                 : "memory");
}

// A warp's tile: kPer elements per lane. With 16-byte loads a lane has runs of kRun elements,
// else neighbouring elements, of bf16 pairs, lie in neighbouring lanes, wherever a row begins:
// equal rows are added up alike. Pairs of a row at an odd element are put together from the halves of
// two words, the second one the next lane's (element by element 9 rows of 166763 took
// 24.5 us, aligned ones 15).
template <bool kBf16, bool kVec>
struct Tile {
    static constexpr int kRun = kBf16 ? 8 : 4, kPer = kLoads * kRun, kSize = 32 * kPer;
    static_assert(kPer <= 32, "a lane's hits are the bits of a word");
    uint32_t w[kLoads * 4];  // two bf16 or one float each
    uint32_t last;           // of words not put together yet: the one behind the last lane's
    bool halves = false;     // they are not
    PKA_DEVICE static int place(int e) {
        const int lane = threadIdx.x & 31;
        return kVec ? (e / kRun * 32 + lane) * kRun + e % kRun : kBf16 ? (e / 2 * 32 + lane) * 2 + e % 2 : e * 32 + lane;
    }
    PKA_DEVICE float operator[](int e) const {
        if constexpr (!kBf16) return __uint_as_float(w[e]);
        else return e % 2 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
    }
    // Elements from `at` of the row on; -infinity from element n of the tile on. `front`: the row's
    // element in front of them may be read.
    PKA_DEVICE void load(const void* row, int at, int n, bool front) {
        const uint32_t none = kBf16 ? 0xff80ff80u : 0xff800000u;
        if constexpr (kBf16 && !kVec) {
            const uintptr_t p = reinterpret_cast<uintptr_t>(row) + 2 * (int64_t)at;
            halves = p % 4 != 0;
            if (halves ? front && n > kSize : n >= kSize) {
                const uint32_t* from = reinterpret_cast<const uint32_t*>(p - p % 4) + (threadIdx.x & 31);
#pragma unroll
                for (int j = 0; j < kPer / 2; ++j) w[j] = __ldcs(from + 32 * j);
                if (halves && (threadIdx.x & 31) == 31) last = __ldcs(from + 16 * kPer - 31);
                return;
            }
            halves = false;
        }
        if (kVec && n >= kSize) {
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const uint4 x = __ldcs(reinterpret_cast<const uint4*>(row) + (at + place(j * kRun)) / kRun);
                w[4 * j] = x.x;
                w[4 * j + 1] = x.y;
                w[4 * j + 2] = x.z;
                w[4 * j + 3] = x.w;
            }
            return;
        }
#pragma unroll
        for (int e = 0; e < kPer; e += kBf16 ? 2 : 1) {
            uint32_t x = none;
            const int i = place(e);
            if constexpr (!kBf16) {
                if (i < n) x = __float_as_uint(static_cast<const float*>(row)[at + i]);
            } else {
                const uint16_t* r = static_cast<const uint16_t*>(row) + at;
                const int k = place(e + 1);
                if (i < n) x = (x & 0xffff0000u) | r[i];
                if (k < n) x = (x & 0xffffu) | ((uint32_t)r[k] << 16);
            }
            w[kBf16 ? e / 2 : e] = x;
        }
    }
    // Puts the pairs together (whole warps).
    PKA_DEVICE void settle() {
        if (kVec || !kBf16 || !halves) return;
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int j = 0; j < kPer / 2; ++j) {
            const uint32_t after = __shfl_sync(0xffffffffu, lane == 0 && j + 1 < kPer / 2 ? w[j + 1 < kPer / 2 ? j + 1 : j] : w[j], (lane + 1) & 31);
            w[j] = __funnelshift_r(w[j], lane == 31 && j + 1 == kPer / 2 ? last : after, 16);
        }
        halves = false;
    }
};

struct Shared {
    u64 keys[kWarps][kBuffer];
    float tops[kEpochs][kThreads];
    uint32_t best[kWarps][32];
    float m[kWarps], s[kWarps];
    u64 limit;
    int count[kWarps];
};

// Cuts the warp's n collected keys back to the best `keep`, sorted, and raises the
// limit to the last of them. Returns how many are left.
PKA_DEVICE int cut(u64* keys, int n, int keep, u64* limit) {
    const int lane = threadIdx.x & 31;
    u64 mine[kBuffer / 32];
    int rank[kBuffer / 32];
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kBuffer / 32; ++j) {
        mine[j] = lane + 32 * j < n ? keys[lane + 32 * j] : 0;
        rank[j] = 0;
    }
    for (int o = n; o < (n + 3) / 4 * 4; ++o)
        if (lane == 0) keys[o] = 0;
    __syncwarp();
#pragma unroll 1
    for (int o = 0; o < n; o += 4) {
        const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(keys + o), b = *reinterpret_cast<const ulonglong2*>(keys + o + 2);
#pragma unroll
        for (int j = 0; j < kBuffer / 32; ++j)
            rank[j] += (a.x > mine[j]) + (a.y > mine[j]) + (b.x > mine[j]) + (b.y > mine[j]);
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kBuffer / 32; ++j) {
        if (mine[j] == 0 || rank[j] >= keep) continue;
        keys[rank[j]] = mine[j];
        if (rank[j] == keep - 1) atomicMax(limit, mine[j]);
    }
    __syncwarp();
    return min(n, keep);
}

// log(s) of a normal s > 0 to 2^-28 (of s up to 2^26: 2.3e-9): e ln 2 + log m with m in [3/4, 3/2) and log m =
// 2 artanh z = 2 z + z^3 (2/3 + 2/5 z^2 + ...), z = (m - 1) / (m + 1) to twice 24 bits, the rest
// in 32 bits, which bounds it (the 64-bit logarithm takes a microsecond, much of it the fetch of its code).
PKA_DEVICE double log_of(float s) {
    int e = (int)(__float_as_uint(s) >> 23) - 127;
    float m = __uint_as_float((__float_as_uint(s) & 0x7fffffu) | 0x3f800000u);
    if (m >= 1.5f) {
        m *= 0.5f;
        ++e;
    }
    const float n = m - 1.f, d = m + 1.f, d_low = (1.f - d) + m;  // (n is exact, d + d_low too)
    const float z = __fdiv_rn(n, d), z_low = __fdiv_rn(fmaf(-z, d, n) - z * d_low, d), q = z * z;
    const float tail = z * q * (0.666666667f + q * (0.4f + q * (0.285714286f + q * (0.222222222f + q * 0.181818182f))));
    return (double)e * 0.69314718055994531 + 2.0 * ((double)z + (double)z_low) + (double)tail;
}

template <bool kBf16, bool kVec>
__global__ void __launch_bounds__(kThreads, kResident) beam_select_kernel(const BeamSelectParams p) {
    using T = Tile<kBf16, kVec>;
    extern __shared__ __align__(16) uint8_t s_dyn[];
    __shared__ __align__(16) Shared sh;
    __shared__ double s_lse[kMaxBeams];
    __shared__ float s_score[kMaxBeams];
    __shared__ int s_state[kMaxBeams];
    __shared__ int s_found, s_bin, s_need;
    grid_dep_launch();
    grid_dep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ncta = (int)cluster_size(), rank = (int)cluster_rank(), group = blockIdx.x / ncta;
    const int keep = p.keep, parts = p.beams * p.slices;
    // in the first CTA's shared memory, written by all of the cluster
    u64* lists = reinterpret_cast<u64*>(s_dyn);                          // [parts][keep], 0 behind the last key
    u64* sums = lists + (size_t)parts * keep;                            // [parts], a Part each
    u64* hi = sums + parts + ((parts * (keep + 1)) & 1);                 // [parts][keep], at 16 bytes
    u64* lo = hi + (size_t)parts * keep;
    u64* best = lo + (size_t)parts * keep;  // [parts * keep][2], those that may be among the best
    cluster_arrive();
    for (int b = tid; b < p.beams; b += kThreads) {
        const int64_t row = (int64_t)group * p.beams + b;
        s_score[b] = p.scores[row];
        s_state[b] = p.finished && p.finished[row] != 0;
    }
    if (tid == 0) s_found = 0;
    __syncthreads();

    bool met = false;  // the first CTA has started
    for (int i = rank; i < parts; i += ncta) {
        const int beam = i / p.slices, slice = i - beam * p.slices;
        const int from = slice * p.slice_len;
        const int n = s_state[beam] || !(fabsf(s_score[beam]) < INFINITY) ? 0 : min(p.slice_len, p.vocab - from);
        const int64_t at = ((int64_t)group * p.beams + beam) * p.row_stride + from;
        const void* logits = static_cast<const uint8_t*>(p.logits) + at * (kBf16 ? 2 : 4);
        if (tid == 0) sh.limit = kNone;
        __syncthreads();
        u64* keys = sh.keys[warp];
        // ---- the stream
        constexpr int kRound = kWarps * T::kSize;
        const int rounds = (n + kRound - 1) / kRound, stretch = (rounds + kEpochs - 1) / kEpochs;
        float m = -INFINITY, s = 0.f, top = -INFINITY;
        T x, next;
        int t = warp * T::kSize;
        const bool inside = at > 0;  // (there is an element in front of the part)
        if (t < n) next.load(logits, t, n - t, inside || t > 0);
        for (int r = 0, in = 0, epoch = 0; r < rounds; ++r, t += kRound) {
            if (t < n) {
                x = next;
                x.settle();
                if (t + kRound < n) next.load(logits, t + kRound, n - t - kRound, true);
                float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < T::kPer; e += 2) tops[e / 2 % 4] = fmax3f(tops[e / 2 % 4], x[e], x[e + 1]);
                top = fmaxf(fmax3f(top, tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                if (top > m) {
                    s *= fast_exp2((m - top) * kLog2e);
                    m = top;
                }
                if (m > -INFINITY) {
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int e = 0; e < T::kPer; e += 2) {
                        float d0, d1;
                        fma2_bcast(d0, d1, x[e], x[e + 1], 1.f, -m);
                        fma2_bcast(d0, d1, d0, d1, kLog2e, 0.f);
                        add2(sum[e % 4], sum[e % 4 + 1], fast_exp2(d0), fast_exp2(d1));
                    }
                    s += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                } else {
#pragma unroll
                    for (int e = 0; e < T::kPer; ++e) s += x[e] == x[e] ? 0.f : x[e];  // a NaN among -infinities
                }
            }
            if (++in == stretch || r == rounds - 1) {
                sh.tops[epoch++][tid] = top;
                top = -INFINITY;
                in = 0;
            }
        }
        // ---- the limit: the keep-th of the lanes' largest, from each warp's first `keep`
        {
            uint32_t left = order_of(m), mine = 0;
            const int take = min(keep, 32);
            for (int k = 0; k < take; ++k) {
                const uint32_t most = __reduce_max_sync(0xffffffffu, left);
                if (lane == k) mine = most;
                const uint32_t who = __ballot_sync(0xffffffffu, left == most);
                if (lane == __ffs(who) - 1) left = 0;
            }
            sh.best[warp][lane] = mine;
        }
        // ... and the part's sum, in a fixed order
        float wm = m;
#pragma unroll
        for (int o = 16; o; o >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, o));
        float ws = m == wm ? s : s * fast_exp2((m - wm) * kLog2e);  // (of -infinities: 0, or NaN)
#pragma unroll
        for (int o = 16; o; o >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, o);
        if (lane == 0) {
            sh.m[warp] = wm;
            sh.s[warp] = ws;
        }
        __syncthreads();
        if (warp == 0) {
            uint32_t left[kWarps], most = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) left[w] = sh.best[w][lane];
            for (int k = 0; k < keep; ++k) {
                uint32_t mine = left[0];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) mine = max(mine, left[w]);
                most = __reduce_max_sync(0xffffffffu, mine);
                const uint32_t who = __ballot_sync(0xffffffffu, mine == most);
                if (lane == __ffs(who) - 1) {
                    bool out = false;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        if (!out && left[w] == most) {
                            left[w] = 0;
                            out = true;
                        }
                    }
                }
            }
            if (lane == 0 && most > kMinusInf) sh.limit = ((u64)most << 32) - 1;
        }
        if (!met) cluster_wait();
        met = true;
        if (tid == 32) {
            float all = sh.m[0], total = 0.f;
#pragma unroll
            for (int w = 1; w < kWarps; ++w) all = fmaxf(all, sh.m[w]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) total += sh.m[w] == all ? sh.s[w] : sh.s[w] * fast_exp2((sh.m[w] - all) * kLog2e);
            store_first64(&sums[i], (u64)__float_as_uint(all) | ((u64)__float_as_uint(total) << 32));
        }
        __syncthreads();
        // ---- what reaches it, from the stretches that do
        int have = 0;
        for (int epoch = 0; epoch * stretch < rounds; ++epoch) {
            u64 limit = *const_cast<volatile u64*>(&sh.limit);
            // (a logit that equals the limit's is decided by its key; -infinity never counts)
            const float reach = limit == kNone ? -FLT_MAX : of_order((uint32_t)(limit >> 32));
            const bool again = sh.tops[epoch][tid] >= reach;
            if (!__any_sync(0xffffffffu, again)) continue;
            t = epoch * stretch * kRound + warp * T::kSize;
            for (int r = 0; r < stretch && t < n; ++r, t += kRound) {
                uint32_t hits = 0;  // of this lane's elements
                if (again || !kVec) {
                    x.load(logits, t, n - t, inside || t > 0);
                    x.settle();
#pragma unroll
                    for (int e = 0; e < T::kPer; ++e) hits |= x[e] >= reach ? 1u << e : 0u;
                }
                while (__any_sync(0xffffffffu, hits != 0)) {
                    if (have > kBuffer - 32) {
                        have = cut(keys, have, keep, &sh.limit);
                        limit = *const_cast<volatile u64*>(&sh.limit);
                    }
                    u64 key = 0;
                    if (hits) {
                        const int at = __ffs(hits) - 1;
                        float v = x[0];
#pragma unroll
                        for (int e = 1; e < T::kPer; ++e) v = at == e ? x[e] : v;
                        key = key_of(v, from + t + T::place(at));
                        hits &= hits - 1;
                    }
                    const uint32_t who = __ballot_sync(0xffffffffu, key > limit);
                    if (key > limit) keys[have + __popc(who & ((1u << lane) - 1))] = key;
                    have += __popc(who);
                }
            }
        }
        // ---- the part's best keys
        if (lane == 0) sh.count[warp] = have;
        __syncthreads();
        int total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) total += sh.count[w];
        for (int k = lane; k < have; k += 32) {
            const u64 mine = keys[k];
            int above = 0;
#pragma unroll 1
            for (int w = 0; w < kWarps; ++w) {
#pragma unroll 4
                for (int o = 0; o < sh.count[w]; ++o) above += sh.keys[w][o] > mine;
            }
            if (above < keep) store_first64(&lists[(size_t)i * keep + above], mine);
        }
        if (tid >= total && tid < keep) store_first64(&lists[(size_t)i * keep + tid], 0);
        __syncthreads();
    }

    if (!met) cluster_wait();
    cluster_arrive();
    if (rank != 0) return;  // (nothing of it is read)
    cluster_wait();
    {
        // ---- log-sums of the rows
        for (int b = tid; b < p.beams; b += kThreads) {
            const float score = s_score[b];
            float m = -INFINITY, s = 0.f;
            for (int k = 0; k < p.slices; ++k) {
                const u64 x = sums[b * p.slices + k];
                const float pm = __uint_as_float((uint32_t)x), ps = __uint_as_float((uint32_t)(x >> 32));
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
            } else if (score > -INFINITY && s_state[b]) {
                state = 2;
            } else if (score > -INFINITY) {
                if (!(s < INFINITY) || m == INFINITY) {
                    set_error(p.err, PKA_DEVERR_LOGITS);
                } else if (m > -INFINITY) {
                    state = 1;
                    lse = (double)m + log_of(s);
                }
            }
            s_lse[b] = lse;
            s_state[b] = state;
        }
        // the joined lists: 64-bit scores, and what decides between equal ones
        __syncthreads();
        const int entries = parts * keep;
        for (int j = tid; j < entries; j += kThreads) {
            const int i = j / keep, k = j - i * keep, b = i / p.slices;
            const u64 key = lists[j];
            u64 h = 0, l = 0;
            uint32_t order = 0;
            int token = -1;
            if (s_state[b] == 1 && key) {
                order = (uint32_t)(key >> 32);
                token = (int)(0xffffffffu - (uint32_t)key);
                h = order_of((double)s_score[b] + ((double)of_order(order) - s_lse[b]));
            } else if (s_state[b] == 2 && i == b * p.slices && k == 0) {
                token = p.end_token;
                h = order_of((double)s_score[b]);
            }
            if (token >= 0)
                l = ((u64)(kMaxBeams - 1 - b) << 58) | ((u64)order << 26) | (u64)(kMaxVocab - 1 - token);
            hi[j] = h;
            lo[j] = l;
        }
        // A bound that the best `keep` reach and few others: the keep-th of the scores' upper 32 bits, found
        // eight bits at a time by counts of their values. (To compare all with all took 7 us of 256
        // entries, 20 of 512.)
        uint32_t least = 1;
        if (entries > kDirect) {
            uint32_t* bins = &sh.best[0][0];
            int need = keep;
            least = 0;
#pragma unroll 1
            for (int shift = 24; shift >= 0; shift -= 8) {
                bins[tid] = 0;
                __syncthreads();
                if (tid == 0) s_bin = -1;
                for (int j = tid; j < entries; j += kThreads) {
                    const uint32_t o = (uint32_t)(hi[j] >> 32);
                    if (o && (shift == 24 || o >> (shift + 8) == least >> (shift + 8))) atomicAdd(&bins[(o >> shift) & 255], 1);
                }
                __syncthreads();
                // from the largest value on
                const int mine = (int)bins[255 - tid];
                int sum = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += y;
                }
                if (lane == 31) sh.count[warp] = sum;
                __syncthreads();
                for (int w = 0; w < warp; ++w) sum += sh.count[w];
                if (sum >= need && sum - mine < need) {
                    s_bin = 255 - tid;
                    s_need = need - (sum - mine);
                }
                __syncthreads();
                if (s_bin < 0) break;  // (only of the first eight: there are no more than `keep`)
                least |= (uint32_t)s_bin << shift;
                need = s_need;
            }
            least = max(least, 1u);
        }
        __syncthreads();
        for (int j = tid; j < entries; j += kThreads) {
            if ((uint32_t)(hi[j] >> 32) < least) continue;
            const int to = atomicAdd(&s_found, 1);
            best[2 * to] = hi[j];
            best[2 * to + 1] = lo[j];
        }
        __syncthreads();
        const int found = s_found;
        const int64_t base = (int64_t)group * keep;
        for (int j = tid; j < found; j += kThreads) {
            const u64 h = best[2 * j], l = best[2 * j + 1];
            int above = 0;
#pragma unroll 4
            for (int o = 0; o < found; ++o) {
                const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(best + 2 * o);
                above += a.x > h || (a.x == h && a.y > l);
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
}

template <bool kBf16, bool kVec>
cudaError_t go(BeamSelectParams p, int num_sms, cudaStream_t stream) {
    // A group's CTAs have a part each where its beams allow: as many slices of a row as give each warp a
    // tile of its own, and no more than a cluster's 16 CTAs and the lists that one of them joins; and
    // three CTAs for two SMs, of the four that they hold: larger clusters leave SMs of a GPC over, and
    // with more of them some wait (17 x 5 beams in 255 CTAs 17.9 us, in 170 11.4).
    int slices = 1;
    while (p.beams * (slices + 1) <= kMaxCluster && (int64_t)p.groups * p.beams * (slices + 1) * 2 <= 3 * num_sms &&
           p.beams * (slices + 1) * p.keep <= kMaxEntries && p.vocab > slices * kWarps * Tile<kBf16, kVec>::kSize)
        ++slices;
    // Clusters of more than 8 CTAs leave many SMs of a GPC over: where not all fit at once, half as many CTAs
    // with twice the parts are faster (36 x 16 beams of 28464 25.5 us, not 36.4). Smaller ones are not halved:
    // 160 x 8 beams of 18432 take 43 us, in clusters of 4 49.
    int ncta = std::min(p.beams * slices, kMaxCluster);
    if (ncta > 8 && (int64_t)p.groups * ncta > 2 * num_sms) ncta = (ncta + 1) / 2;
    p.slices = slices;
    p.slice_len = ((p.vocab + slices - 1) / slices + 7) & ~7;  // (16-byte pieces stay whole)
    const size_t entries = (size_t)p.beams * slices * p.keep;
    const size_t smem = (5 * entries + p.beams * slices + 1) * sizeof(u64);
    auto kern = beam_select_kernel<kBf16, kVec>;
    if (smem > 47 * 1024 - sizeof(Shared) - 1024) {  // past what every kernel may use; the most that any call takes
        const cudaError_t e = cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
            (int)((size_t)(kMaxEntries * 6 + 1) * sizeof(u64)));
        if (e != cudaSuccess) return e;
    }
    if (ncta > 8) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
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
