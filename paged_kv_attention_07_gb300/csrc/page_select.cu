// page_select.cu -- the pages each new token reads: the best of its request's
// pages by an upper bound of its scores over each page.
//
// Token t at position p of request r, kv head g: pages 0 .. p / bs, the last
// one its own. With q's 8-bit codes c (2^x the least power of two with
// max |q| <= 127 * 2^x, c = q / 2^x rounded to nearest even) and a page's bounds
//   score = max over the heads h of the group of 2^x_h * 2^e * sum_i max(c_i lo_i, c_i hi_i)
// which no product of c 2^x with a key of the page exceeds (one with q itself may, by
// half a unit 2^x of each element at most). Every term is an integer and the sum
// stays below 2^21: its accumulation is exact in any order. The two factors are
// powers of two from 2^-60 to 2^122 each, further apart than float32's exponents
// reach, so a score is kept as a 32-bit integer of its order (score_key): exact at
// any magnitude, and ties are real ties.
//
// sum_i max(c_i lo_i, c_i hi_i) = <min(c, 0), lo> + <max(c, 0), hi>: one product
// of length 2 d with the page's record as it lies in memory (lo then hi).
// One warp scores 16 pages: it loads their 16 records (2 d bytes each) straight
// into the fragments of the product. The block ids of the CTA's pages are
// fetched together beforehand, into the places where the scores will go: the
// chain id -> record costs the time. A tile's registers take the next tile's
// records span by span as they are multiplied (96 requests of 4096 to 65536 tokens,
// 8 kv heads: 25.4 us, 2.77 TB/s; 27.7 us with the loads behind the products. Slower
// before that change: two whole tiles in registers 30.0 us, records by asynchronous
// copies 28.4, by one bulk copy each 39, bound by the rate at which an SM takes
// copies; int8 products 39 us. Contexts of one length, 95 requests of 23000 tokens,
// leave no SM waiting for another's long one: 17.1 us, 4.2 TB/s).
//
// The product runs on the f16 tensor cores: an int8 MMA takes 65 cycles here
// and two f16 ones of half its length 16. A code c becomes the f16 number
// 1152 + c with one byte permutation (the byte of c + 128 under the exponent of
// 1024), the queries' codes are f16, and 1152 * sum c_q is taken off at the end.
// All of it is exact: of a pair min(c, 0), max(c, 0) one is zero, so each of the
// two accumulators sums at most d / 2 <= 64 products of at most 1279 * 127, below
// 2^24. Which of a fragment's columns holds which element does not matter as long
// as A and B agree: a lane's 16-byte read of a record is the A operand of four
// MMAs.
//
// One cluster per (token, kv head): its CTAs score a slice of the pages each
// and leave the scores in the first CTA's shared memory, which then picks the
// pages. The scores never go to memory. The pick is a radix selection of the
// want-th largest score over the range the scores take: one histogram of 256
// bins usually leaves a handful of pages in the border bin, and those are
// ranked one against all. The chosen pages become a bit map, whose prefix sum
// gives ascending output (ties: the lowest page). HBM-bound for a full batch:
// 2 d + 4 bytes per (page, kv head).
#include "common.cuh"
#include "params.cuh"

namespace pka {

namespace {

constexpr int kBatch = 4;  // keys of a thread read together
constexpr uint32_t kFew = 32;  // pages in the border bin that are ranked one against all
constexpr int kCtaTiles = 4;  // of 16 pages: a CTA of a cluster takes part with these at least

template <int D, int NT, int kThreads>
struct PsCfg {
    static constexpr int kWarps = kThreads / 32;
    static constexpr int kQRow = 4 * D + 16;  // a head's codes in f16, padded by a quarter of the banks
    static constexpr int kFixed = NT * 8 * kQRow;  // then a key and a bit per page
};

// Queries' units are held as 2^(x + kUnitBias): sums below 2^21 times these are normal float32 numbers.
constexpr int kUnitBias = -62;

// An integer of the order of y * 2^e: y = sum * 2^(x + kUnitBias) is from 2^-122 to 2^81 or zero, 2^e a page's
// scale from 2^-60 to 2^122. Their exponent fields add up to 457 at most: 9 bits, for which the last bit of y's
// mantissa (21 bits of it count) makes room. Below INT_MAX, and -INT_MAX + 1.
PKA_DEVICE int score_key(float y, float scale) {
    const int size = (int)((__float_as_uint(fabsf(y)) + __float_as_uint(scale)) >> 1);
    return y == 0.f ? 0 : y < 0.f ? -size : size;
}

// Exclusive sum of v over the block's threads.
template <int kThreads>
PKA_DEVICE uint32_t block_scan(uint32_t v, uint32_t* s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    uint32_t before = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) before += w < warp ? s_warp[w] : 0u;
    __syncthreads();
    return before + incl - v;
}

template <int D, int NT, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 128 && NT == 1 ? 5 : 2) page_select_kernel(PageSelectParams p) {
    using C = PsCfg<D, NT, kThreads>;
    constexpr int kBins = kThreads;  // of a histogram: one per thread
    constexpr int kBinBits = kThreads == 256 ? 8 : 7;
    constexpr int kSpans = 2 * D / 64;  // 64-byte pieces of a record: four MMAs each
    constexpr int kE = D / 32;          // elements of a head per lane
    constexpr int kQHeads = NT * 8 / C::kWarps;  // heads whose codes a warp makes
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* s_q = smem;  // per head: min(c, 0) then max(c, 0), in the records' order
    uint32_t* s_key = reinterpret_cast<uint32_t*>(smem + C::kFixed);  // the candidates' scores (first CTA's is used)
    uint32_t* s_bits = s_key + ((p.max_seq_len - 1) / p.block_size + 1);  // the chosen candidates
    __shared__ float s_unit[NT * 8], s_zero[NT * 8][2];
    __shared__ uint32_t s_hist[kBins];
    __shared__ uint32_t s_warp[C::kWarps];
    __shared__ uint2 s_list[kFew];  // key and page
    __shared__ uint32_t s_min, s_max, s_digit, s_above, s_inside, s_count;
    grid_dep_launch();
    grid_dep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ncta = cluster_size(), cta = cluster_rank();
    if (tid == 0) s_min = 0xffffffffu, s_max = 0u, s_count = 0;
    s_hist[tid] = 0;
    // (waited for before the first store to the first CTA; here, where there is
    // nothing in flight that it would wait for itself)
    if (ncta > 1) cluster_arrive();
    // the heads of a token side by side: their records of a page are neighbours in memory
    const uint32_t unit_index = blockIdx.x / ncta;
    const int t = (int)(unit_index / (uint32_t)p.Hkv), g = (int)(unit_index - (uint32_t)t * (uint32_t)p.Hkv);
    // ---- this warp's part of the queries (needed later), and the token's request
    // and position (the same for the whole cluster)
    float x[kQHeads][kE];
#pragma unroll
    for (int j = 0; j < kQHeads; ++j) {
        const int h = warp + j * C::kWarps;
        const uint32_t* src = reinterpret_cast<const uint32_t*>(
            p.q + ((int64_t)t * p.Hq + g * p.G + (h < p.G ? h : 0)) * D + lane * kE);
#pragma unroll
        for (int i = 0; i < kE / 2; ++i) {
            const uint32_t v = h < p.G ? __ldg(src + i) : 0u;
            x[j][2 * i] = bf16_lo(v);
            x[j][2 * i + 1] = bf16_hi(v);
        }
    }
    const TokenPlace place = place_of(p.qsl, p.seq_lens, p.num_reqs, t);
    const int r = place.r;
    if (r < 0) {  // a row behind the last sequence
        if (ncta > 1) cluster_wait();
        return;
    }
    const long long pos = (long long)place.len - place.q1 + t;
    if (t < place.q0 || pos < 0 || pos >= place.len || place.len > p.max_seq_len) {
        if (tid == 0) set_error(p.err, PKA_DEVERR_SEQ_LEN);
        if (ncta > 1) cluster_wait();
        return;
    }
    const int n = (int)((uint32_t)pos / (uint32_t)p.block_size) + 1;  // pages up to the token's own
    int32_t* out = p.sel + ((int64_t)t * p.Hkv + g) * p.num_pages;
    const int K = p.num_pages;
    const int nf = p.num_first, m = n - nf - p.num_last, want = K - nf - p.num_last;
    const int tiles = (m + 15) / 16;
    // CTAs that take part: the token's first `parts` of the cluster
    const uint32_t parts = (uint32_t)max(1, min((int)ncta, tiles / kCtaTiles));
    if (n <= K || want == 0) {  // all pages, or only those that are always read
        for (int i = cta * kThreads + tid; i < K; i += ncta * kThreads) out[i] = i >= n ? -1 : n <= K || i < nf ? i : n - K + i;
        if (ncta > 1) cluster_wait();
        return;
    }
    if (cta >= parts) {
        cluster_wait();
        return;
    }

    // ---- this warp's tiles of 16 candidates [nf, nf + m): records and block ids ahead
    const int32_t* bt = p.block_table + (int64_t)r * p.max_blocks + nf;
    const int first = (int)((uint32_t)tiles * cta / parts), tiles_end = (int)((uint32_t)tiles * (cta + 1) / parts);
    {
        const int i1 = min(m, tiles_end * 16);
        for (int i0 = first * 16 + tid; i0 < i1; i0 += kBatch * kThreads) {
            int id[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) id[j] = i0 + j * kThreads < i1 ? __ldg(bt + i0 + j * kThreads) : 0;
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (i0 + j * kThreads < i1) s_key[i0 + j * kThreads] = (uint32_t)id[j];
        }
    }
    __syncthreads();
    // a tile's records as A fragments: rows lane / 4 and 8 more, piece lane % 4 of each span
    struct Rows {
        const uint4* src;
        float scale;
    };
    auto locate = [&](Rows (&x)[2], int tile) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int i = tile * 16 + half * 8 + (lane >> 2);
            int id = i < m ? (int)s_key[i] : 0;
            const bool ok = id >= 0 && id < p.num_blocks;
            if (!ok) {
                set_error(p.err, PKA_DEVERR_BLOCK_ID);
                id = 0;
            }
            const int64_t page = (int64_t)id * p.Hkv + g;
            x[half].src = reinterpret_cast<const uint4*>(p.bounds + page * 2 * D) + (lane & 3);
            x[half].scale = ok ? __ldg(p.scales + page) : -INFINITY;
        }
        __syncwarp();  // (the ids' places are written by the scores only after all lanes have read them)
    };
    const int tile0 = first + warp;
    uint4 rec[2][kSpans];
    Rows now[2];
    if (tile0 < tiles_end) {
        locate(now, tile0);
#pragma unroll
        for (int s = 0; s < kSpans; ++s) {
            rec[0][s] = __ldg(now[0].src + s * 4);
            rec[1][s] = __ldg(now[1].src + s * 4);
        }
    }

    // ---- the queries' codes
#pragma unroll
    for (int j = 0; j < kQHeads; ++j) {
        const int h = warp + j * C::kWarps;
        if (h >= p.G) break;  // (the columns of other heads are not looked at)
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < kE; ++i) a = fabsf(x[j][i]) <= 3.4e38f ? fmaxf(a, fabsf(x[j][i])) : INFINITY;
#pragma unroll
        for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        const bool finite = a <= 3.4e38f;  // a head with a NaN or an infinity scores 0 everywhere
        const int e = finite ? bound_exponent(a) : 0;
        const float unit = exp2i(-e);
        int sum = 0;
        __half* row = reinterpret_cast<__half*>(s_q + h * C::kQRow) + lane * kE;
#pragma unroll
        for (int i = 0; i < kE; ++i) {
            const int c = finite ? __float2int_rn(x[j][i] * unit) : 0;
            row[i] = __int2half_rn(min(c, 0));
            row[D + i] = __int2half_rn(max(c, 0));
            sum += c;
        }
        // an accumulator takes 8 elements of every 16: the offset of each
        const bool second = lane * kE & 8;
        const int s0 = __reduce_add_sync(0xffffffffu, second ? 0 : sum), s1 = __reduce_add_sync(0xffffffffu, second ? sum : 0);
        if (lane == 0) {
            s_unit[h] = exp2i(e + kUnitBias);
            s_zero[h][0] = 1152.f * (float)s0;
            s_zero[h][1] = 1152.f * (float)s1;
        }
    }
    __syncthreads();
    float unit[NT][2], zero[NT][2][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int h = nt * 8 + 2 * (lane & 3) + j;
            unit[nt][j] = s_unit[h];
            zero[nt][j][0] = s_zero[h][0];
            zero[nt][j][1] = s_zero[h][1];
        }
    // B: head (lane / 4), the 16 codes of piece (lane % 4) of each span
    const uint8_t* qrow = s_q + (lane >> 2) * C::kQRow + (lane & 3) * 32;
    auto load_b = [&](uint32_t (&b)[8], int nt, int s) {
        const uint4 u = *reinterpret_cast<const uint4*>(qrow + nt * 8 * C::kQRow + s * 128);
        const uint4 v = *reinterpret_cast<const uint4*>(qrow + nt * 8 * C::kQRow + s * 128 + 16);
        b[0] = u.x, b[1] = u.y, b[2] = u.z, b[3] = u.w, b[4] = v.x, b[5] = v.y, b[6] = v.z, b[7] = v.w;
    };
    if (ncta > 1) cluster_wait();

    // ---- scores; a span's registers take the next tile's as soon as it is multiplied
    uint32_t lo = 0xffffffffu, hi = 0u;
    for (int tile = tile0; tile < tiles_end; tile += C::kWarps) {
        const bool more = tile + C::kWarps < tiles_end;
        Rows next[2] = {};
        if (more) locate(next, tile + C::kWarps);
        float c[NT][2][4] = {};
#pragma unroll
        for (int s = 0; s < kSpans; ++s) {
            const uint4 a = rec[0][s], b = rec[1][s];
            const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
            uint32_t f[4][4];  // 1152 + code, f16 pairs
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t u = aw[j] ^ 0x80808080u, v = bw[j] ^ 0x80808080u;
                f[j][0] = __byte_perm(u, 0x64646464u, 0x4140);
                f[j][1] = __byte_perm(v, 0x64646464u, 0x4140);
                f[j][2] = __byte_perm(u, 0x64646464u, 0x4342);
                f[j][3] = __byte_perm(v, 0x64646464u, 0x4342);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                uint32_t q[8];
                load_b(q, nt, s);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mma_f16(c[nt][j >> 1], f[j][0], f[j][1], f[j][2], f[j][3], q[2 * j], q[2 * j + 1]);
            }
            if (more) {
                rec[0][s] = __ldg(next[0].src + s * 4);
                rec[1][s] = __ldg(next[1].src + s * 4);
            }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float y = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (nt * 8 + 2 * (lane & 3) + j < p.G)
                        y = fmaxf(y, ((c[nt][0][half * 2 + j] - zero[nt][j][0]) + (c[nt][1][half * 2 + j] - zero[nt][j][1])) *
                                         unit[nt][j]);
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 1));
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
            // a page that bounds nothing (scale +inf) comes first, one that does not exist last
            int v = score_key(y, now[half].scale);
            if (fabsf(now[half].scale) == INFINITY) v = now[half].scale > 0.f ? INT32_MAX : INT32_MIN;
            const int i = tile * 16 + half * 8 + (lane >> 2);
            if (i < m) {
                const uint32_t k = (uint32_t)v ^ 0x80000000u;  // in unsigned order
                lo = min(lo, k);
                hi = max(hi, k);
                if ((lane & 3) == 0) store_cluster(&s_key[i], 0, k);
            }
            now[half].scale = next[half].scale;
        }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0 && lo <= hi) {
        min_cluster(&s_min, 0, lo);
        max_cluster(&s_max, 0, hi);
    }
    if (parts == 1) __syncthreads();
    else cluster_barrier();
    if (cta != 0) return;

    // ---- the border: keys as distances from the least, `bits` low bits of them
    // undecided, the higher ones equal to the border's; `rank` pages are still
    // to be taken from the `inside` ones that share them
    const uint32_t base = s_min;
    int bits = 32 - __clz(s_max - base);  // 0: all equal
    uint32_t border = 0, rank = want, inside = m;
    while (bits > 0 && inside > kFew) {
        const int shift = max(0, bits - kBinBits);
        for (int i0 = tid; i0 < m; i0 += kBatch * kThreads) {
            uint32_t k[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) k[j] = i0 + j * kThreads < m ? s_key[i0 + j * kThreads] - base : 0u;
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (i0 + j * kThreads < m && (bits == 32 || (k[j] >> bits) == (border >> bits)))
                    atomicAdd(&s_hist[(k[j] >> shift) & ((1u << (bits - shift)) - 1)], 1u);
        }
        __syncthreads();
        // bins from the largest down: thread d takes bin kBins - 1 - d
        const int bin = kBins - 1 - tid;
        const uint32_t cnt = s_hist[bin];
        const uint32_t before = block_scan<kThreads>(cnt, s_warp);
        s_hist[bin] = 0;
        if (before < rank && before + cnt >= rank) {
            s_digit = bin;
            s_above = before;
            s_inside = cnt;
        }
        __syncthreads();
        border |= s_digit << shift;
        rank -= s_above;
        inside = s_inside;
        bits = shift;
        __syncthreads();
    }
    // ---- a bit per candidate: above the border; inside it, either a short list
    // to rank one against all, or (all equal) the first ones
    const bool few = inside <= kFew;
    const int words = (m + 31) / 32;
    for (int w0 = warp; w0 < words; w0 += kBatch * C::kWarps) {
        uint32_t k[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = (w0 + j * C::kWarps) * 32 + lane;
            k[j] = i < m ? s_key[i] - base : 0u;
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int w = w0 + j * C::kWarps, i = w * 32 + lane;
            if (w >= words) break;
            const uint32_t top = bits == 32 ? 0u : k[j] >> bits, edge = bits == 32 ? 0u : border >> bits;
            const uint32_t above = __ballot_sync(0xffffffffu, i < m && top > edge);
            if (lane == 0) s_bits[w] = above;
            if (few && i < m && top == edge) s_list[atomicAdd(&s_count, 1u)] = make_uint2(k[j], i);
        }
    }
    __syncthreads();
    if (few) {
        if (tid < inside) {
            const uint2 mine = s_list[tid];
            uint32_t better = 0;
            for (uint32_t j = 0; j < inside; ++j) {
                const uint2 o = s_list[j];
                better += o.x > mine.x || (o.x == mine.x && o.y < mine.y);
            }
            if (better < rank) atomicOr(&s_bits[mine.y >> 5], 1u << (mine.y & 31));
        }
    } else {
        // more than a few equal keys (bits == 0): by index, `rank` of them
        const int per = (m + kThreads - 1) / kThreads;
        const int i0 = min(m, tid * per), i1 = min(m, i0 + per);
        uint32_t equal = 0;
        for (int i = i0; i < i1; ++i) equal += s_key[i] - base == border;
        uint32_t at = block_scan<kThreads>(equal, s_warp);
        for (int i = i0; i < i1 && at < rank; ++i)
            if (s_key[i] - base == border) {
                atomicOr(&s_bits[i >> 5], 1u << (i & 31));
                ++at;
            }
    }
    __syncthreads();
    // ---- the chosen pages in ascending order, between those that are always
    // read: each thread a run of words
    for (int i = tid; i < nf + p.num_last; i += kThreads) {
        const bool front = i < nf;
        out[front ? i : want + i] = front ? i : n - K + want + i;
    }
    const int per = (words + kThreads - 1) / kThreads;
    const int w0 = min(words, tid * per), w1 = min(words, w0 + per);
    uint32_t cnt = 0;
    for (int w = w0; w < w1; ++w) cnt += __popc(s_bits[w]);
    const uint32_t end = nf + want;
    uint32_t at = nf + block_scan<kThreads>(cnt, s_warp);
    for (int w = w0; w < w1; ++w)
        for (uint32_t x = s_bits[w]; x && at < end; x &= x - 1) out[at++] = nf + w * 32 + __ffs(x) - 1;
}

template <int D, int NT, int kThreads>
cudaError_t go(const PageSelectParams& p, int cluster, cudaStream_t stream) {
    auto kern = page_select_kernel<D, NT, kThreads>;
    const int pages = (p.max_seq_len - 1) / p.block_size + 1;
    auto smem_of = [](int n) { return PsCfg<D, NT, kThreads>::kFixed + 4 * (n + (n + 31) / 32); };
    const int smem = smem_of(pages);
    // (the most that any call takes: calls of several threads set the same)
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_of(kPageSelectMaxPages));
    if (e != cudaSuccess) return e;
    return launch_cluster(kern, dim3((unsigned)(cluster * p.num_tokens * p.Hkv)), dim3(kThreads), smem, cluster, stream,
                          p);
}

}  // namespace

cudaError_t launch_page_select(const PageSelectParams& p, int head_dim, int num_sms, cudaStream_t stream) {
    const int pages = (p.max_seq_len - 1) / p.block_size + 1;
    const int64_t units = (int64_t)p.num_tokens * p.Hkv;
    // All CTAs run at once where they can, each with as many warps as that leaves
    // room for: CTAs of 256 threads (two per SM), in clusters, up to two units per
    // SM; beyond that CTAs of 128 threads (five per SM), two to a unit up to three
    // units per SM. Measured with 8 kv heads, contexts of 4096 to 65536 tokens, in
    // clusters of 1 / 2 / 4 / 8:
    //     requests   256 threads                 128 threads
    //        4        9.2 / 7.9 / 7.4 / 7.2      12.2 / 9.1 / 7.9 / 7.5 us
    //       16       11.8 / 10.1 / 11.9 / 15.7   13.5 / 11.0 / 10.0 / 10.4
    //       32       12.6 / 16.3 / 20.6 / 29.7   17.7 / 14.4 / 13.0 / 16.0
    //       48       18.7 / 21.6 / 29.0 / 43.1   22.9 / 15.8 / 17.6 / 22.3
    //       96       29.3 / 44.0 / 64.5 / 107    25.4 / 26.6 / 33.3 / 43.8
    // (where that many CTAs fit beside their scores: 4 bytes per page of max_seq_len. 96
    // requests of 4096 to 16384 tokens with max_seq_len of up to 9600 pages 11.8 us, of 16384
    // pages 14.5, of 32768 pages 29.1; 16 requests 6.5, 6.5 and 10.3.)
    const bool two = p.G > 8, wide = units <= 2 * num_sms;
    int n = 1;
    while (wide && n < 8 && units * n <= num_sms && pages > n * 16 * kCtaTiles) n *= 2;
    if (!wide && units <= 3 * num_sms && pages > 16 * kCtaTiles) n = 2;
    auto by_width = [&](auto d, auto nt) {
        return wide ? go<decltype(d)::value, decltype(nt)::value, 256>(p, n, stream)
                    : go<decltype(d)::value, decltype(nt)::value, 128>(p, n, stream);
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    using N1 = std::integral_constant<int, 1>;
    using N2 = std::integral_constant<int, 2>;
    if (head_dim == 128) return two ? by_width(D128{}, N2{}) : by_width(D128{}, N1{});
    if (head_dim == 64) return two ? by_width(D64{}, N2{}) : by_width(D64{}, N1{});
    return cudaErrorInvalidValue;
}

}  // namespace pka
