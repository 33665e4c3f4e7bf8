// page_select.cu -- the pages each new token reads: the best of its request's
// pages by an upper bound of its scores over each page.
//
// Token t at position p of request r, kv head g: pages 0 .. p / bs, the last
// one its own. With q's 8-bit codes c (2^x the least power of two with
// max |q| <= 127 * 2^x, c = q / 2^x rounded to nearest even) and a page's bounds
//   score = max over the heads h of the group of 2^x_h * 2^e * sum_i max(c_i lo_i, c_i hi_i)
// which no product <q, key> of the page exceeds (up to q's rounding). Every
// term is an integer and the sum stays below 2^21: int32 tensor-core
// accumulation is exact, the two factors are powers of two, so the scores are
// the same bits in any order of work and ties are real ties.
//
// sum_i max(c_i lo_i, c_i hi_i) = <min(c, 0), lo> + <max(c, 0), hi>: one product
// of length 2 d with the page's record as it lies in memory (lo then hi).
// One warp scores 16 pages: it loads their 16 records (2 d bytes each) straight
// into the A fragments of m16n8k32 -- which of a fragment's columns holds which
// element does not matter as long as B agrees, so each lane's 16-byte load
// feeds two MMAs -- and the queries' codes wait as B fragments in registers.
//
// One cluster per (token, kv head): its CTAs score a slice of the pages each
// and leave the scores in the first CTA's shared memory, which then picks the
// pages: a radix selection of the num_pages-th largest score, digit by digit,
// and one prefix sum that writes the chosen pages in ascending order (ties: the
// lowest page). The scores never go to memory. HBM-bound for a full batch:
// 2 d + 4 bytes per (page, kv head).
#include "common.cuh"
#include "params.cuh"

namespace pka {

namespace {

constexpr int kPsThreads = 256;
constexpr int kPsWarps = kPsThreads / 32;

PKA_DEVICE void mma_s8(int32_t (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A float's bits as an unsigned key of the same order.
PKA_DEVICE uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);  // -0 -> +0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Exclusive sum of v over the block's threads (packed counts); total to all.
PKA_DEVICE uint32_t block_scan(uint32_t v, uint32_t* s_warp, uint32_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPsWarps; ++w) {
        const uint32_t x = s_warp[w];
        before += w < warp ? x : 0u;
        all += x;
    }
    __syncthreads();
    *total = all;
    return before + incl - v;
}

template <int D, int NT>
__global__ void __launch_bounds__(kPsThreads) page_select_kernel(PageSelectParams p) {
    constexpr int kSteps = 2 * D / 32;            // MMAs per 16 pages and 8 heads
    extern __shared__ uint32_t s_key[];           // scores of the candidates, as keys (first CTA's is used)
    __shared__ __align__(16) int8_t s_q[NT * 8][2 * D];         // per head: min(c, 0) then max(c, 0), in the records' order
    __shared__ float s_unit[NT * 8];
    __shared__ uint32_t s_hist[256];
    __shared__ uint32_t s_warp[kPsWarps];
    __shared__ uint32_t s_min, s_max, s_digit, s_above;
    grid_dep_launch();
    grid_dep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ncta = cluster_size(), cta = cluster_rank();
    const int g = blockIdx.y;
    const int t = (int)(blockIdx.x / ncta);
    // ---- the token's request and position (the same for the whole cluster)
    const int r = request_of(p.qsl, p.num_reqs, t);
    if (r < 0) return;  // a row behind the last sequence
    const int q1 = __ldg(p.qsl + r + 1), sl = __ldg(p.seq_lens + r);
    const long long pos = (long long)sl - q1 + t;
    if (t < __ldg(p.qsl + r) || pos < 0 || sl > p.max_seq_len || pos >= sl) {
        if (tid == 0) set_error(p.err, PKA_DEVERR_SEQ_LEN);
        return;
    }
    const int n = (int)pos / p.block_size + 1;  // pages up to the token's own
    int32_t* out = p.sel + ((int64_t)t * p.Hkv + g) * p.num_pages;
    const int K = p.num_pages;
    if (n <= K) {  // all of them
        for (int i = cta * kPsThreads + tid; i < K; i += ncta * kPsThreads) out[i] = i < n ? i : -1;
        return;
    }
    const int nf = p.num_first, m = n - nf - p.num_last, want = K - nf - p.num_last;
    for (int i = cta * kPsThreads + tid; i < nf + p.num_last; i += ncta * kPsThreads)
        out[i < nf ? i : K - p.num_last + (i - nf)] = i < nf ? i : n - p.num_last + (i - nf);
    if (want == 0) return;
    cluster_arrive();  // waited for before the first store to the first CTA

    // ---- the queries' codes, one warp per head
    if (tid < NT * 8) s_unit[tid] = 0.f;
    __syncthreads();
    for (int h = warp; h < NT * 8; h += kPsWarps) {
        constexpr int kE = D / 32;
        float x[kE];
        float a = 0.f;
        const bool ok = h < p.G;
#pragma unroll
        for (int i = 0; i < kE; ++i) {
            x[i] = ok ? __bfloat162float(p.q[((int64_t)t * p.Hq + g * p.G + h) * D + lane * kE + i]) : 0.f;
            a = fmaxf(a, fabsf(x[i]));
            if (!(fabsf(x[i]) <= 3.4e38f)) a = INFINITY;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        const bool finite = a <= 3.4e38f;  // a head with a NaN or an infinity scores 0 everywhere
        const int e = finite ? bound_exponent(a) : 0;
        const float unit = exp2i(-e);
#pragma unroll
        for (int i = 0; i < kE; ++i) {
            const int c = finite ? __float2int_rn(x[i] * unit) : 0;
            s_q[h][lane * kE + i] = (int8_t)min(c, 0);
            s_q[h][D + lane * kE + i] = (int8_t)max(c, 0);
        }
        if (lane == 0) s_unit[h] = exp2i(e);
    }
    __syncthreads();
    // B fragments: head (lane / 4), 16-byte piece (lane % 4) of each 64 bytes of the record
    uint32_t b[NT][kSteps][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int s = 0; s < kSteps; s += 2) {
            const uint4 v = *reinterpret_cast<const uint4*>(&s_q[nt * 8 + (lane >> 2)][s * 32 + (lane & 3) * 16]);
            b[nt][s][0] = v.x, b[nt][s][1] = v.y, b[nt][s + 1][0] = v.z, b[nt][s + 1][1] = v.w;
        }
    float unit[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        unit[nt][0] = s_unit[nt * 8 + 2 * (lane & 3)];
        unit[nt][1] = s_unit[nt * 8 + 2 * (lane & 3) + 1];
    }

    // ---- scores of this CTA's slice of the candidates [nf, nf + m)
    const int32_t* bt = p.block_table + (int64_t)r * p.max_blocks + nf;
    const int tiles = (m + 15) / 16;
    cluster_wait();
    for (int tile = cta * kPsWarps + warp; tile < tiles; tile += ncta * kPsWarps) {
        uint32_t a[2][kSteps / 2][4];
        float scale[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int i = tile * 16 + half * 8 + (lane >> 2);
            int blk = i < m ? __ldg(bt + i) : 0;
            const bool ok = blk >= 0 && blk < p.num_blocks;
            if (!ok) {
                set_error(p.err, PKA_DEVERR_BLOCK_ID);
                blk = 0;
            }
            const int64_t page = (int64_t)blk * p.Hkv + g;
            const uint4* rec = reinterpret_cast<const uint4*>(p.bounds + page * 2 * D) + (lane & 3);
#pragma unroll
            for (int s = 0; s < kSteps / 2; ++s) {
                const uint4 v = __ldg(rec + s * 4);
                a[half][s][0] = v.x, a[half][s][1] = v.y, a[half][s][2] = v.z, a[half][s][3] = v.w;
            }
            scale[half] = ok ? __ldg(p.scales + page) : -INFINITY;
        }
        float best[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            int32_t c[4] = {0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < kSteps / 2; ++s) {
                mma_s8(c, a[0][s][0], a[1][s][0], a[0][s][1], a[1][s][1], b[nt][2 * s][0], b[nt][2 * s][1]);
                mma_s8(c, a[0][s][2], a[1][s][2], a[0][s][3], a[1][s][3], b[nt][2 * s + 1][0], b[nt][2 * s + 1][1]);
            }
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (nt * 8 + 2 * (lane & 3) + j < p.G)
                        best[half] = fmaxf(best[half], (float)c[half * 2 + j] * scale[half] * unit[nt][j]);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float v = best[half];
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
            // a page that bounds nothing (scale +inf) comes first, one that does not exist last
            if (fabsf(scale[half]) == INFINITY) v = scale[half];
            const int i = tile * 16 + half * 8 + (lane >> 2);
            if ((lane & 3) == 0 && i < m) store_cluster(&s_key[i], 0, order_key(v));
        }
    }
    cluster_barrier();
    if (cta != 0) return;

    // ---- the want-th largest key: the bits that all keys share are skipped,
    // then eight bits at a time from the top
    uint32_t lo = 0xffffffffu, hi = 0u;
    for (int i = tid; i < m; i += kPsThreads) {
        lo = min(lo, s_key[i]);
        hi = max(hi, s_key[i]);
    }
    if (tid == 0) s_min = 0xffffffffu, s_max = 0u;
    __syncthreads();
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
        atomicMin(&s_min, lo);
        atomicMax(&s_max, hi);
    }
    __syncthreads();
    lo = s_min, hi = s_max;
    int bits = lo == hi ? 0 : 32 - __clz(lo ^ hi);  // low bits in which keys differ
    uint32_t prefix = bits == 32 ? 0u : (hi >> bits) << bits;
    uint32_t rank = want;  // among the keys that share the prefix
    while (bits > 0) {
        const int shift = max(0, bits - 8), width = bits - shift;
        for (int i = tid; i < 256; i += kPsThreads) s_hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < m; i += kPsThreads) {
            const uint32_t k = s_key[i];
            if (bits == 32 || (k >> bits) == (prefix >> bits)) atomicAdd(&s_hist[(k >> shift) & ((1u << width) - 1)], 1u);
        }
        __syncthreads();
        // digits from the largest down: thread d takes digit 255 - d
        const uint32_t cnt = s_hist[255 - tid];
        uint32_t total;
        const uint32_t before = block_scan(cnt, s_warp, &total);
        if (before < rank && before + cnt >= rank) {
            s_digit = 255 - tid;
            s_above = before;
        }
        __syncthreads();
        prefix |= s_digit << shift;
        rank -= s_above;
        bits = shift;
        __syncthreads();
    }
    // ---- write the chosen pages in ascending order: each thread a contiguous
    // run of pages; keys above the threshold, and the first `rank` that equal it
    const int per = (m + kPsThreads - 1) / kPsThreads;
    const int i0 = min(m, tid * per), i1 = min(m, i0 + per);
    uint32_t above = 0, equal = 0;
    for (int i = i0; i < i1; ++i) {
        above += s_key[i] > prefix;
        equal += s_key[i] == prefix;
    }
    uint32_t total;
    const uint32_t packed = block_scan(above << 16 | equal, s_warp, &total);
    uint32_t at_above = packed >> 16, at_equal = packed & 0xffffu;
    for (int i = i0; i < i1; ++i) {
        const uint32_t k = s_key[i];
        if (k > prefix || (k == prefix && at_equal < rank)) out[nf + at_above + min(at_equal, rank)] = nf + i;
        at_above += k > prefix;
        at_equal += k == prefix;
    }
}

template <int D, int NT>
cudaError_t go(const PageSelectParams& p, int num_sms, cudaStream_t stream) {
    auto kern = page_select_kernel<D, NT>;
    const int pages = (p.max_seq_len + p.block_size - 1) / p.block_size;
    const size_t smem = sizeof(uint32_t) * (size_t)pages;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kPageSelectMaxPages * 4);
    if (e != cudaSuccess) return e;
    // as many CTAs per (token, kv head) as fill the GPU once, each with at
    // least one tile of 16 pages per warp
    int n = 1;
    while (n < 8 && (int64_t)p.num_tokens * p.Hkv * n < num_sms && pages > n * kPsWarps * 16) n *= 2;
    return launch_cluster(kern, dim3((unsigned)n * (unsigned)p.num_tokens, p.Hkv), dim3(kPsThreads), smem, n, stream, p);
}

}  // namespace

cudaError_t launch_page_select(const PageSelectParams& p, int head_dim, int num_sms, cudaStream_t stream) {
    const bool two = p.G > 8;
    if (head_dim == 128) return two ? go<128, 2>(p, num_sms, stream) : go<128, 1>(p, num_sms, stream);
    if (head_dim == 64) return two ? go<64, 2>(p, num_sms, stream) : go<64, 1>(p, num_sms, stream);
    return cudaErrorInvalidValue;
}

}  // namespace pka
