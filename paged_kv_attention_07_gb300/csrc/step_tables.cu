// step_tables.cu -- the metadata of one serving step, made on the GPU from the
// requests' lengths: new pages taken from a free list into the block table,
// query_start_loc, seq_lens, and each new token's position and cache slot.
//
//   seq_r   = ctx_r + new_r
//   need_r  = ceil(seq_r / bs) - ceil(ctx_r / bs)      pages the request takes
//   page j of request r's need is free_pages[head + sum_{i<r} need_i + j]
//   token t of request r: p = ctx_r + (t - qsl_r), slot = table[r][p / bs] * bs + p % bs
//
// Two prefix sums over at most kMaxRequests requests, then one search and write
// per token. The bytes are few (12 per token), so the cost is latency and, with
// many tokens, instructions: a warp takes a contiguous run of tokens and starts
// each search where the last one ended (300 requests with 67214 tokens on 8 CTAs
// 8.2 us, 11.4 us with a search of its own for every token; 48 requests with one
// token each 3.3 us). Every CTA repeats the prefix sums in its own shared memory
// (a few kilobytes from L2) and writes its share of the tokens and pages; the
// page of a token on a new page comes from the free list itself, not from the
// table entry another CTA writes. So no CTA waits for another, but where the
// list's head is advanced in place: then one cluster, whose barrier separates
// the reads of the head from its update (67214 tokens 8.2 us, 5.1 us
// otherwise).
#include "common.cuh"
#include "params.cuh"
#include "plan.cuh"

namespace pka {

namespace {

// Threads of a CTA: few for a decode step of few requests (one each), else enough
// for kMaxRequests at a handful each (48 requests 3.3 us, 3.7 us with 1024).
constexpr int kStFew = 256, kStMany = 1024;
constexpr int kStBatch = 4;  // tokens of a thread in flight
constexpr int kStCluster = 8;  // CTAs at most, where the head is advanced in place
constexpr int kStCtas = 128;   // and where it is not

// x / bs: a shift where the page size is a power of two (log2 >= 0).
PKA_DEVICE int page_of(uint32_t x, int bs, int log2) { return (int)(log2 >= 0 ? x >> log2 : x / (uint32_t)bs); }
PKA_DEVICE int pages_of(int tokens, int bs, int log2) { return page_of((uint32_t)tokens + (uint32_t)bs - 1, bs, log2); }

// Last r in [lo, hi] with first[r] <= x (first[lo] <= x).
PKA_DEVICE int last_at_most(const int32_t* first, int lo, int hi, int x) {
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) step_tables_kernel(StepTablesParams p) {
    constexpr int kWarps = kThreads / 32;
    constexpr int kPer = kThreads == kStFew ? 1 : kMaxRequests / kThreads;  // requests of a thread, at most
    static_assert(kWarps <= 32 && (kThreads == kStFew || kPer * kThreads == kMaxRequests), "");
    extern __shared__ int32_t s_req[];
    int32_t* s_qsl = s_req;                   // first token of each request
    int32_t* s_first = s_qsl + p.num_reqs;    // pages taken by the requests before it
    int32_t* s_ctx = s_first + p.num_reqs;    // its cached tokens
    __shared__ long long s_tok[kWarps + 1], s_pag[kWarps + 1];
    grid_dep_launch();
    grid_dep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ncta = gridDim.x, cta = blockIdx.x;
    const int B = p.num_reqs, bs = p.block_size, log2 = p.bs_log2;
    const int head = *p.free_head;
    const long long longest = (long long)p.max_blocks * bs;

    // ---- lengths: validate, sum, scan (each thread a contiguous run of requests)
    const int per = (B + kThreads - 1) / kThreads;  // <= kPer
    const int r0 = min(B, tid * per), r1 = min(B, r0 + per);
    int err = 0;
    long long tok = 0, pag = 0;
    int nw[kPer], nd[kPer], cl[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        nw[i] = nd[i] = cl[i] = 0;
        const int r = r0 + i;
        if (r >= r1) continue;
        const int c = p.ctx_lens[r], q = p.query_lens[r];
        const long long s = (long long)c + q;
        if (q < 0) err |= PKA_DEVERR_QUERY_LEN;
        if (c < 0) err |= PKA_DEVERR_SEQ_LEN;
        if (s > longest) err |= PKA_DEVERR_BLOCK_TABLE;
        if (q < 0 || c < 0 || s > longest) continue;
        nw[i] = q;
        cl[i] = c;
        nd[i] = pages_of((int)s, bs, log2) - pages_of(c, bs, log2);  // (s <= longest, which fits)
        tok += q;
        pag += nd[i];
    }
    long long ti = tok, pi = pag;  // inclusive scans within the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, ti, o), b = __shfl_up_sync(0xffffffffu, pi, o);
        if (lane >= o) {
            ti += a;
            pi += b;
        }
    }
    if (lane == 31) {
        s_tok[warp] = ti;
        s_pag[warp] = pi;
    }
    __syncthreads();
    if (warp == 0) {
        const long long a = lane < kWarps ? s_tok[lane] : 0, b = lane < kWarps ? s_pag[lane] : 0;
        long long ai = a, bi = b;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, ai, o), y = __shfl_up_sync(0xffffffffu, bi, o);
            if (lane >= o) {
                ai += x;
                bi += y;
            }
        }
        if (lane < kWarps) {
            s_tok[lane] = ai - a;
            s_pag[lane] = bi - b;
        }
        if (lane == 31) {
            s_tok[kWarps] = ai;
            s_pag[kWarps] = bi;
        }
    }
    __syncthreads();
    const long long total = s_tok[kWarps], taken = s_pag[kWarps];
    if (total > p.num_tokens) err |= PKA_DEVERR_QUERY_START_LOC;
    if (head < 0 || taken > (long long)p.num_free - head) err |= PKA_DEVERR_CAPACITY;
    const int any = __syncthreads_or(err);
    cluster_arrive();  // this CTA has read the list's head (here, where no stores are in flight to wait for)
    if (any) {
        // nothing is taken: empty requests and no slots, so that the calls
        // that read these tables write and read nothing
        if (err) set_error(p.err, err);
        for (int r = cta * kThreads + tid; r < B; r += ncta * kThreads) {
            p.qsl[r + 1] = 0;
            p.seq_lens[r] = 0;
        }
        if (cta == 0 && tid == 0) p.qsl[0] = 0;
        for (int64_t t = (int64_t)cta * kThreads + tid; t < p.num_tokens; t += (int64_t)ncta * kThreads) {
            if (p.positions) p.positions[t] = -1;
            p.slots[t] = -1;
        }
    } else {
        // the sums fit 32 bits: total <= num_tokens, taken <= num_free
        int t0 = (int)(s_tok[warp] + ti - tok), g0 = (int)(s_pag[warp] + pi - pag);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int r = r0 + i;
            if (r >= r1) continue;
            s_qsl[r] = t0;
            s_first[r] = g0;
            s_ctx[r] = cl[i];
            t0 += nw[i];
            g0 += nd[i];
            if (r % ncta == cta) {
                p.qsl[r + 1] = t0;
                p.seq_lens[r] = cl[i] + nw[i];
            }
        }
        if (cta == 0 && tid == 0) p.qsl[0] = 0;
        __syncthreads();
        const int32_t* list = p.free_pages + head;
        // ---- the new pages' table entries
        for (int j = cta * kThreads + tid; j < (int)taken; j += ncta * kThreads) {
            const int r = last_at_most(s_first, 0, B - 1, j);
            const int held = pages_of(s_ctx[r], bs, log2);
            p.block_table[(int64_t)r * p.max_blocks + held + (j - s_first[r])] = list[j];
        }
        // ---- the tokens: 32 neighbours at a time, kStBatch times, so that their table loads overlap
        const int nwarps = ncta * (kThreads / 32), me = cta * (kThreads / 32) + warp;
        const int rounds = (int)((p.num_tokens + 31) / 32);  // (num_tokens <= INT32_MAX)
        const int i0 = (int)((int64_t)rounds * me / nwarps), i1 = (int)((int64_t)rounds * (me + 1) / nwarps);
        const int last = (int)total - 1;
        int r0 = i0 < i1 && last >= 0 ? last_at_most(s_qsl, 0, B - 1, min(i0 * 32, last)) : 0;
        for (int ib = i0; ib < i1; ib += kStBatch) {
            int pos[kStBatch], off[kStBatch], id[kStBatch];
#pragma unroll
            for (int i = 0; i < kStBatch; ++i) {
                pos[i] = id[i] = -1;
                off[i] = 0;
                const int tb = (ib + i) * 32, t = tb + lane;
                if (ib + i >= i1 || tb > last) continue;  // (the same for the whole warp)
                const int end = min(tb + 31, last), x = min(t, last);
                int r = r0;
                if (r0 + 1 < B && s_qsl[r0 + 1] <= end) {
                    const int far = min(r0 + 31, B - 1);  // more only with requests that have no tokens
                    r = last_at_most(s_qsl, r0, s_qsl[far] > end ? far : B - 1, x);
                }
                r0 = __shfl_sync(0xffffffffu, r, 31);
                if (t > last) continue;
                const int c = s_ctx[r];
                pos[i] = c + (t - s_qsl[r]);
                const int held = pages_of(c, bs, log2), page = page_of((uint32_t)pos[i], bs, log2);
                off[i] = pos[i] - page * bs;
                id[i] = page < held ? p.block_table[(int64_t)r * p.max_blocks + page] : list[s_first[r] + page - held];
            }
#pragma unroll
            for (int i = 0; i < kStBatch; ++i) {
                const int64_t t = (int64_t)(ib + i) * 32 + lane;
                if (ib + i >= i1 || t >= p.num_tokens) continue;
                if (p.positions) p.positions[t] = pos[i];
                p.slots[t] = id[i] >= 0 ? (int64_t)id[i] * bs + off[i] : -1;
            }
        }
    }
    // every CTA has read the list's head before it is advanced (in place, perhaps)
    cluster_wait();
    if (cta == 0 && tid == 0) *p.free_head_out = any ? head : head + (int)taken;
}

}  // namespace

template <int kThreads>
static cudaError_t go(const StepTablesParams& p, cudaStream_t stream) {
    auto kern = step_tables_kernel<kThreads>;
    const size_t smem = sizeof(int32_t) * 3 * (size_t)p.num_reqs;
    if (smem > 47 * 1024) {  // past what every kernel may use; the most that any call takes
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)sizeof(int32_t) * 3 * kMaxRequests);
        if (e != cudaSuccess) return e;
    }
    // a token per thread, up to the CTAs there may be; in place, a cluster from some tokens on
    const bool in_place = p.free_head == p.free_head_out;
    const int64_t ctas = (p.num_tokens + kThreads - 1) / kThreads;
    const int n = in_place ? (ctas < 4 ? 1 : kStCluster) : (int)std::max<int64_t>(1, std::min<int64_t>(ctas, kStCtas));
    return launch_cluster(kern, dim3(n), dim3(kThreads), smem, in_place ? n : 1, stream, p);
}

cudaError_t launch_step_tables(const StepTablesParams& p, cudaStream_t stream) {
    return p.num_reqs <= kStFew && p.num_tokens <= 4 * kStFew ? go<kStFew>(p, stream) : go<kStMany>(p, stream);
}

}  // namespace pka
