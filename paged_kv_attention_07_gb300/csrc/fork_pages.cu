// fork_pages.cu -- block tables whose rows go on from other rows (beams and
// samples that fork, change places and end), with shared pages counted and freed,
// and the copies of partly filled pages.
//
// fork_pages_kernel. Row r with n_r rows that go on from it adds n_r - 1 to the
// count of each of its pages (its partly filled last page, which only the first
// of those rows keeps: 0, or -1 when there is none), so rows with n_r = 1, most
// of them in a server's batch, touch no count. Only a row with n_r = 0 can free a
// page. The order of the freed pages must not hang on that of the atomics: each
// entry of such a row that finds its page's count below 0 enters its place into
// the count (the least place stays), after which the page's first entry knows
// that it is the first, and the freed pages are numbered by counts per row and a
// prefix sum. Three barriers separate these steps, so the work is one cluster's;
// what bounds it is their latency and the table's bytes.
//
// copy_pages_kernel: bytes.
#include <algorithm>

#include "common.cuh"
#include "params.cuh"
#include "plan.cuh"

namespace pka {

namespace {

constexpr int kFpThreads = 1024, kFpWarps = kFpThreads / 32;
constexpr int kFpCluster = 8;

// Exclusive prefix sum of v over the CTA's threads; *total its sum. `s`: kFpWarps + 1 words.
PKA_DEVICE int block_scan(int v, int* s, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s[warp] = x;
    __syncthreads();
    if (warp == 0) {
        const int w = s[lane];
        int y = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
        }
        s[lane] = y - w;
        if (lane == 31) s[kFpWarps] = y;
    }
    __syncthreads();
    const int before = s[warp] + x - v;
    *total = s[kFpWarps];
    __syncthreads();
    return before;
}

__global__ void __launch_bounds__(kFpThreads) fork_pages_kernel(const ForkPagesParams p) {
    extern __shared__ int32_t s_rows[];
    int32_t* s_children = s_rows;              // [num_rows] rows that go on from each
    int32_t* s_first = s_children + p.num_rows;  // [num_rows] the first of them
    int32_t* s_held = s_first + p.num_rows;      // [num_rows] its pages; bit 31: the last one is partly filled
    int32_t* s_freed = s_held + p.num_rows;      // [num_rows] pages that it is the first to free
    int32_t* s_fresh = s_freed + p.num_rows;     // [num_rows_out] the taken page's number, or -1
    __shared__ int s_scan[kFpWarps + 1];
    static_assert(kFpWarps == 32, "");
    grid_dep_launch();
    grid_dep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ncta = (int)cluster_size(), cta = (int)cluster_rank();
    const int B = p.num_rows, N = p.num_rows_out, bs = p.block_size;
    const int head = *p.free_head;
    int err = 0;

    // ---- lengths and parents
    for (int r = tid; r < B; r += kFpThreads) {
        const int c = p.ctx_lens[r];
        if (c < 0) err |= PKA_DEVERR_SEQ_LEN;
        if (c > (long long)p.max_blocks * bs) err |= PKA_DEVERR_BLOCK_TABLE;
        s_children[r] = 0;
        s_first[r] = INT32_MAX;
        s_freed[r] = 0;
        s_held[r] = err ? 0 : (c / bs + (c % bs != 0)) | (c % bs != 0 ? 1 << 31 : 0);
    }
    __syncthreads();
    for (int i = tid; i < N; i += kFpThreads) {
        const int r = p.parents[i];
        if (r >= B) err |= PKA_DEVERR_INDEX;
        if (r < 0 || r >= B) continue;
        atomicAdd(&s_children[r], 1);
        atomicMin(&s_first[r], i);
    }
    __syncthreads();
    int taken = 0;  // rows that take a page, numbered in order
    for (int i0 = 0; i0 < N; i0 += kFpThreads) {
        const int i = i0 + tid, r = i < N ? p.parents[i] : -1;
        const bool fresh = r >= 0 && r < B && s_held[r] < 0 && s_first[r] != i;
        int sum;
        const int before = block_scan(fresh, s_scan, &sum);
        if (i < N) s_fresh[i] = fresh ? taken + before : -1;
        taken += sum;
    }
    if (head < 0 || taken > (long long)p.num_free - head) err |= PKA_DEVERR_CAPACITY;
    const int any = __syncthreads_or(err);
    if (any) {
        if (cta == 0) {
            if (err) set_error(p.err, err);
            for (int i = tid; i < N; i += kFpThreads) {
                p.ctx_lens_out[i] = 0;
                p.copy_src[i] = p.copy_dst[i] = -1;
            }
        }
        cluster_barrier();  // every CTA has read the list's head
        if (cta == 0 && tid == 0) *p.free_head_out = head;
        return;
    }

    // ---- the new rows
    const int me = cta * kFpWarps + warp, nwarps = ncta * kFpWarps;
    for (int i = me; i < N; i += nwarps) {
        const int r = p.parents[i];
        const int held = r < 0 ? 0 : s_held[r] & INT32_MAX, fresh = s_fresh[i];
        const int32_t* from = p.block_table + (int64_t)max(r, 0) * p.max_blocks;
        int32_t* to = p.block_table_out + (int64_t)i * p.max_blocks;
        const int same = fresh >= 0 ? held - 1 : held;
        for (int c = lane; c < same; c += 32) to[c] = from[c];
        if (lane == 0) {
            const int page = fresh >= 0 ? p.free_pages[head + fresh] : -1;
            if (fresh >= 0) to[held - 1] = page;
            p.ctx_lens_out[i] = r < 0 ? 0 : p.ctx_lens[r];
            p.copy_src[i] = fresh >= 0 ? from[held - 1] : -1;
            p.copy_dst[i] = page;
        }
    }
    // ---- the counts
    for (int r = me; r < B; r += nwarps) {
        const int n = s_children[r], held = s_held[r] & INT32_MAX;
        const bool partial = s_held[r] < 0;
        if (n == 1) continue;
        const int32_t* row = p.block_table + (int64_t)r * p.max_blocks;
        for (int c = lane; c < held; c += 32) {
            const int page = row[c];
            const int more = partial && c == held - 1 ? min(n, 1) - 1 : n - 1;
            if (page >= p.num_blocks) set_error(p.err, PKA_DEVERR_BLOCK_ID);
            else if (page >= 0 && more != 0) atomicAdd(&p.share_counts[page], more);
        }
    }
    cluster_barrier();
    // ---- the first place of each page that nobody holds
    for (int r = me; r < B; r += nwarps) {
        if (s_children[r] != 0) continue;
        const int held = s_held[r] & INT32_MAX;
        const int32_t* row = p.block_table + (int64_t)r * p.max_blocks;
        for (int c = lane; c < held; c += 32) {
            const int page = row[c];
            if (page >= 0 && page < p.num_blocks && __ldcg(&p.share_counts[page]) < 0)
                atomicMin(&p.share_counts[page], INT32_MIN + r * p.max_blocks + c);
        }
    }
    cluster_barrier();
    for (int r = me; r < B; r += nwarps) {
        if (s_children[r] != 0) continue;
        const int held = s_held[r] & INT32_MAX;
        const int32_t* row = p.block_table + (int64_t)r * p.max_blocks;
        int freed = 0;
        for (int c0 = 0; c0 < held; c0 += 32) {
            const int c = c0 + lane, page = c < held ? row[c] : -1;
            const bool mine = page >= 0 && page < p.num_blocks &&
                              __ldcg(&p.share_counts[page]) == INT32_MIN + r * p.max_blocks + c;
            freed += __popc(__ballot_sync(0xffffffffu, mine));
        }
        if (lane < ncta) store_cluster(reinterpret_cast<uint32_t*>(&s_freed[r]), lane, (uint32_t)freed);
    }
    cluster_barrier();
    // ---- their places in the list
    int total = 0;
    for (int r0 = 0; r0 < B; r0 += kFpThreads) {
        const int r = r0 + tid;
        int sum;
        const int before = block_scan(r < B ? s_freed[r] : 0, s_scan, &sum);
        if (r < B) s_first[r] = total + before;  // (the first rows are not asked for any more)
        total += sum;
    }
    __syncthreads();
    const int end = head + taken, start = end - total;
    for (int r = me; r < B; r += nwarps) {
        if (s_freed[r] == 0) continue;
        const int held = s_held[r] & INT32_MAX;
        const int32_t* row = p.block_table + (int64_t)r * p.max_blocks;
        int at = start + s_first[r];
        for (int c0 = 0; c0 < held; c0 += 32) {
            const int c = c0 + lane, page = c < held ? row[c] : -1;
            const bool mine = page >= 0 && page < p.num_blocks &&
                              __ldcg(&p.share_counts[page]) == INT32_MIN + r * p.max_blocks + c;
            const uint32_t all = __ballot_sync(0xffffffffu, mine);
            if (mine) {
                const int to = at + __popc(all & ((1u << lane) - 1));
                if (to >= 0) p.free_pages[to] = page;
                p.share_counts[page] = 0;
            }
            at += __popc(all);
        }
    }
    if (cta == 0 && tid == 0) {
        if (start < 0) set_error(p.err, PKA_DEVERR_CAPACITY);
        *p.free_head_out = max(start, 0);  // (every CTA has read the head: barriers)
    }
}

// A CTA's step: kCpPiece bytes of one page of one cache.
constexpr int kCpThreads = 256, kCpPiece = kCpThreads * 16 * 4;

__global__ void __launch_bounds__(kCpThreads) copy_pages_kernel(const __grid_constant__ CopyPagesParams p) {
    grid_dep_launch();
    grid_dep_wait();
    const int64_t total = (int64_t)p.num_pairs * p.num_caches * p.pieces;
    for (int64_t i = blockIdx.x; i < total; i += gridDim.x) {
        const int piece = (int)(i % p.pieces);
        const int64_t j = i / p.pieces;
        const int cache = (int)(j % p.num_caches), pair = (int)(j / p.num_caches);
        const int src = p.src[pair], dst = p.dst[pair];
        if (src < 0 || dst < 0) continue;
        if (src >= p.num_blocks || dst >= p.num_blocks) {
            if (threadIdx.x == 0) set_error(p.err, PKA_DEVERR_BLOCK_ID);
            continue;
        }
        const int64_t off = (int64_t)piece * kCpPiece;
        const uint8_t* from = p.caches[cache] + src * p.page_bytes + off;
        uint8_t* to = p.caches[cache] + dst * p.page_bytes + off;
        const int n = (int)min((int64_t)kCpPiece, p.page_bytes - off) / 16;
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int at = (int)threadIdx.x + k * kCpThreads;
            if (at < n) v[k] = __ldcs(reinterpret_cast<const uint4*>(from) + at);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int at = (int)threadIdx.x + k * kCpThreads;
            if (at < n) __stcs(reinterpret_cast<uint4*>(to) + at, v[k]);
        }
    }
}

}  // namespace

cudaError_t launch_fork_pages(const ForkPagesParams& p, cudaStream_t stream) {
    const size_t smem = sizeof(int32_t) * (4 * (size_t)p.num_rows + p.num_rows_out);
    if (smem > 47 * 1024) {  // past what every kernel may use; the most that any call takes
        const cudaError_t e = cudaFuncSetAttribute(fork_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)sizeof(int32_t) * 5 * kMaxRequests);
        if (e != cudaSuccess) return e;
    }
    const int rows = std::max(p.num_rows, p.num_rows_out);
    const int n = rows <= kFpWarps ? 1 : kFpCluster;
    return launch_cluster(fork_pages_kernel, dim3(n), dim3(kFpThreads), smem, n, stream, p);
}

cudaError_t launch_copy_pages(CopyPagesParams p, int num_sms, cudaStream_t stream) {
    p.pieces = (int)((p.page_bytes + kCpPiece - 1) / kCpPiece);
    const int64_t total = (int64_t)p.num_pairs * p.num_caches * p.pieces;
    const int64_t n = std::min<int64_t>(total, (int64_t)num_sms * 8);
    return launch_dependent(copy_pages_kernel, dim3((unsigned)n), dim3(kCpThreads), 0, stream, p);
}

}  // namespace pka
