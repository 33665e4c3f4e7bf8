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
// that it is the first, and the freed pages are numbered by counts per stretch of
// a row and a prefix sum. Three barriers separate these steps, so they are one
// cluster's work (one CTA's for a small table); the copies of the rows need no
// barrier and go to further clusters. What bounds it is the latency of the steps:
// a warp takes 256 columns at a time, all loads of them in flight. Measured: 4 rows of 125 pages 6.6 us
// (one CTA), 512 rows of 32 to 1024 pages, half of which end, 25.9 us: counts 10, claims and
// owners 8.5, each a scattered word per entry of 16 SMs. A kernel per step over all SMs took
// 22.9 there, but 1 to 1.5 us more for every table up to 131072 entries. 376 rows of 4 pages take 10.7.
//
// copy_pages_kernel: bytes; a CTA's step is 16 KB of one page. Measured: 256 pages of 16 KB in 32 caches 45.8 us
// (0.86 of the rate of one long copy), 2 of 32 KB in 16 caches 2.0 us.
#include <algorithm>

#include "common.cuh"
#include "params.cuh"
#include "plan.cuh"

namespace pka {

namespace {

constexpr int kFpFew = 256, kFpMany = 1024;  // threads of a CTA
constexpr int kFpCluster = 16;
constexpr int kFpSpan = 8;                   // columns of a lane in flight
constexpr int kFpStep = 32 * kFpSpan;
constexpr int kFpTasks = 8192;               // stretches of ending rows that are counted apart

// Exclusive prefix sum of v over the CTA's threads; *total its sum. `s`: 33 words.
template <int kThreads>
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
        const int w = lane < kThreads / 32 ? s[lane] : 0;
        int y = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
        }
        s[lane] = y - w;
        if (lane == 31) s[32] = y;
    }
    __syncthreads();
    const int before = s[warp] + x - v;
    *total = s[32];
    __syncthreads();
    return before;
}

// The pages of columns [c0, c0 + kFpStep) of a row before `end`, those that are pages; -1 for the others.
PKA_DEVICE void load_span(int (&page)[kFpSpan], const int32_t* row, int c0, int end, int num_blocks) {
#pragma unroll
    for (int j = 0; j < kFpSpan; ++j) {
        const int c = c0 + 32 * j + (int)(threadIdx.x & 31);
        page[j] = c < end ? __ldg(row + c) : -1;
    }
#pragma unroll
    for (int j = 0; j < kFpSpan; ++j)
        if (page[j] >= num_blocks) page[j] = -1;
}

PKA_DEVICE void load_counts(int (&count)[kFpSpan], const int (&page)[kFpSpan], const int32_t* counts) {
#pragma unroll
    for (int j = 0; j < kFpSpan; ++j) count[j] = page[j] >= 0 ? __ldcg(counts + page[j]) : 0;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) fork_pages_kernel(const ForkPagesParams p) {
    constexpr int kWarps = kThreads / 32;
    extern __shared__ int32_t s_rows[];
    int32_t* s_children = s_rows;                // [num_rows] rows that go on from each
    int32_t* s_first = s_children + p.num_rows;  // [num_rows] the first of them
    int32_t* s_held = s_first + p.num_rows;      // [num_rows] its pages; bit 31: the last one is partly filled
    int32_t* s_dead = s_held + p.num_rows;       // [num_rows] the rows that end
    int32_t* s_fresh = s_dead + p.num_rows;      // [num_rows_out] the taken page's number, or -1
    int32_t* s_freed = s_fresh + p.num_rows_out;  // [kFpTasks] pages that a stretch is the first to free
    __shared__ int s_scan[33];
    __shared__ int s_most;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ncta = (int)cluster_size(), cta = (int)cluster_rank();
    const bool copies_only = blockIdx.x >= ncta;  // not of the first cluster
    const int B = p.num_rows, N = p.num_rows_out, bs = p.block_size;
    if (tid == 0) s_most = 0;
    for (int k = tid; k < kFpTasks; k += kThreads) s_freed[k] = 0;
    grid_dep_launch();
    grid_dep_wait();
    const int head = copies_only ? 0 : *p.free_head;
    int err = 0;

    // ---- lengths and parents
    int most = 0;
    for (int r = tid; r < B; r += kThreads) {
        const int c = p.ctx_lens[r];
        if (c < 0) err |= PKA_DEVERR_SEQ_LEN;
        if (c > (long long)p.max_blocks * bs) err |= PKA_DEVERR_BLOCK_TABLE;
        s_children[r] = 0;
        s_first[r] = INT32_MAX;
        const int held = err ? 0 : c / bs + (c % bs != 0);
        s_held[r] = held | (!err && c % bs != 0 ? 1 << 31 : 0);
        most = max(most, held);
    }
    __syncthreads();
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) atomicMax(&s_most, most);
    for (int i = tid; i < N; i += kThreads) {
        const int r = p.parents[i];
        if (r >= B) err |= PKA_DEVERR_INDEX;
        if (r < 0 || r >= B) continue;
        atomicAdd(&s_children[r], 1);
        atomicMin(&s_first[r], i);
    }
    __syncthreads();
    most = s_most;
    int taken = 0, ending = 0;  // rows that take a page and rows that end, numbered in order
    for (int i0 = 0; i0 < N; i0 += kThreads) {
        const int i = i0 + tid, r = i < N ? p.parents[i] : -1;
        const bool fresh = r >= 0 && r < B && s_held[r] < 0 && s_first[r] != i;
        int sum;
        const int before = block_scan<kThreads>(fresh, s_scan, &sum);
        if (i < N) s_fresh[i] = fresh ? taken + before : -1;
        taken += sum;
    }
    if (!copies_only) {
        for (int r0 = 0; r0 < B; r0 += kThreads) {
            const int r = r0 + tid;
            const bool ends = r < B && s_children[r] == 0 && s_held[r] != 0;
            int sum;
            const int before = block_scan<kThreads>(ends, s_scan, &sum);
            if (ends) s_dead[ending + before] = r;
            ending += sum;
        }
        if (head < 0 || taken > (long long)p.num_free - head) err |= PKA_DEVERR_CAPACITY;
    }
    const int any = __syncthreads_or(err);
    if (any) {
        if (copies_only) return;
        if (cta == 0) {
            if (err) set_error(p.err, err);
            for (int i = tid; i < N; i += kThreads) {
                p.ctx_lens_out[i] = 0;
                p.copy_src[i] = p.copy_dst[i] = -1;
            }
        }
        cluster_barrier();  // every CTA has read the list's head
        if (cta == 0 && tid == 0) *p.free_head_out = head;
        return;
    }

    // ---- the new rows, by the further clusters where there are any; taken pages by the first
    const int chunks = (most + kFpStep - 1) / kFpStep;
    const bool alone = gridDim.x == ncta;
    if (copies_only || alone) {
        const int ctas = alone ? ncta : gridDim.x - ncta, c = alone ? cta : blockIdx.x - ncta;
        for (int task = c * kWarps + warp; task < N * chunks; task += ctas * kWarps) {
            const int i = task / chunks, r = p.parents[i], c0 = (task - i * chunks) * kFpStep;
            const int end = r < 0 ? 0 : (s_held[r] & INT32_MAX) - (s_fresh[i] >= 0);
            if (c0 >= end) continue;
            const int32_t* from = p.block_table + (int64_t)r * p.max_blocks;
            int32_t* to = p.block_table_out + (int64_t)i * p.max_blocks;
            int page[kFpSpan];
#pragma unroll
            for (int j = 0; j < kFpSpan; ++j) page[j] = c0 + 32 * j + lane < end ? __ldg(from + c0 + 32 * j + lane) : 0;
            // (ids of rows that go on as one are looked at here only)
            bool bad = false;
#pragma unroll
            for (int j = 0; j < kFpSpan; ++j) {
                if (c0 + 32 * j + lane >= end) continue;
                to[c0 + 32 * j + lane] = page[j];
                bad |= page[j] >= p.num_blocks;
            }
            if (bad) set_error(p.err, PKA_DEVERR_BLOCK_ID);
        }
        if (copies_only) return;
    }
    for (int i = cta * kThreads + tid; i < N; i += ncta * kThreads) {
        const int r = p.parents[i], fresh = s_fresh[i];
        int src = -1, dst = -1;
        if (fresh >= 0) {
            const int last = (s_held[r] & INT32_MAX) - 1;
            src = p.block_table[(int64_t)r * p.max_blocks + last];
            dst = p.free_pages[head + fresh];
            p.block_table_out[(int64_t)i * p.max_blocks + last] = dst;
        }
        p.ctx_lens_out[i] = r < 0 ? 0 : p.ctx_lens[r];
        p.copy_src[i] = src;
        p.copy_dst[i] = dst;
    }
    // ---- the counts
    const int me = cta * kWarps + warp, nwarps = ncta * kWarps;
    for (int task = me; task < B * chunks; task += nwarps) {
        const int r = task / chunks, c0 = (task - r * chunks) * kFpStep, n = s_children[r], end = s_held[r] & INT32_MAX;
        if (n == 1 || c0 >= end) continue;
        const int32_t* row = p.block_table + (int64_t)r * p.max_blocks;
        const int last = s_held[r] < 0 ? end - 1 : -1;  // the column of a partly filled page
        int page[kFpSpan];
#pragma unroll
        for (int j = 0; j < kFpSpan; ++j) page[j] = c0 + 32 * j + lane < end ? __ldg(row + c0 + 32 * j + lane) : -1;
#pragma unroll
        for (int j = 0; j < kFpSpan; ++j) {
            const int more = c0 + 32 * j + lane == last ? min(n, 1) - 1 : n - 1;
            if (page[j] >= p.num_blocks) set_error(p.err, PKA_DEVERR_BLOCK_ID);
            else if (page[j] >= 0 && more != 0) atomicAdd(&p.share_counts[page[j]], more);
        }
    }
    if (ending == 0) {
        cluster_barrier();  // (the list's head has been read)
        if (cta == 0 && tid == 0) *p.free_head_out = head + taken;
        return;
    }
    cluster_barrier();
    // ---- ending rows in stretches of `span` columns
    const int parts = min(max(1, kFpTasks / ending), chunks), span = (chunks + parts - 1) / parts * kFpStep;
    const int tasks = ending * parts;
    // the first place of each page that nobody holds
    for (int task = me; task < tasks; task += nwarps) {
        const int d = task / parts, r = s_dead[d], end = s_held[r] & INT32_MAX;
        const int from = (task - d * parts) * span;
        bool some = false;
        for (int c0 = from; c0 < min(end, from + span); c0 += kFpStep) {
            int page[kFpSpan], count[kFpSpan];
            load_span(page, p.block_table + (int64_t)r * p.max_blocks, c0, end, p.num_blocks);
            load_counts(count, page, p.share_counts);
#pragma unroll
            for (int j = 0; j < kFpSpan; ++j) {
                if (count[j] >= 0) continue;
                atomicMin(&p.share_counts[page[j]], INT32_MIN + r * p.max_blocks + c0 + 32 * j + lane);
                some = true;
            }
        }
        // (the same warp counts the stretch below, where there is something to count)
        if (__any_sync(0xffffffffu, some) && lane == 0) s_freed[task] = 1;
    }
    cluster_barrier();
    for (int task = me; task < tasks; task += nwarps) {
        if (s_freed[task] == 0) continue;
        const int d = task / parts, r = s_dead[d], end = s_held[r] & INT32_MAX;
        const int from = (task - d * parts) * span;
        int freed = 0;
        for (int c0 = from; c0 < min(end, from + span); c0 += kFpStep) {
            int page[kFpSpan], count[kFpSpan];
            load_span(page, p.block_table + (int64_t)r * p.max_blocks, c0, end, p.num_blocks);
            load_counts(count, page, p.share_counts);
#pragma unroll
            for (int j = 0; j < kFpSpan; ++j)
                freed += count[j] == INT32_MIN + r * p.max_blocks + c0 + 32 * j + lane;
        }
        freed = __reduce_add_sync(0xffffffffu, freed);  // (every lane has read the flag)
        if (lane < ncta) store_cluster(reinterpret_cast<uint32_t*>(&s_freed[task]), lane, (uint32_t)freed);
    }
    cluster_barrier();
    // ---- their places in the list
    int total = 0;
    for (int k0 = 0; k0 < tasks; k0 += kThreads) {
        const int k = k0 + tid, n = k < tasks ? s_freed[k] : 0;
        int sum;
        const int before = block_scan<kThreads>(n, s_scan, &sum);
        if (k < tasks) s_freed[k] = n ? total + before : -1;
        total += sum;
    }
    __syncthreads();
    const int start = head + taken - total;
    for (int task = me; task < tasks; task += nwarps) {
        int at = s_freed[task];
        if (at < 0) continue;
        at += start;
        const int d = task / parts, r = s_dead[d], end = s_held[r] & INT32_MAX;
        const int from = (task - d * parts) * span;
        for (int c0 = from; c0 < min(end, from + span); c0 += kFpStep) {
            int page[kFpSpan], count[kFpSpan];
            load_span(page, p.block_table + (int64_t)r * p.max_blocks, c0, end, p.num_blocks);
            load_counts(count, page, p.share_counts);
#pragma unroll
            for (int j = 0; j < kFpSpan; ++j) {
                const bool mine = count[j] == INT32_MIN + r * p.max_blocks + c0 + 32 * j + lane;
                const uint32_t all = __ballot_sync(0xffffffffu, mine);
                if (mine) {
                    const int to = at + __popc(all & ((1u << lane) - 1));
                    if (to >= 0) p.free_pages[to] = page[j];
                    p.share_counts[page[j]] = 0;
                }
                at += __popc(all);
            }
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

template <int kThreads>
static cudaError_t go(const ForkPagesParams& p, int cluster, int clusters, cudaStream_t stream) {
    auto kern = fork_pages_kernel<kThreads>;
    const size_t smem = sizeof(int32_t) * (4 * (size_t)p.num_rows + p.num_rows_out + kFpTasks);
    if (smem > 47 * 1024) {  // past what every kernel may use; the most that any call takes
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)sizeof(int32_t) * (5 * kMaxRequests + kFpTasks));
        if (e != cudaSuccess) return e;
    }
    if (cluster > 8) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    return launch_cluster(kern, dim3(cluster * clusters), dim3(kThreads), smem, cluster, stream, p);
}

cudaError_t launch_fork_pages(const ForkPagesParams& p, int num_sms, cudaStream_t stream) {
    // By what the table may hold: one small CTA of 8 warps, one cluster of 512, or further ones for the copies
    // (8 rows of 3 pages 7.6 us with the first, 8.5 with the second; 32 rows 12.5 and 9.3, 376 rows 97 and 10.7).
    const int rows = std::max(p.num_rows, p.num_rows_out);
    const int64_t entries = (int64_t)rows * p.max_blocks;
    if (rows <= 16 && entries <= 4096) return go<kFpFew>(p, 1, 1, stream);
    const int64_t more = (int64_t)p.num_rows_out * p.max_blocks / (kFpCluster * kFpMany * kFpSpan);
    return go<kFpMany>(p, kFpCluster, 1 + (int)std::min<int64_t>(more, num_sms / kFpCluster - 1), stream);
}

cudaError_t launch_copy_pages(CopyPagesParams p, int num_sms, cudaStream_t stream) {
    p.pieces = (int)((p.page_bytes + kCpPiece - 1) / kCpPiece);
    const int64_t total = (int64_t)p.num_pairs * p.num_caches * p.pieces;
    const int64_t n = std::min<int64_t>(total, (int64_t)num_sms * 8);
    return launch_dependent(copy_pages_kernel, dim3((unsigned)n), dim3(kCpThreads), 0, stream, p);
}

}  // namespace pka
