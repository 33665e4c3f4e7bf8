// page_bounds.cu -- element-wise bounds of a page's keys, as 8-bit codes.
//
// For a page whose last place was just written, kv head h, element i:
//   lo_i = min over the page's keys, hi_i = max;  a = max_i max(-lo_i, hi_i)
//   2^e  = the least power of two with a <= 127 * 2^e, and e >= kBoundMinExp
//   codes: floor(lo_i / 2^e), ceil(hi_i / 2^e);   scale: 2^e
// so that code * scale still bounds every key of the page. Minima and maxima do
// not depend on the order of the keys and a power of two divides exactly:
// the codes are the same bits for any split of the work. A page that holds a
// NaN or an infinity gets codes 0 and the scale +inf (it bounds nothing).
//
// The pages are found from the slot mapping alone: a page is filled by the
// token that goes to its last slot. HBM-bound: block_size x d elements read
// per filled (page, kv head), 2 d + 4 bytes written.
#include "common.cuh"
#include "params.cuh"

namespace pka {

namespace {

constexpr int kPbThreads = 128;
constexpr int kPbTokens = 8;  // tokens whose slots one CTA looks at

template <bool kFp8>
__global__ void __launch_bounds__(kPbThreads) page_bounds_kernel(PageBoundsParams p) {
    constexpr int kVec = kFp8 ? 16 : 8;          // elements of a 16-byte piece
    __shared__ float s_lo[kPbThreads * kVec], s_hi[kPbThreads * kVec];
    __shared__ uint32_t s_bad;
    grid_dep_launch();
    grid_dep_wait();
    const int tid = threadIdx.x;
    const int g = blockIdx.y;
    const int pieces = p.head_dim / kVec;        // 16-byte pieces of a key: a power of two, at most 16
    const int rows = kPbThreads / pieces;        // keys read side by side
    const int c = tid % pieces, r0 = tid / pieces;
    for (int64_t t0 = (int64_t)blockIdx.x * kPbTokens; t0 < p.num_tokens; t0 += (int64_t)gridDim.x * kPbTokens) {
        for (int64_t t = t0; t < t0 + kPbTokens && t < p.num_tokens; ++t) {
            const int64_t slot = __ldg(p.slots + t);
            if (slot < 0) continue;
            if (slot >= p.num_slots) {
                if (tid == 0 && g == 0) set_error(p.err, PKA_DEVERR_SLOT);
                continue;
            }
            const int64_t blk = slot / p.block_size;
            if (slot - blk * p.block_size != p.block_size - 1) continue;  // the same for the whole CTA
            const int64_t page = blk * p.Hkv + g;
            float lo[kVec], hi[kVec];
            bool bad = false;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                lo[i] = INFINITY;
                hi[i] = -INFINITY;
            }
            for (int r = r0; r < p.block_size; r += rows) {
                const uint4 v = *reinterpret_cast<const uint4*>(
                    static_cast<const uint8_t*>(p.k_cache) +
                    ((page * p.block_size + r) * p.head_dim + c * kVec) * (kFp8 ? 1 : 2));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                float x[kVec];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (kFp8) {
                        const float2 a = __half22float2(h2(e4m3x2_to_f16x2(w[i] & 0xffffu)));
                        const float2 b = __half22float2(h2(e4m3x2_to_f16x2(w[i] >> 16)));
                        x[4 * i % kVec] = a.x, x[(4 * i + 1) % kVec] = a.y;
                        x[(4 * i + 2) % kVec] = b.x, x[(4 * i + 3) % kVec] = b.y;
                    } else {
                        x[2 * i] = bf16_lo(w[i]);
                        x[2 * i + 1] = bf16_hi(w[i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    bad |= !(fabsf(x[i]) <= 3.4e38f);
                    lo[i] = fminf(lo[i], x[i]);
                    hi[i] = fmaxf(hi[i], x[i]);
                }
            }
            __syncthreads();  // the last page's results have been read
            if (tid == 0) s_bad = 0;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                s_lo[r0 * p.head_dim + c * kVec + i] = lo[i];
                s_hi[r0 * p.head_dim + c * kVec + i] = hi[i];
            }
            __syncthreads();
            if (bad) s_bad = 1;
            // element tid (head_dim <= kPbThreads): join the rows, then the largest magnitude
            float l = 0.f, h = 0.f;
            if (tid < p.head_dim) {
                l = s_lo[tid], h = s_hi[tid];
                const int n = min(rows, p.block_size);
                for (int r = 1; r < n; ++r) {
                    l = fminf(l, s_lo[r * p.head_dim + tid]);
                    h = fmaxf(h, s_hi[r * p.head_dim + tid]);
                }
            }
            __shared__ float s_amax[kPbThreads / 32];
            float a = fmaxf(-l, h);
#pragma unroll
            for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
            if ((tid & 31) == 0) s_amax[tid >> 5] = a;
            __syncthreads();
            a = 0.f;
#pragma unroll
            for (int i = 0; i < kPbThreads / 32; ++i) a = fmaxf(a, s_amax[i]);
            const bool nan = s_bad != 0;
            const int e = nan ? 0 : bound_exponent(a);
            const float unit = exp2i(-e);
            if (tid < p.head_dim) {
                int8_t* code = p.bounds + page * 2 * p.head_dim;
                code[tid] = nan ? 0 : (int8_t)(int)floorf(l * unit);
                code[p.head_dim + tid] = nan ? 0 : (int8_t)(int)ceilf(h * unit);
            }
            if (tid == 0) p.scales[page] = nan ? INFINITY : exp2i(e);
        }
    }
}

}  // namespace

cudaError_t launch_page_bounds(const PageBoundsParams& p, bool fp8, cudaStream_t stream) {
    const int64_t chunks = (p.num_tokens + kPbTokens - 1) / kPbTokens;
    const dim3 grid((unsigned)std::min<int64_t>(chunks, 1 << 20), (unsigned)p.Hkv);
    return fp8 ? launch_dependent(page_bounds_kernel<true>, grid, dim3(kPbThreads), 0, stream, p)
               : launch_dependent(page_bounds_kernel<false>, grid, dim3(kPbThreads), 0, stream, p);
}

}  // namespace pka
