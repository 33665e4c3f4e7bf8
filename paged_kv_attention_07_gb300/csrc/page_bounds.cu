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
// token that goes to its last slot. A CTA looks at the slots of `chunk` tokens
// with one load per warp and takes the filled pages of its kv head: its 128
// threads together one after another, or, pages of up to 4 KB, each warp its
// own (256 decodes over an 8-bit cache, pages of 2 KB: 2.9 us, 3.9 us with all
// threads on each; 16384 tokens in pages of 4 KB: 7.1 us, 9.0 us). A page is
// read in 16-byte pieces, all of a thread's pieces in flight together, minima
// and maxima are packed 16-bit pairs (bf16 as it is, codes widened to f16,
// exact). Bound by latency (a slot, a page, the join) up to some thousand
// tokens, by HBM beyond: block_size x d elements read per filled (page, kv
// head), 2 d + 4 bytes written (16384 tokens in pages of 16 KB: 5.2 us, 3.3 TB/s).
#include "common.cuh"
#include "params.cuh"

namespace pka {

namespace {

constexpr int kPbThreads = 128;
constexpr int kPbWarps = kPbThreads / 32;
constexpr int kPbBatch = 8;  // 16-byte pieces per thread in flight
constexpr int64_t kPbWarpBytes = 32 * kPbBatch * 16;  // a page that one warp holds

// Packed pairs: bf16, or f16 of codes. NaN wins over any value.
template <bool kFp8>
PKA_DEVICE uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t r;
    if (kFp8) asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <bool kFp8>
PKA_DEVICE uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    if (kFp8) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
PKA_DEVICE __half2 h2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
PKA_DEVICE uint16_t two(float x, float y) { return (uint16_t)((uint8_t)(int8_t)(int)x | (uint8_t)(int8_t)(int)y << 8); }
// Codes of a pair: floor (ceil) of x times the power of two `unit`. The products are exact but where they are below
// float32's least number, far below the page's largest: rounded away from the keys they still give -1 and 1 there.
PKA_DEVICE uint16_t low_codes(float2 x, float unit) {
    return two(floorf(__fmul_rd(x.x, unit)), floorf(__fmul_rd(x.y, unit)));
}
PKA_DEVICE uint16_t high_codes(float2 x, float unit) {
    return two(ceilf(__fmul_ru(x.x, unit)), ceilf(__fmul_ru(x.y, unit)));
}
template <bool kFp8>
PKA_DEVICE float2 pair(uint32_t x) {
    return kFp8 ? __half22float2(h2(x)) : make_float2(bf16_lo(x), bf16_hi(x));
}

// kWarp: a page per warp instead of a page per CTA.
template <bool kFp8, bool kWarp>
__global__ void __launch_bounds__(kPbThreads) page_bounds_kernel(PageBoundsParams p) {
    constexpr int kLanes = kWarp ? 32 : kPbThreads;  // on a page
    constexpr int kVec = kFp8 ? 16 : 8;  // elements of a 16-byte piece
    constexpr int kWords = kVec / 2;     // and their packed pairs
    constexpr uint32_t kInf = kFp8 ? 0x7c007c00u : 0x7f807f80u, kMinusInf = kInf | 0x80008000u;
    __shared__ uint32_t s_lo[kWarp ? 1 : kPbWarps][64], s_hi[kWarp ? 1 : kPbWarps][64];  // head_dim / 2 pairs per warp
    __shared__ float s_amax[2];
    grid_dep_launch();
    grid_dep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = blockIdx.y;
    const int pieces = p.head_dim / kVec;  // of a key: a power of two, 4 to 16
    const int rows = kLanes / pieces;      // keys read side by side
    const int c = tid % kLanes % pieces, r0 = tid % kLanes / pieces;
    for (int64_t t0 = (int64_t)blockIdx.x * p.chunk; t0 < p.num_tokens; t0 += (int64_t)gridDim.x * p.chunk) {
        // the pages that this chunk fills: one token per lane, the same in every warp
        int64_t blk = -1;
        if (lane < p.chunk && t0 + lane < p.num_tokens) {
            const int64_t slot = __ldg(p.slots + t0 + lane);
            if (slot >= p.num_slots) {
                if (warp == 0 && g == 0) set_error(p.err, PKA_DEVERR_SLOT);
            } else if (slot >= 0) {
                const int64_t b = slot / p.block_size;
                if (slot - b * p.block_size == p.block_size - 1) blk = b;
            }
        }
        uint32_t todo = __ballot_sync(0xffffffffu, blk >= 0);
        for (int turn = 0; todo; todo &= todo - 1, ++turn) {
            const int64_t page = __shfl_sync(0xffffffffu, blk, __ffs(todo) - 1) * p.Hkv + g;
            if (kWarp && turn % kPbWarps != warp) continue;
            const uint8_t* src = static_cast<const uint8_t*>(p.k_cache) +
                                 (page * p.block_size * p.head_dim + c * kVec) * (kFp8 ? 1 : 2);
            const int64_t row = (int64_t)p.head_dim * (kFp8 ? 1 : 2);
            uint32_t lo[kWords], hi[kWords];
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                lo[i] = kInf;
                hi[i] = kMinusInf;
            }
            for (int r = r0; r < p.block_size; r += kPbBatch * rows) {
                uint4 v[kPbBatch];
#pragma unroll
                for (int j = 0; j < kPbBatch; ++j)
                    if (r + j * rows < p.block_size) v[j] = *reinterpret_cast<const uint4*>(src + (r + j * rows) * row);
#pragma unroll
                for (int j = 0; j < kPbBatch; ++j) {
                    if (r + j * rows >= p.block_size) continue;
                    const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (kFp8) {
                            const uint32_t a = e4m3x2_to_f16x2(w[i] & 0xffffu), b = e4m3x2_to_f16x2(w[i] >> 16);
                            lo[2 * i % kWords] = min2<kFp8>(lo[2 * i % kWords], a);
                            hi[2 * i % kWords] = max2<kFp8>(hi[2 * i % kWords], a);
                            lo[(2 * i + 1) % kWords] = min2<kFp8>(lo[(2 * i + 1) % kWords], b);
                            hi[(2 * i + 1) % kWords] = max2<kFp8>(hi[(2 * i + 1) % kWords], b);
                        } else {
                            lo[i] = min2<kFp8>(lo[i], w[i]);
                            hi[i] = max2<kFp8>(hi[i], w[i]);
                        }
                    }
                }
            }
            // ---- join: the warp's rows by shuffles, the warps in shared memory
            for (int o = pieces; o < 32; o <<= 1) {
#pragma unroll
                for (int i = 0; i < kWords; ++i) {
                    lo[i] = min2<kFp8>(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
                    hi[i] = max2<kFp8>(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
                }
            }
            if constexpr (kWarp) {  // the elements of piece c, in every lane that reads it
                float a = 0.f;
#pragma unroll
                for (int i = 0; i < kWords; ++i) {
                    const float2 l = pair<kFp8>(lo[i]), h = pair<kFp8>(hi[i]);
                    a = fmaxf(a, fmaxf(fmaxf(-l.x, h.x), fmaxf(-l.y, h.y)));
                    if (isnan(l.x) || isnan(l.y)) a = INFINITY;
                }
                for (int o = 1; o < pieces; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
                const bool none = a == INFINITY;
                const int e = none ? 0 : bound_exponent(a);
                const float unit = none ? 0.f : exp2i(-e);
                if (lane < pieces) {
                    uint16_t codes[2][kWords];
#pragma unroll
                    for (int i = 0; i < kWords; ++i) {
                        const float2 l = pair<kFp8>(lo[i]), h = pair<kFp8>(hi[i]);
                        codes[0][i] = none ? 0 : low_codes(l, unit);
                        codes[1][i] = none ? 0 : high_codes(h, unit);
                    }
                    uint2* dst = reinterpret_cast<uint2*>(p.bounds + page * 2 * p.head_dim + c * kVec);
#pragma unroll
                    for (int i = 0; i < kWords / 4; ++i) {
                        auto four = [&](const uint16_t* x) { return make_uint2(x[0] | x[1] << 16, x[2] | x[3] << 16); };
                        dst[i] = four(codes[0] + 4 * i);
                        dst[i + p.head_dim / 8] = four(codes[1] + 4 * i);
                    }
                    if (lane == 0) p.scales[page] = none ? INFINITY : exp2i(e);
                }
                continue;
            }
            __syncthreads();  // the last page's results have been read
            if (lane < pieces) {
#pragma unroll
                for (int i = 0; i < kWords; ++i) {
                    s_lo[warp][lane * kWords + i] = lo[i];
                    s_hi[warp][lane * kWords + i] = hi[i];
                }
            }
            __syncthreads();
            // ---- two elements per thread of the first two warps (head_dim <= 128)
            const int pairs = p.head_dim / 2;
            float2 l = make_float2(0.f, 0.f), h = l;
            if (tid < pairs) {
                uint32_t x = s_lo[0][tid], y = s_hi[0][tid];
#pragma unroll
                for (int w = 1; w < kPbWarps; ++w) {
                    x = min2<kFp8>(x, s_lo[w][tid]);
                    y = max2<kFp8>(y, s_hi[w][tid]);
                }
                l = pair<kFp8>(x);
                h = pair<kFp8>(y);
            }
            // the largest magnitude, an infinity where there is a NaN
            float a = fmaxf(fmaxf(-l.x, h.x), fmaxf(-l.y, h.y));
            if (isnan(l.x) || isnan(l.y)) a = INFINITY;
#pragma unroll
            for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
            if (lane == 0 && warp < 2) s_amax[warp] = a;
            __syncthreads();
            a = fmaxf(s_amax[0], s_amax[1]);
            const bool none = a == INFINITY;
            const int e = none ? 0 : bound_exponent(a);
            const float unit = none ? 0.f : exp2i(-e);
            if (tid < pairs) {
                uint16_t* code = reinterpret_cast<uint16_t*>(p.bounds + page * 2 * p.head_dim);
                code[tid] = none ? 0 : low_codes(l, unit);
                code[pairs + tid] = none ? 0 : high_codes(h, unit);
            }
            if (tid == 0) p.scales[page] = none ? INFINITY : exp2i(e);
        }
    }
}

}  // namespace

cudaError_t launch_page_bounds(PageBoundsParams p, bool fp8, int num_sms, cudaStream_t stream) {
    // a chunk of tokens may fill up to as many pages (decodes): small chunks
    // while the GPU has room for them, a warp's lanes at most
    p.chunk = 32;
    while (p.chunk > 4 && (p.num_tokens + p.chunk - 1) / p.chunk * p.Hkv < num_sms) p.chunk /= 2;
    const int64_t chunks = (p.num_tokens + p.chunk - 1) / p.chunk;
    const dim3 grid((unsigned)std::min<int64_t>(chunks, 1 << 20), (unsigned)p.Hkv);
    const bool small = (int64_t)p.block_size * p.head_dim * (fp8 ? 1 : 2) <= kPbWarpBytes;
    auto go = [&](auto kern) { return launch_dependent(kern, grid, dim3(kPbThreads), 0, stream, p); };
    if (small) return fp8 ? go(page_bounds_kernel<true, true>) : go(page_bounds_kernel<false, true>);
    return fp8 ? go(page_bounds_kernel<true, false>) : go(page_bounds_kernel<false, false>);
}

}  // namespace pka
