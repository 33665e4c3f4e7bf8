// qk_rope.cu -- norms of the new tokens' query and key heads, the position
// rotation, and the cache write, in one pass over the projections' output.
//
//   y = x / sqrt(mean(x^2) + eps) * w           (per head; left out without weights)
//   (a, b) -> (a c - b s, b c + a s)            for the rotated pairs, c / s of the token's position
//   q -> q_out;  k, v -> their cache slots, and k_out / v_out when wanted
//
// Everything between the load and the store is float32: one rounding, to bf16
// or to the 8-bit cache's E4M3 code. HBM-bound: reads T (Hq + 2 Hkv) d bf16 and
// the rotation rows, writes q, k and v once (twice with k_out / v_out).
//
// A head is d / 8 pieces of 16 bytes on kLanes neighbouring lanes, so the mean
// is a shuffle sum inside the head and the partner of a half-split pair is a
// fixed lane distance away. A warp takes kQrRows rows of heads of ONE token:
// all their loads are issued before any is used, and the token's cosines and
// sines are read once per warp.
#include "common.cuh"
#include "params.cuh"

namespace pka {

namespace {

constexpr int kQrRows = 4;  // head rows (16-byte pieces) per lane in flight
constexpr int kQrWarps = 8;

PKA_DEVICE void unpack8(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}

PKA_DEVICE uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

template <int kLanes, bool kFp8, bool kInterleaved>
__global__ void __launch_bounds__(kQrWarps * 32) qk_rope_kernel(QkRopeParams p) {
    grid_dep_launch();
    grid_dep_wait();
    constexpr int kPerWarp = 32 / kLanes;           // heads side by side in a warp
    constexpr int kHeads = kPerWarp * kQrRows;      // heads of a warp's unit
    const int lane = threadIdx.x & 31, sub = lane / kLanes, l = lane % kLanes;
    const int pieces = p.head_dim >> 3;
    const bool mine = l < pieces;
    const int heads = p.Hq + 2 * p.Hkv;
    const int groups = (heads + kHeads - 1) / kHeads;
    const int half = p.rotary >> 1, e0 = l * 8;
    // half-split: this piece's pairs sit `half` elements (half / 8 lanes) away
    const bool turned = mine && e0 < p.rotary;
    const bool second = !kInterleaved && e0 >= half;
    const int partner = turned && !kInterleaved ? (second ? lane - (half >> 3) : lane + (half >> 3)) : lane;
    const int a0 = kInterleaved ? e0 >> 1 : (second ? e0 - half : e0);
    const int64_t units = p.num_tokens * groups;
    for (int64_t u = (int64_t)blockIdx.x * kQrWarps + (threadIdx.x >> 5); u < units;
         u += (int64_t)gridDim.x * kQrWarps) {
        const int64_t t = u / groups;
        const int h0 = (int)(u - t * groups) * kHeads + sub;
        const int pos = __ldg(p.positions + t);
        const int64_t slot = __ldg(p.slots + t);
        uint4 raw[kQrRows];
#pragma unroll
        for (int i = 0; i < kQrRows; ++i) {
            const int h = h0 + i * kPerWarp;
            raw[i] = make_uint4(0, 0, 0, 0);
            if (!mine || h >= heads) continue;
            const __nv_bfloat16* src = h < p.Hq ? p.q + t * p.q_stride + (int64_t)h * p.head_dim
                                       : h < p.Hq + p.Hkv
                                           ? p.k + t * p.k_stride + (int64_t)(h - p.Hq) * p.head_dim
                                           : p.v + t * p.v_stride + (int64_t)(h - p.Hq - p.Hkv) * p.head_dim;
            raw[i] = *reinterpret_cast<const uint4*>(src + e0);
        }
        if (pos < 0) continue;  // a row behind the last sequence
        if (p.rotary > 0 && pos >= p.max_position) {
            if (lane == 0) set_error(p.err, PKA_DEVERR_INDEX);
            continue;
        }
        const bool stored = slot >= 0 && slot < p.num_slots;
        if (slot >= p.num_slots && lane == 0) set_error(p.err, PKA_DEVERR_SLOT);
        float cs[8], sn[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            cs[j] = 1.f;
            sn[j] = 0.f;
        }
        if (turned) {
            const float4* c = reinterpret_cast<const float4*>(p.cos_sin + (int64_t)pos * p.rotary + a0);
            const float4* s = reinterpret_cast<const float4*>(p.cos_sin + (int64_t)pos * p.rotary + half + a0);
#pragma unroll
            for (int j = 0; j < (kInterleaved ? 1 : 2); ++j) {
                const float4 x = __ldg(c + j), y = __ldg(s + j);
                cs[4 * j] = x.x, cs[4 * j + 1] = x.y, cs[4 * j + 2] = x.z, cs[4 * j + 3] = x.w;
                sn[4 * j] = y.x, sn[4 * j + 1] = y.y, sn[4 * j + 2] = y.z, sn[4 * j + 3] = y.w;
            }
        }
        const int64_t blk = stored ? slot / p.block_size : 0;
        const int off = stored ? (int)(slot - blk * p.block_size) : 0;
#pragma unroll
        for (int i = 0; i < kQrRows; ++i) {
            const int h = h0 + i * kPerWarp;
            const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
            float x[8];
            unpack8(raw[i], x);
            // every lane takes part in the shuffles; rows past the last head hold zeros
            const __nv_bfloat16* weight = is_q ? p.q_weight : p.k_weight;
            if (p.q_weight) {
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) ss += x[j] * x[j];
#pragma unroll
                for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float r = 1.f / sqrtf(ss / (float)p.head_dim + p.eps);
                if (!is_v && mine) {
                    float w[8];
                    unpack8(__ldg(reinterpret_cast<const uint4*>(weight + e0)), w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = x[j] * r * w[j];
                }
            }
            if (p.rotary > 0) {
                float y[8];
                if (kInterleaved) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        y[2 * j] = x[2 * j] * cs[j] - x[2 * j + 1] * sn[j];
                        y[2 * j + 1] = x[2 * j + 1] * cs[j] + x[2 * j] * sn[j];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float z = __shfl_sync(0xffffffffu, x[j], partner);
                        y[j] = second ? x[j] * cs[j] + z * sn[j] : x[j] * cs[j] - z * sn[j];
                    }
                }
                if (turned && !is_v) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = y[j];
                }
            }
            if (!mine || h >= heads) continue;
            if (is_q) {
                *reinterpret_cast<uint4*>(p.q_out + (t * p.Hq + h) * p.head_dim + e0) = pack8(x);
                continue;
            }
            const int hk = is_v ? h - p.Hq - p.Hkv : h - p.Hq;
            __nv_bfloat16* copy = is_v ? p.v_out : p.k_out;
            const uint4 b = is_v ? raw[i] : pack8(x);
            if (copy) *reinterpret_cast<uint4*>(copy + (t * p.Hkv + hk) * p.head_dim + e0) = b;
            if (!stored) continue;
            void* cache = is_v ? p.v_cache : p.k_cache;
            const int64_t at = ((blk * p.Hkv + hk) * p.block_size + off) * p.head_dim + e0;
            if (kFp8) {
                const float s = is_v ? p.v_scale : p.k_scale;
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + at) =
                    make_uint2(quantize4(x[0], x[1], x[2], x[3], s), quantize4(x[4], x[5], x[6], x[7], s));
            } else {
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(cache) + at) = b;
            }
        }
    }
}

template <int kLanes, bool kFp8, bool kInterleaved>
cudaError_t go(const QkRopeParams& p, int num_sms, cudaStream_t stream) {
    auto kern = qk_rope_kernel<kLanes, kFp8, kInterleaved>;
    static const int per_sm = [&] {
        int n = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kQrWarps * 32, 0) != cudaSuccess || n < 1) n = 1;
        return n;
    }();
    const int heads = 32 / kLanes * kQrRows;
    const int64_t units = p.num_tokens * ((p.Hq + 2 * p.Hkv + heads - 1) / heads);
    const int64_t blocks = std::min<int64_t>((units + kQrWarps - 1) / kQrWarps, (int64_t)num_sms * per_sm);
    return launch_dependent(kern, dim3((unsigned)blocks), dim3(kQrWarps * 32), 0, stream, p);
}

}  // namespace

cudaError_t launch_qk_rope(const QkRopeParams& p, bool fp8, int num_sms, cudaStream_t stream) {
    auto by_form = [&](auto lanes) {
        constexpr int L = decltype(lanes)::value;
        if (fp8) return p.interleaved ? go<L, true, true>(p, num_sms, stream) : go<L, true, false>(p, num_sms, stream);
        return p.interleaved ? go<L, false, true>(p, num_sms, stream) : go<L, false, false>(p, num_sms, stream);
    };
    if (p.head_dim <= 64) return by_form(std::integral_constant<int, 8>{});
    if (p.head_dim <= 128) return by_form(std::integral_constant<int, 16>{});
    return by_form(std::integral_constant<int, 32>{});
}

}  // namespace pka
