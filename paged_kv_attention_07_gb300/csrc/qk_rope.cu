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
// A head lies on d / 8 neighbouring lanes, each with four pairs: eight
// neighbouring elements where pairs are neighbours, four and their partners
// where pairs are half the rotated part apart, so a pair never crosses lanes, a
// lane needs four cosines and four sines, and the mean is a shuffle sum inside
// the head. A warp takes a unit of kQrRows rows of heads of one token and one
// kind (query, key or value), all their loads issued before any is used;
// neighbouring warps take neighbouring units. Bound by issue as much as by
// HBM: one kind per unit keeps the choices out of the rows, weights and
// rotation are multiplied together once per unit, values are only copied (8192
// tokens of 32 + 8 + 8 heads of 128: 39.4 us, 6.07 TB/s of the 239 MB; 64 tokens
// 2.5 us). 32 resident warps per SM: 28 take 40.2 us, 20 with all the registers
// they ask for 45.6 us.
#include "common.cuh"
#include "params.cuh"

namespace pka {

namespace {

constexpr int kQrRows = 4;  // rows of heads in a unit: a lane's 16-byte pieces in flight
constexpr int kQrWarps = 4;

PKA_DEVICE void unpack8(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}

// x / s, as far as E4M3 codes need it: x times the reciprocal, mended by the
// remainder over s, which a fused multiply-add leaves exact (Newton's step for a
// quotient; Markstein, IBM J. Res. Dev. 34, 1990). The result is within 2^-24 of an
// ulp of the exact quotient before its own rounding, so it is not the float32
// quotient only where that is as near to the middle of two floats. With x a
// bf16 number no such quotient lies next to the border of two codes unless all
// mantissa bits of s are set (that one takes two reciprocals), so values
// get the codes that a division gives (each code of every pattern was compared).
// Quotients past the codes, infinities and zeros need no mending. 5003 tokens of 4 kv
// heads: 21.2 us, 23.7 us with divisions.
PKA_DEVICE float quotient(float x, const QuotientBy& u) {
    const float y = x * u.pre, q = y * u.start;
    const float mended = __fmaf_rn(__fmaf_rn(-q, u.s, y), u.mend, q);
    return fabsf(fabsf(q) - 256.f) < 256.f ? mended : q;
}
PKA_DEVICE uint32_t codes4(const float* x, const QuotientBy& u) {
    return e4m3x4(quotient(x[0], u), quotient(x[1], u), quotient(x[2], u), quotient(x[3], u));
}

// A lane's eight elements of a head: x[0..3] at `first`, x[4..7] at `second`
// (first + 4 in the interleaved form: one piece).
template <bool kInterleaved>
PKA_DEVICE uint4 load_piece(const __nv_bfloat16* head, int first, int second) {
    if (kInterleaved) return *reinterpret_cast<const uint4*>(head + first);
    const uint2 a = *reinterpret_cast<const uint2*>(head + first), b = *reinterpret_cast<const uint2*>(head + second);
    return make_uint4(a.x, a.y, b.x, b.y);
}
template <bool kInterleaved>
PKA_DEVICE void store_piece(__nv_bfloat16* head, int first, int second, const uint4& v) {
    if (kInterleaved) {
        *reinterpret_cast<uint4*>(head + first) = v;
    } else {
        *reinterpret_cast<uint2*>(head + first) = make_uint2(v.x, v.y);
        *reinterpret_cast<uint2*>(head + second) = make_uint2(v.z, v.w);
    }
}

template <int kLanes, bool kFp8, bool kInterleaved>
__global__ void __launch_bounds__(kQrWarps * 32, 8) qk_rope_kernel(QkRopeParams p) {
    grid_dep_launch();
    grid_dep_wait();
    constexpr int kPerWarp = 32 / kLanes;       // heads side by side in a warp
    constexpr int kHeads = kPerWarp * kQrRows;  // heads of a unit
    const int lane = threadIdx.x & 31, sub = lane / kLanes, l = lane % kLanes;
    const int d = p.head_dim;
    const bool mine = l < (d >> 3);
    const int half = p.rotary >> 1;
    // this lane's elements, and its first pair
    const bool turned = mine && (kInterleaved ? l * 8 < p.rotary : l * 4 < half);
    const int first = kInterleaved ? l * 8 : (turned ? l * 4 : half + l * 4);  // (behind: rotary + (4 l - half))
    const int second = kInterleaved ? first + 4 : (turned ? half + l * 4 : first + ((d - p.rotary) >> 1));
    const float inv_d = 1.f / (float)d;
    const int gq = (p.Hq + kHeads - 1) / kHeads, gk = (p.Hkv + kHeads - 1) / kHeads, groups = gq + 2 * gk;
    const int64_t units = p.num_tokens * groups;
    for (int64_t u = (int64_t)blockIdx.x * kQrWarps + (threadIdx.x >> 5); u < units;
         u += (int64_t)gridDim.x * kQrWarps) {
        const int64_t t = units <= INT32_MAX ? (int64_t)((uint32_t)u / (uint32_t)groups) : u / groups;
        const int g = (int)(u - t * groups);
        const int kind = g < gq ? 0 : g < gq + gk ? 1 : 2;  // q, k, v
        const int n = kind == 0 ? p.Hq : p.Hkv;
        const int h0 = (kind == 0 ? g : kind == 1 ? g - gq : g - gq - gk) * kHeads + sub;
        const int pos = __ldg(p.positions + t);
        const int64_t slot = __ldg(p.slots + t);
        const __nv_bfloat16* src = (kind == 0   ? p.q + t * p.q_stride
                                    : kind == 1 ? p.k + t * p.k_stride
                                                : p.v + t * p.v_stride) + h0 * d;
        uint4 raw[kQrRows];
#pragma unroll
        for (int i = 0; i < kQrRows; ++i) {
            raw[i] = make_uint4(0, 0, 0, 0);
            if (mine && h0 + i * kPerWarp < n) raw[i] = load_piece<kInterleaved>(src + i * kPerWarp * d, first, second);
        }
        const bool past = p.rotary > 0 && pos >= p.max_position;
        if (past && lane == 0 && g == 0) set_error(p.err, PKA_DEVERR_INDEX);
        if (pos < 0 || past) continue;  // a row behind the last sequence, or past the rotation table
        if (slot >= p.num_slots && lane == 0 && g == 0) set_error(p.err, PKA_DEVERR_SLOT);
        // what the four pairs are multiplied by: a -> a ac - b bs, b -> b bc + a as
        float ac[4], as[4], bc[4], bs[4];
        if (kind < 2) {
            float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
            if (turned) {
                const float* row = p.cos_sin + (int64_t)pos * p.rotary + l * 4;
                cs = __ldg(reinterpret_cast<const float4*>(row));
                sn = __ldg(reinterpret_cast<const float4*>(row + half));
            }
            ac[0] = cs.x, ac[1] = cs.y, ac[2] = cs.z, ac[3] = cs.w;
            as[0] = sn.x, as[1] = sn.y, as[2] = sn.z, as[3] = sn.w;
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 1.f;
            if (p.q_weight && mine)
                unpack8(load_piece<kInterleaved>(kind == 0 ? p.q_weight : p.k_weight, first, second), w);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float wa = w[kInterleaved ? 2 * j : j], wb = w[kInterleaved ? 2 * j + 1 : 4 + j];
                bc[j] = wb * ac[j];
                bs[j] = wb * as[j];
                ac[j] *= wa;
                as[j] *= wa;
            }
        }
        const bool stored = kind > 0 && slot >= 0 && slot < p.num_slots;
        int64_t cache0 = 0;
        if (stored) {
            const int64_t blk = p.num_slots <= INT32_MAX ? (int64_t)((uint32_t)slot / (uint32_t)p.block_size)
                                                         : slot / p.block_size;
            cache0 = ((blk * p.Hkv + h0) * p.block_size + (slot - blk * p.block_size)) * d;
        }
        __nv_bfloat16* copy = kind == 0 ? p.q_out : kind == 1 ? p.k_out : p.v_out;
        if (copy) copy += (t * n + h0) * d;
        void* cache = kind == 1 ? p.k_cache : p.v_cache;
        const QuotientBy unit = kind == 1 ? p.k_unit : p.v_unit;
#pragma unroll
        for (int i = 0; i < kQrRows; ++i) {
            uint4 out = raw[i];
            float x[8];
            if (kind < 2 || kFp8) unpack8(raw[i], x);
            if (kind < 2) {
                float r = 1.f;
                if (p.q_weight) {  // every lane takes part in the shuffles; rows past the last head hold zeros
                    float ss = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) ss += x[j] * x[j];
#pragma unroll
                    for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    r = rsqrtf(ss * inv_d + p.eps);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float& a = x[kInterleaved ? 2 * j : j];
                    float& b = x[kInterleaved ? 2 * j + 1 : 4 + j];
                    const float xa = a, xb = b;
                    // (elements that are not turned have no part in each other, infinities included)
                    a = turned ? (xa * ac[j] - xb * bs[j]) * r : xa * ac[j] * r;
                    b = turned ? (xb * bc[j] + xa * as[j]) * r : xb * bc[j] * r;
                }
                out = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                                 pack_bf16(x[6], x[7]));
            }
            if (!mine || h0 + i * kPerWarp >= n) continue;
            if (copy) store_piece<kInterleaved>(copy + i * kPerWarp * d, first, second, out);
            if (!stored) continue;
            const int64_t at = cache0 + (int64_t)(i * kPerWarp) * p.block_size * d;
            if (kFp8) {
                uint8_t* dst = static_cast<uint8_t*>(cache) + at;
                const uint32_t lo = codes4(x, unit), hi = codes4(x + 4, unit);
                if (kInterleaved) {
                    *reinterpret_cast<uint2*>(dst + first) = make_uint2(lo, hi);
                } else {
                    *reinterpret_cast<uint32_t*>(dst + first) = lo;
                    *reinterpret_cast<uint32_t*>(dst + second) = hi;
                }
            } else {
                store_piece<kInterleaved>(static_cast<__nv_bfloat16*>(cache) + at, first, second, out);
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
    const int groups = (p.Hq + heads - 1) / heads + 2 * ((p.Hkv + heads - 1) / heads);
    const int64_t units = p.num_tokens * groups;
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
