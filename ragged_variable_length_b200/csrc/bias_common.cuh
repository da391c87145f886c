// Shared parts of the attention kernels with a learned relative position bias.
//
// For sequence b (query rows cu_q[b] .. , key rows cu_k[b] ..), query head h
// and key / value head z = h / (H / Hkv), with integer positions p of the
// tokens and buckets of the clamped relative distance:
//
//   s[i, j] = scale q_i . k_j + table[bucket(p_j - p_i), h]
//   bucket(d) = buckets[clamp(d, -D, D) + D]
//
// Scores are formed in base e, one fused multiply-add each, in every kernel: so
// far from 0, where fp32 no longer tells them from their bias, all kernels hold
// the same score.  exp(s - m) is one more multiply-add and ex2.approx,
// 2^(s log2 e - m log2 e), as long as m is near 0; far from it the rounding of
// m log2 e alone would move the exponent by more than the sum can bear (328 for a
// bias of -1e10), and the difference s - m, which is exact, is formed first.
#pragma once

#include "common.cuh"
#include "mma_common.cuh"

namespace ragged {
namespace bias {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxBuckets = 64;
constexpr int kMaxDistance = 1024;
constexpr int kQTile = 128;   // query rows per tile (also the grain of the table gradient's partial sums)

// One attention problem, as the kernels see it.
struct Problem {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    int64_t q_tok, q_head, kv_tok, kv_head;   // strides in elements
    const int32_t* cu_q;
    const int32_t* cu_k;
    const int32_t* pos_q;                     // or NULL: i + (Lk - Lq)
    const int32_t* pos_k;                     // or NULL: j
    const uint16_t* table;                    // [num_buckets, H]
    const int32_t* buckets;                   // [2 D + 1]
    float* lse;                               // [H, lse_stride]
    int64_t lse_stride;
    int B, max_q, max_k, H, Hkv, group;
    int num_buckets, D;
    float scale, scale_log2;
};

// Row ranges of sequence b; false when it must be skipped (and flagged).
struct Seq {
    int q_start, q_len, k_start, k_len;
};
__device__ __forceinline__ bool read_pair(const Problem& p, int b, Seq& s) {
    bool ok = read_sequence(p.cu_q, b, p.max_q, s.q_start, s.q_len);
    ok &= read_sequence(p.cu_k, b, p.max_k, s.k_start, s.k_len);
    if (ok && static_cast<int64_t>(s.q_start) + s.q_len > p.lse_stride) {   // rows that lse, and the scratch of its size, do not hold
        raise_status(RAGGED_DEV_BAD_SEQLENS);
        ok = false;
    }
    return ok;
}

// Whether the sequence's keys lie in rows of `held` elements.
__device__ __forceinline__ bool keys_held(const Seq& s, int64_t held) {
    if (static_cast<int64_t>(s.k_start) + s.k_len <= held) return true;
    raise_status(RAGGED_DEV_BAD_SEQLENS);
    return false;
}

template <typename T>
__device__ __forceinline__ float to_float(uint16_t x);
template <>
__device__ __forceinline__ float to_float<__half>(uint16_t x) {
    return __half2float(__ushort_as_half(x));
}
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(uint16_t x) {
    return __bfloat162float(__ushort_as_bfloat16(x));
}
template <typename T>
__device__ __forceinline__ uint16_t from_float(float x);
template <>
__device__ __forceinline__ uint16_t from_float<__half>(float x) {
    return __half_as_ushort(__float2half_rn(x));
}
template <>
__device__ __forceinline__ uint16_t from_float<__nv_bfloat16>(float x) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// Bucket of a relative distance, or -1 (and a flag) for a map entry outside
// the table; such a pair gets no bias and passes no gradient to the table.
__device__ __forceinline__ int bucket_of(const Problem& p, int delta) {
    const int d = max(-p.D, min(p.D, delta));
    const int b = __ldg(p.buckets + d + p.D);
    if (static_cast<unsigned>(b) >= static_cast<unsigned>(p.num_buckets)) {
        raise_status(RAGGED_DEV_BAD_BUCKETS);
        return -1;
    }
    return b;
}
// Difference of two positions (wraps instead of overflowing).
__device__ __forceinline__ int pos_diff(int a, int b) {
    return static_cast<int>(static_cast<unsigned>(a) - static_cast<unsigned>(b));
}
__device__ __forceinline__ int query_pos(const Problem& p, const Seq& s, int i) {
    return p.pos_q != nullptr ? __ldg(p.pos_q + s.q_start + i) : i + s.k_len - s.q_len;
}
__device__ __forceinline__ int key_pos(const Problem& p, const Seq& s, int j) {
    return p.pos_k != nullptr ? __ldg(p.pos_k + s.k_start + j) : j;
}

// log-sum-exp in base 2 for a gradient or weight pass: a row without any
// finite score (-inf) contributes nothing, so its reference is +inf.
__device__ __forceinline__ float lse_log2(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2e; }

// A row whose reference is beyond kFar is far: there the fp32 log-sum-exp is
// off by 2^-15 and more, from some 2^28 on it is the largest score and nothing of
// the sum.  The gradient and weight passes then form the logarithm of the row's
// sum again (row_log_sum).  Its largest score follows: lse was that score plus
// the logarithm, rounded, so lse less the logarithm, rounded, is the score.  No
// probability exceeds the largest score's: a score of another product that came
// out a step above it counts as it.
constexpr float kFar = 512.f;
__device__ __forceinline__ bool is_far(float x) { return fabsf(x) > kFar && fabsf(x) < INFINITY; }

// log sum_j exp(s[i, j] - max_j s[i, j]) of query row i and head h, by the lanes
// of a warp.  Plain products from global memory: tables with mask constants on
// all keys of a row are rare, and all else skips this.  Eight lanes read a key,
// each eight of its elements; of 32 keys each lane then gets one sum.
template <typename T>
__device__ __forceinline__ float row_log_sum(const Problem& p, const Seq& s, int i, int h) {
    const int lane = threadIdx.x & 31, r = lane >> 3, c = lane & 7;
    const uint16_t* keys = p.k + s.k_start * p.kv_tok + (h / p.group) * p.kv_head + c * 8;
    float q[8];
    auto floats = [](const uint4& w, float (&f)[8]) {
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[2 * e] = to_float<T>(static_cast<uint16_t>(ws[e]));
            f[2 * e + 1] = to_float<T>(static_cast<uint16_t>(ws[e] >> 16));
        }
    };
    floats(__ldg(reinterpret_cast<const uint4*>(p.q + static_cast<int64_t>(s.q_start + i) * p.q_tok + h * p.q_head) + c), q);
    const int pos = query_pos(p, s, i);
    float m = -INFINITY, l = 0.f;
#pragma unroll 1
    for (int j0 = 0; j0 < s.k_len; j0 += 32) {
        float sum[8];   // this lane's part of keys j0 + r, + 4, ...
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int j = min(j0 + 4 * u + r, s.k_len - 1);
            float k[8];
            floats(__ldg(reinterpret_cast<const uint4*>(keys + static_cast<int64_t>(j) * p.kv_tok)), k);
            sum[u] = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[u] = fmaf(q[e], k[e], sum[u]);
        }
#pragma unroll
        for (int n = 4; n > 0; n >>= 1) {   // each lane keeps half of its keys and hands over the other
            const bool upper = (c & n) != 0;
#pragma unroll
            for (int u = 0; u < n; ++u)
                sum[u] = (upper ? sum[u + n] : sum[u]) + __shfl_xor_sync(0xffffffffu, upper ? sum[u] : sum[u + n], n);
        }
        const int j = j0 + 4 * c + r;
        if (j >= s.k_len) continue;
        const int id = bucket_of(p, pos_diff(key_pos(p, s, j), pos));
        const float x = fmaf(sum[0], p.scale, id < 0 ? 0.f : to_float<T>(__ldg(p.table + static_cast<int64_t>(id) * p.H + h)));
        if (x == -INFINITY) continue;
        if (x > m) {
            l = fmaf(l, mma_attn::fast_exp2((m - x) * kLog2e), 1.f);
            m = x;
        } else {
            l += mma_attn::fast_exp2((x - m) * kLog2e);
        }
    }
    __syncwarp();
    float top = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    l = m == -INFINITY ? 0.f : l * mma_attn::fast_exp2((m - top) * kLog2e);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    return log2f(l) * kLn2;
}

}  // namespace bias
}  // namespace ragged
