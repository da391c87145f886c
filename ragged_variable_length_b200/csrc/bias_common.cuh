// Shared parts of the attention kernels with a learned relative position bias.
//
// For sequence b (query rows cu_q[b] .. , key rows cu_k[b] ..), query head h
// and key / value head z = h / (H / Hkv), with integer positions p of the
// tokens and buckets of the clamped relative distance:
//
//   s[i, j] = scale q_i . k_j + table[bucket(p_j - p_i), h]
//   bucket(d) = buckets[clamp(d, -D, D) + D]
//
// All kernels work in base 2: s' = s log2(e), so that one fused multiply-add
// and ex2.approx give exp(s - m) = 2^(s' - m').
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
    return ok;
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

// A table entry in base 2.  A finite entry stays finite (the lowest bf16 value
// times log2 e would not): a row whose keys all carry the lowest value keeps
// its softmax over them, as it does in base e.
template <typename T>
__device__ __forceinline__ float bias_log2(uint16_t x) {
    const float v = to_float<T>(x);
    const float s = v * kLog2e;
    return fabsf(v) == INFINITY ? v : fminf(fmaxf(s, -1.7e38f), 1.7e38f);
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

}  // namespace bias
}  // namespace ragged
