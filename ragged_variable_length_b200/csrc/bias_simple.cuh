// Plain kernels of the attention with a relative position bias: one warp per
// row, one lane per row of the other side, fp32 arithmetic on the CUDA cores.
#pragma once

#include "bias_common.cuh"

namespace ragged {
namespace bias {

constexpr int kSimpleWarps = 4;

// Dot product of 64 fp32 values in shared memory with a 16-bit row.
template <typename T>
__device__ __forceinline__ float dot64(const float* x, const uint16_t* row) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(row) + c);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s = fmaf(x[c * 8 + 2 * i], to_float<T>(static_cast<uint16_t>(u[i])), s);
            s = fmaf(x[c * 8 + 2 * i + 1], to_float<T>(static_cast<uint16_t>(u[i] >> 16)), s);
        }
    }
    return s;
}
__device__ __forceinline__ float warp_add(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
template <typename T>
__device__ __forceinline__ float score_log2(const Problem& p, float qk, int delta, int h) {
    const int b = bucket_of(p, delta);
    return fmaf(qk, p.scale_log2, b < 0 ? 0.f : bias_log2<T>(p.table[static_cast<int64_t>(b) * p.H + h]));
}

// grid (query tiles of 128, H, B)
template <typename T>
__global__ void bias_fwd_simple(Problem p, uint16_t* out, int64_t out_tok) {
    __shared__ float s_q[kSimpleWarps][64];
    const int h = blockIdx.y, b = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Seq s;
    if (!read_pair(p, b, s)) return;
    const uint16_t* kb = p.k + s.k_start * p.kv_tok + (h / p.group) * p.kv_head;
    const uint16_t* vb = p.v + s.k_start * p.kv_tok + (h / p.group) * p.kv_head;
    for (int r = warp; r < kQTile; r += kSimpleWarps) {
        const int i = blockIdx.x * kQTile + r;
        if (i >= s.q_len) break;
        const uint16_t* q = p.q + (s.q_start + i) * p.q_tok + h * p.q_head;
        __syncwarp();
        s_q[warp][lane] = to_float<T>(q[lane]);
        s_q[warp][lane + 32] = to_float<T>(q[lane + 32]);
        __syncwarp();
        const int pq = query_pos(p, s, i);
        float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
        for (int j0 = 0; j0 < s.k_len; j0 += 32) {
            const int j = j0 + lane;
            float x = -INFINITY;
            if (j < s.k_len)
                x = score_log2<T>(p, dot64<T>(s_q[warp], kb + j * p.kv_tok), pos_diff(key_pos(p, s, j), pq), h);
            const float mt = fmaxf(m, warp_max(x));
            const float ref = mt == -INFINITY ? 0.f : mt;
            const float alpha = exp2f(m - ref), e = exp2f(x - ref);
            m = mt;
            l = l * alpha + warp_add(e);
            o0 *= alpha;
            o1 *= alpha;
            const int n = min(32, s.k_len - j0);
            for (int u = 0; u < n; ++u) {
                const float w = __shfl_sync(0xffffffffu, e, u);
                const uint16_t* v = vb + (j0 + u) * p.kv_tok;
                o0 = fmaf(w, to_float<T>(v[2 * lane]), o0);
                o1 = fmaf(w, to_float<T>(v[2 * lane + 1]), o1);
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint16_t* dst = out + (s.q_start + i) * out_tok + h * 64;
        dst[2 * lane] = from_float<T>(o0 * inv);
        dst[2 * lane + 1] = from_float<T>(o1 * inv);
        if (lane == 0) p.lse[h * p.lse_stride + s.q_start + i] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
}

struct BwdArgs {
    const uint16_t* out;
    const uint16_t* dout;
    int64_t out_tok, dout_tok;
    uint16_t* dq;
    uint16_t* dk;
    uint16_t* dv;
    int64_t dq_tok, dq_head, dkv_tok, dkv_head;
    float* delta;     // [H, lse_stride]: sum over the head dimension of out * d out
    float* partial;   // [B][H][query tiles][num_buckets]
    uint16_t* dtable;
    int q_tiles;
};

// Gradient of the queries, delta, and partial sums of the table's gradient.
// grid (query tiles, H, B)
template <typename T>
__global__ void bias_bwd_q_simple(Problem p, BwdArgs a) {
    __shared__ float s_q[kSimpleWarps][64], s_do[kSimpleWarps][64];
    __shared__ float s_acc[kMaxBuckets][kSimpleWarps * 32];
    const int h = blockIdx.y, b = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int n = 0; n < p.num_buckets; ++n) s_acc[n][threadIdx.x] = 0.f;
    Seq s;
    if (!read_pair(p, b, s)) s.q_len = 0;
    const uint16_t* kb = p.k + s.k_start * p.kv_tok + (h / p.group) * p.kv_head;
    const uint16_t* vb = p.v + s.k_start * p.kv_tok + (h / p.group) * p.kv_head;
    for (int r = warp; r < kQTile; r += kSimpleWarps) {
        const int i = blockIdx.x * kQTile + r;
        if (i >= s.q_len) break;
        const int64_t t = s.q_start + i;
        const uint16_t* q = p.q + t * p.q_tok + h * p.q_head;
        const uint16_t* d = a.dout + t * a.dout_tok + h * 64;
        const uint16_t* o = a.out + t * a.out_tok + h * 64;
        __syncwarp();
        s_q[warp][lane] = to_float<T>(q[lane]);
        s_q[warp][lane + 32] = to_float<T>(q[lane + 32]);
        s_do[warp][lane] = to_float<T>(d[lane]);
        s_do[warp][lane + 32] = to_float<T>(d[lane + 32]);
        __syncwarp();
        const float delta = warp_add(s_do[warp][lane] * to_float<T>(o[lane]) + s_do[warp][lane + 32] * to_float<T>(o[lane + 32]));
        if (lane == 0) a.delta[h * p.lse_stride + t] = delta;
        const float lse = lse_log2(p.lse[h * p.lse_stride + t]);
        const int pq = query_pos(p, s, i);
        float g0 = 0.f, g1 = 0.f;
        for (int j0 = 0; j0 < s.k_len; j0 += 32) {
            const int j = j0 + lane;
            float ds = 0.f;
            if (j < s.k_len) {
                const int dist = pos_diff(key_pos(p, s, j), pq), bk = bucket_of(p, dist);
                const float x = score_log2<T>(p, dot64<T>(s_q[warp], kb + j * p.kv_tok), dist, h);
                ds = exp2f(x - lse) * (dot64<T>(s_do[warp], vb + j * p.kv_tok) - delta);
                if (bk >= 0) s_acc[bk][threadIdx.x] += ds;
            }
            const int n = min(32, s.k_len - j0);
            for (int u = 0; u < n; ++u) {
                const float w = __shfl_sync(0xffffffffu, ds, u);
                const uint16_t* k = kb + (j0 + u) * p.kv_tok;
                g0 = fmaf(w, to_float<T>(k[2 * lane]), g0);
                g1 = fmaf(w, to_float<T>(k[2 * lane + 1]), g1);
            }
        }
        uint16_t* dst = a.dq + t * a.dq_tok + h * a.dq_head;
        dst[2 * lane] = from_float<T>(g0 * p.scale);
        dst[2 * lane + 1] = from_float<T>(g1 * p.scale);
    }
    __syncthreads();
    float* dst = a.partial + ((static_cast<int64_t>(b) * p.H + h) * a.q_tiles + blockIdx.x) * p.num_buckets;
    for (int n = warp; n < p.num_buckets; n += kSimpleWarps) {
        float x = 0.f;
        for (int u = lane; u < kSimpleWarps * 32; u += 32) x += s_acc[n][u];
        x = warp_add(x);
        if (lane == 0) dst[n] = x;
    }
}

// Gradients of the keys and values.  grid (key tiles of 128, Hkv, B)
template <typename T>
__global__ void bias_bwd_kv_simple(Problem p, BwdArgs a) {
    __shared__ float s_k[kSimpleWarps][64], s_v[kSimpleWarps][64];
    const int z = blockIdx.y, b = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Seq s;
    if (!read_pair(p, b, s)) return;
    for (int r = warp; r < kQTile; r += kSimpleWarps) {
        const int j = blockIdx.x * kQTile + r;
        if (j >= s.k_len) break;
        const int64_t t = s.k_start + j;
        const uint16_t* k = p.k + t * p.kv_tok + z * p.kv_head;
        const uint16_t* v = p.v + t * p.kv_tok + z * p.kv_head;
        __syncwarp();
        s_k[warp][lane] = to_float<T>(k[lane]);
        s_k[warp][lane + 32] = to_float<T>(k[lane + 32]);
        s_v[warp][lane] = to_float<T>(v[lane]);
        s_v[warp][lane + 32] = to_float<T>(v[lane + 32]);
        __syncwarp();
        const int pk = key_pos(p, s, j);
        float dk0 = 0.f, dk1 = 0.f, dv0 = 0.f, dv1 = 0.f;
        for (int h = z * p.group; h < (z + 1) * p.group; ++h) {
            const uint16_t* qb = p.q + s.q_start * p.q_tok + h * p.q_head;
            const uint16_t* db = a.dout + s.q_start * a.dout_tok + h * 64;
            for (int i0 = 0; i0 < s.q_len; i0 += 32) {
                const int i = i0 + lane;
                float e = 0.f, ds = 0.f;
                if (i < s.q_len) {
                    const int64_t u = h * p.lse_stride + s.q_start + i;
                    const float x = score_log2<T>(p, dot64<T>(s_k[warp], qb + i * p.q_tok), pos_diff(pk, query_pos(p, s, i)), h);
                    e = exp2f(x - lse_log2(p.lse[u]));
                    ds = e * (dot64<T>(s_v[warp], db + i * a.dout_tok) - a.delta[u]);
                }
                const int n = min(32, s.q_len - i0);
                for (int u = 0; u < n; ++u) {
                    const float w = __shfl_sync(0xffffffffu, e, u), x = __shfl_sync(0xffffffffu, ds, u);
                    const uint16_t* d = db + (i0 + u) * a.dout_tok;
                    const uint16_t* q = qb + (i0 + u) * p.q_tok;
                    dv0 = fmaf(w, to_float<T>(d[2 * lane]), dv0);
                    dv1 = fmaf(w, to_float<T>(d[2 * lane + 1]), dv1);
                    dk0 = fmaf(x, to_float<T>(q[2 * lane]), dk0);
                    dk1 = fmaf(x, to_float<T>(q[2 * lane + 1]), dk1);
                }
            }
        }
        uint16_t* gk = a.dk + t * a.dkv_tok + z * a.dkv_head;
        uint16_t* gv = a.dv + t * a.dkv_tok + z * a.dkv_head;
        gk[2 * lane] = from_float<T>(dk0 * p.scale);
        gk[2 * lane + 1] = from_float<T>(dk1 * p.scale);
        gv[2 * lane] = from_float<T>(dv0);
        gv[2 * lane + 1] = from_float<T>(dv1);
    }
}

// dtable[n, h] = sum of the partial sums, in a fixed order.  grid (num_buckets, H)
template <typename T>
__global__ void bias_bwd_table(Problem p, BwdArgs a) {
    __shared__ float s_sum[8];
    const int n = blockIdx.x, h = blockIdx.y, tiles = a.q_tiles;
    float x = 0.f;
    for (int i = threadIdx.x; i < p.B * tiles; i += 256) {
        const int b = i / tiles, t = i - b * tiles;
        x += a.partial[((static_cast<int64_t>(b) * p.H + h) * tiles + t) * p.num_buckets + n];
    }
    x = warp_add(x);
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = x;
    __syncthreads();
    if (threadIdx.x == 0) {
        x = 0.f;
        for (int w = 0; w < 8; ++w) x += s_sum[w];
        a.dtable[static_cast<int64_t>(n) * p.H + h] = from_float<T>(x);
    }
}

// weight[h, j] = prev[h, j] + sum_i exp(s[i, j] - lse_i).  grid (key tiles of 128, H, B)
template <typename T>
__global__ void bias_weight_simple(Problem p, const float* prev, float* weight, int64_t weight_stride) {
    __shared__ float s_k[kSimpleWarps][64];
    const int h = blockIdx.y, b = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Seq s;
    if (!read_pair(p, b, s)) return;
    for (int r = warp; r < kQTile; r += kSimpleWarps) {
        const int j = blockIdx.x * kQTile + r;
        if (j >= s.k_len) break;
        const uint16_t* k = p.k + (s.k_start + j) * p.kv_tok + (h / p.group) * p.kv_head;
        __syncwarp();
        s_k[warp][lane] = to_float<T>(k[lane]);
        s_k[warp][lane + 32] = to_float<T>(k[lane + 32]);
        __syncwarp();
        const int pk = key_pos(p, s, j);
        float sum = 0.f;
        for (int i = lane; i < s.q_len; i += 32) {
            const int64_t t = s.q_start + i;
            const float x = score_log2<T>(p, dot64<T>(s_k[warp], p.q + t * p.q_tok + h * p.q_head), pos_diff(pk, query_pos(p, s, i)), h);
            sum += exp2f(x - lse_log2(p.lse[h * p.lse_stride + t]));
        }
        sum = warp_add(sum);
        if (lane == 0) {
            const int64_t u = h * weight_stride + s.k_start + j;
            weight[u] = (prev != nullptr ? prev[u] : 0.f) + sum;
        }
    }
}

}  // namespace bias
}  // namespace ragged
