// Attention with a learned relative position bias for few query rows per key /
// value head (one new token, or a few, against a cache; very short
// sequences), and the weights that the keys collect from them.
//
// The group * q_len rows that share a key / value head make one MMA tile of
// 16 rows (or two), so every key and value is read once for all of them: the
// kernels are bound by those reads.  Each warp streams blocks of 16 keys
// through a ring of its own (cp.async, no barrier across warps) and keeps its
// own softmax state; mma.sync is enough, because a block of 4 KB costs a warp
// 8 to 24 MMAs.  The keys of a sequence are split over the warps of a CTA and
// over the CTAs of a cluster, whose states are joined through (distributed)
// shared memory: one launch, no workspace, a fixed order.
//
// P is split into two 16-bit parts (value and residual) for P V, which costs
// nothing next to the loads and leaves the result with its own rounding only.
//
// Measured: 32 sequences of 4,096 to 8,192 keys, one query, 16 over 4 heads,
// bf16: 40 us, 5.5 TB/s of keys and values; their weights, with those so far
// read and written: 36 us.  One sequence of 577, 12 heads, f16: 7.4 and 5.1 us,
// a launch and two dependent reads.
#pragma once

#include <limits.h>

#include "bias_common.cuh"

namespace ragged {
namespace bias {

// Warps of a CTA: few for many short sequences, so that many CTAs share an SM
// (200 sequences of 4 to 6 tokens, 8 heads: 18 us, 33 us with eight warps, whose
// rings take 100 KB).
constexpr int kFewWarps = 8, kFewShortWarps = 2;
constexpr int kFewShortKeys = 512;
constexpr int kFewKeys = 16;          // keys per block
constexpr int kFewStages = 3;         // ring of a warp: two blocks in flight beside the current one
constexpr int kFewMaxRows = 32;
constexpr int kFewMaxSplits = 8;      // CTAs of a cluster

// Shared memory: the warps' rings (K, V and positions of a block), the query
// rows, the bucket map as bytes, the rows' table entries.
template <int MT, bool WEIGHT>
__host__ __device__ constexpr int few_stage_bytes() {   // keys, then values or the weights so far, then positions
    return kFewKeys * 128 + (WEIGHT ? MT * 16 * kFewKeys * 4 : kFewKeys * 128) + kFewKeys * 4;
}
// The bucket map is staged by eight warps only: a short sequence meets few distances.
template <int MT, int NW>
__host__ __device__ constexpr int few_map_bytes(int D) { return NW == kFewWarps ? (2 * D + 1 + 15) & ~15 : 0; }
template <int MT, int NW, bool WEIGHT>
__host__ __device__ constexpr int few_ring_bytes() {   // at least what the warps' states take at the end
    return WEIGHT || kFewStages * few_stage_bytes<MT, WEIGHT>() > MT * 16 * 256 ? NW * kFewStages * few_stage_bytes<MT, WEIGHT>() : NW * MT * 16 * 256;
}
template <int MT, int NW, bool WEIGHT>
__host__ __device__ constexpr int few_smem_bytes(int D, int num_buckets) {
    return few_ring_bytes<MT, NW, WEIGHT>() + MT * 16 * 128 + few_map_bytes<MT, NW>(D) + 4 * num_buckets * MT * 16;
}

__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src, int src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ float cluster_read(const float* p, uint32_t rank) {
    uint32_t a = smem_addr(p);
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %0, %2;\n\tld.shared::cluster.f32 %1, [%0];" : "+r"(a), "=f"(v) : "r"(rank) : "memory");
    return v;
}

// The residual of a pair's rounding, rounded again.
template <typename T>
__device__ __forceinline__ uint32_t pack_rest(float lo, float hi, uint32_t rounded) {
    return mma_attn::Mma<T>::pack(lo - to_float<T>(static_cast<uint16_t>(rounded)),
                                  hi - to_float<T>(static_cast<uint16_t>(rounded >> 16)));
}

// What both kernels set up: the sequence, this warp's key blocks, the query
// fragments, the rows' positions and the bias in shared memory.
template <typename T, int MT, int NW, bool WEIGHT>
struct Few {
    static constexpr int kThreadsF = 32 * NW;
    static constexpr bool kMap = NW == kFewWarps;
    static constexpr int kStage = few_stage_bytes<MT, WEIGHT>();
    Seq s;
    int z, rows, warp, lane, g, c2;   // g: row in a tile, c2: first of this lane's two columns
    int pq[MT][2];                    // positions of this lane's rows
    int q_min, q_max;
    float left[MT][2], right[MT][2];  // bias past either end of the map
    uint32_t qf[MT][4][4];
    uint32_t ring;
    const uint8_t* map;
    const float* tab;                 // [num_buckets][MT * 16]
    const uint16_t* kb;
    int64_t v_off;                    // from a key's row to its value's, elements

    __device__ __forceinline__ int head_of(const Problem& p, int row) const { return z * p.group + row / s.q_len; }
    __device__ __forceinline__ int query_of(int row) const { return row % s.q_len; }

    // What the loads need.
    __device__ __forceinline__ void begin(const Problem& p, uint8_t* smem) {
        warp = threadIdx.x >> 5;
        lane = threadIdx.x & 31;
        g = lane >> 2;
        c2 = (lane & 3) * 2;
        rows = p.group * s.q_len;
        ring = smem_addr(smem) + warp * kFewStages * kStage;
        const int64_t head = z * p.kv_head;
        kb = p.k + s.k_start * p.kv_tok + head;
        v_off = static_cast<int64_t>(reinterpret_cast<intptr_t>(p.v) - reinterpret_cast<intptr_t>(p.k)) / 2;
    }
    // What the scores need (the first blocks are on their way meanwhile).
    __device__ __forceinline__ void setup(const Problem& p, uint8_t* smem) {
        const int tid = threadIdx.x;
        uint8_t* sq = smem + few_ring_bytes<MT, NW, WEIGHT>();
        uint8_t* m = sq + MT * 16 * 128;
        float* t = reinterpret_cast<float*>(m + few_map_bytes<MT, NW>(p.D));
        map = m;
        tab = t;
        for (int i = tid; i < MT * 16 * 8; i += kThreadsF) {
            const int r = i >> 3, c = i & 7;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (r < rows)
                w = __ldg(reinterpret_cast<const uint4*>(p.q + static_cast<int64_t>(s.q_start + query_of(r)) * p.q_tok + head_of(p, r) * p.q_head) + c);
            *reinterpret_cast<uint4*>(sq + mma_attn::swz(r, c)) = w;
        }
        for (int i = tid; i < p.num_buckets * MT * 16; i += kThreadsF) {
            const int b = i / (MT * 16), r = i - b * (MT * 16);
            t[i] = r < rows ? to_float<T>(__ldg(p.table + static_cast<int64_t>(b) * p.H + head_of(p, r))) : 0.f;
        }
        if constexpr (kMap)
            for (int i = tid; i <= 2 * p.D; i += kThreadsF) m[i] = static_cast<uint8_t>(bucket_of(p, i - p.D));   // -1: 255
        q_min = INT_MAX;
        q_max = INT_MIN;
        for (int i = 0; i < s.q_len; ++i) {
            const int x = query_pos(p, s, i);
            q_min = min(q_min, x);
            q_max = max(q_max, x);
        }
#pragma unroll
        for (int t2 = 0; t2 < MT; ++t2)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = t2 * 16 + g + 8 * k;
                pq[t2][k] = r < rows ? query_pos(p, s, query_of(r)) : q_min;
            }
        __syncthreads();
        const uint32_t sQ = smem_addr(sq);
#pragma unroll
        for (int t2 = 0; t2 < MT; ++t2) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)   // rows 0-7 / 8-15 of the first, then of the second eight columns
                mma_attn::ldmatrix_x4(qf[t2][ks], sQ + mma_attn::swz(t2 * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), 2 * ks + (lane >> 4)));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                left[t2][k] = entry(p, t2 * 16 + g + 8 * k, -p.D);
                right[t2][k] = entry(p, t2 * 16 + g + 8 * k, p.D);
            }
        }
    }
    // Bias of a row for a clamped distance.
    __device__ __forceinline__ float entry(const Problem& p, int row, int d) const {
        const int b = kMap ? static_cast<int8_t>(map[d + p.D]) : bucket_of(p, d);
        return b < 0 ? 0.f : tab[b * (MT * 16) + row];
    }
    __device__ __forceinline__ uint32_t stage(int n) const { return ring + (n % kFewStages) * kStage; }
    // One block of keys (and values, positions) into stage n of this warp's ring.
    __device__ __forceinline__ void load(const Problem& p, int n, int key0) const {
        const int r = lane >> 3, c = lane & 7;
        const uint32_t st = stage(n), even = st + mma_attn::swz(r, c), odd = st + mma_attn::swz(r + 4, c);
        const uint16_t* k = kb + static_cast<int64_t>(key0 + r) * p.kv_tok + c * 8;
        const int64_t four = 4 * p.kv_tok;
        if (key0 + kFewKeys <= s.k_len) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t dst = ((i & 1) ? odd : even) + (i >> 1) * 1024;
                cp_async_16(dst, k, 16);
                if constexpr (!WEIGHT) cp_async_16(dst + kFewKeys * 128, k + v_off, 16);
                k += four;
            }
            if (p.pos_k != nullptr && lane < kFewKeys)
                cp_async_4(st + kStage - kFewKeys * 4 + 4 * lane, p.pos_k + s.k_start + key0 + lane, 4);
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // past the end: zeros
            const bool in = key0 + r + 4 * i < s.k_len;
            const uint32_t dst = ((i & 1) ? odd : even) + (i >> 1) * 1024;
            cp_async_16(dst, in ? k : kb, in ? 16 : 0);
            if constexpr (!WEIGHT) cp_async_16(dst + kFewKeys * 128, in ? k + v_off : kb, in ? 16 : 0);
            k += four;
        }
        if (p.pos_k != nullptr && lane < kFewKeys)   // past the end: a position of the block
            cp_async_4(st + kStage - kFewKeys * 4 + 4 * lane, p.pos_k + s.k_start + min(key0 + lane, s.k_len - 1), 4);
    }
    // Scores of block n (keys from key0): x[tile][8 keys][row g: 2 columns, row g + 8: 2 columns].
    __device__ __forceinline__ void scores(const Problem& p, int n, int key0, float (&x)[MT][2][4]) const {
        const uint32_t st = stage(n);
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[t][i][j] = 0.f;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            uint32_t b[4];
            mma_attn::ldmatrix_x4(b, st + mma_attn::swz((lane >> 4) * 8 + (lane & 7), 2 * ks + ((lane >> 3) & 1)));
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                mma_attn::Mma<T>::run(x[t][0], qf[t][ks], b[0], b[1]);
                mma_attn::Mma<T>::run(x[t][1], qf[t][ks], b[2], b[3]);
            }
        }
        // A block whose keys are all past one end of the map has one bias per row.
        int mine = key0 + (lane & 15);
        int64_t lo = key0, hi = key0 + kFewKeys - 1;
        if (p.pos_k != nullptr) {
            asm volatile("ld.shared.s32 %0, [%1];" : "=r"(mine) : "r"(st + kStage - kFewKeys * 4 + 4 * (lane & 15)) : "memory");
            lo = __reduce_min_sync(0xffffffffu, mine);
            hi = __reduce_max_sync(0xffffffffu, mine);
        }
        const bool all_left = hi - q_min <= -p.D;
        if (all_left || lo - q_max >= p.D) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float e = all_left ? left[t][k] : right[t][k];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j) x[t][i][2 * k + j] = fmaf(x[t][i][2 * k + j], p.scale, e);
                }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int pk = __shfl_sync(0xffffffffu, mine, i * 8 + c2 + j);
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int d = max(-p.D, min(p.D, pos_diff(pk, pq[t][k])));
                            x[t][i][2 * k + j] = fmaf(x[t][i][2 * k + j], p.scale, entry(p, t * 16 + g + 8 * k, d));
                        }
                }
        }
        if (key0 + kFewKeys > s.k_len) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (key0 + i * 8 + c2 + j >= s.k_len)
#pragma unroll
                        for (int t = 0; t < MT; ++t) x[t][i][j] = x[t][i][2 + j] = -INFINITY;
        }
    }
};

// grid (splits, Hkv, B), cluster (splits, 1, 1)
template <typename T, int MT, int NW>
__global__ void __launch_bounds__(32 * NW) bias_few_kernel(const Problem p, uint16_t* __restrict__ out, int64_t out_tok) {
    extern __shared__ __align__(128) uint8_t few_smem[];
    __shared__ float s_m[NW][MT * 16], s_l[NW][MT * 16];
    __shared__ float s_mc[MT * 16], s_lc[MT * 16];
    const int splits = gridDim.x, rank = blockIdx.x;
    Few<T, MT, NW, false> f;
    f.z = blockIdx.y;
    if (!read_pair(p, blockIdx.z, f.s) || f.s.q_len == 0) return;   // the same for the whole cluster
    f.begin(p, few_smem);
    const int blocks = (f.s.k_len + kFewKeys - 1) / kFewKeys;
    const int per = (blocks + splits * NW - 1) / (splits * NW);   // of one warp
    // A CTA's blocks are one run of keys; its warps take them in turn.
    const int first = min(blocks, rank * per * NW) + f.warp, end = min(blocks, (rank + 1) * per * NW);
#pragma unroll
    for (int n = 0; n < kFewStages - 1; ++n) {
        if (first + n * NW < end) f.load(p, n, (first + n * NW) * kFewKeys);
        cp_async_commit();
    }
    f.setup(p, few_smem);
    float m[MT][2], l[MT][2], o[MT][8][4];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        m[t][0] = m[t][1] = -INFINITY;
        l[t][0] = l[t][1] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[t][i][j] = 0.f;
    }
    int n = 0;
    for (int blk = first; blk < end; blk += NW, ++n) {
        cp_async_wait<kFewStages - 2>();
        __syncwarp();
        const int ahead = blk + (kFewStages - 1) * NW;
        if (ahead < end) f.load(p, n + kFewStages - 1, ahead * kFewKeys);
        cp_async_commit();
        float x[MT][2][4];
        f.scores(p, n, blk * kFewKeys, x);
        uint32_t hi[MT][4], lo[MT][4];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            // The reference maximum is raised only by a block that exceeds it by 2^8
            // (the first one always does); until then lanes need not agree on a maximum.
            bool grow = false;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                grow |= fmaxf(fmaxf(x[t][0][2 * k], x[t][0][2 * k + 1]), fmaxf(x[t][1][2 * k], x[t][1][2 * k + 1])) > m[t][k] + 8.f * kLn2;
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float v = fmaxf(fmaxf(x[t][0][2 * k], x[t][0][2 * k + 1]), fmaxf(x[t][1][2 * k], x[t][1][2 * k + 1]));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                    const float next = fmaxf(m[t][k], v);
                    const float alpha = next == -INFINITY ? 1.f : mma_attn::fast_exp2((m[t][k] - next) * kLog2e);
                    m[t][k] = next;
                    l[t][k] *= alpha;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        o[t][i][2 * k] *= alpha;
                        o[t][i][2 * k + 1] *= alpha;
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float ref = m[t][k] == -INFINITY ? 0.f : m[t][k];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float a = mma_attn::fast_exp2((x[t][i][2 * k] - ref) * kLog2e), b = mma_attn::fast_exp2((x[t][i][2 * k + 1] - ref) * kLog2e);
                    l[t][k] += a + b;
                    const uint32_t w = mma_attn::Mma<T>::pack(a, b);
                    hi[t][2 * i + k] = w;
                    lo[t][2 * i + k] = pack_rest<T>(a, b, w);
                }
            }
        }
        const uint32_t sv = f.stage(n) + kFewKeys * 128;
#pragma unroll
        for (int c = 0; c < 4; ++c) {   // 16 value columns
            uint32_t b[4];
            mma_attn::ldmatrix_x4_trans(b, sv + mma_attn::swz(((f.lane >> 3) & 1) * 8 + (f.lane & 7), 2 * c + (f.lane >> 4)));
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                mma_attn::Mma<T>::run(o[t][2 * c], hi[t], b[0], b[1]);
                mma_attn::Mma<T>::run(o[t][2 * c], lo[t], b[0], b[1]);
                mma_attn::Mma<T>::run(o[t][2 * c + 1], hi[t], b[2], b[3]);
                mma_attn::Mma<T>::run(o[t][2 * c + 1], lo[t], b[2], b[3]);
            }
        }
        __syncwarp();   // the stage may be overwritten
    }
    cp_async_wait<0>();
    __syncthreads();
    // The warps' states, then the CTA's, then the cluster's: out = sum e^(m - M) o / sum e^(m - M) l.
    float* so = reinterpret_cast<float*>(few_smem);   // [warp][row][64], over the rings
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = t * 16 + f.g + 8 * k;
            float v = l[t][k];
            v += __shfl_xor_sync(0xffffffffu, v, 1);
            v += __shfl_xor_sync(0xffffffffu, v, 2);
            if (f.c2 == 0) {
                s_m[f.warp][r] = m[t][k];
                s_l[f.warp][r] = v;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                *reinterpret_cast<float2*>(so + (f.warp * MT * 16 + r) * 64 + i * 8 + f.c2) = make_float2(o[t][i][2 * k], o[t][i][2 * k + 1]);
        }
    __syncthreads();
    const int rows = f.rows;
    for (int i = threadIdx.x; i < rows * 64; i += (32 * NW)) {
        const int r = i >> 6, d = i & 63;
        float top = s_m[0][r];
#pragma unroll
        for (int w = 1; w < NW; ++w) top = fmaxf(top, s_m[w][r]);
        const float ref = top == -INFINITY ? 0.f : top;
        float acc = 0.f, sum = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float a = mma_attn::fast_exp2((s_m[w][r] - ref) * kLog2e);
            acc = fmaf(a, so[(w * MT * 16 + r) * 64 + d], acc);
            sum = fmaf(a, s_l[w][r], sum);
        }
        so[r * 64 + d] = acc;   // of warp 0's part, which only this thread reads
        if (d == 0) {
            s_mc[r] = top;
            s_lc[r] = sum;
        }
    }
    if (splits > 1) cluster_sync();
    else __syncthreads();
    for (int i = rank * (32 * NW) + threadIdx.x; i < rows * 32; i += splits * (32 * NW)) {
        const int r = i >> 5, d = (i & 31) * 2;
        float a0, a1, sum, top;
        if (splits == 1) {
            top = s_mc[r];
            sum = s_lc[r];
            a0 = so[r * 64 + d];
            a1 = so[r * 64 + d + 1];
        } else {
            float mc[kFewMaxSplits];
            top = -INFINITY;
#pragma unroll
            for (int c = 0; c < kFewMaxSplits; ++c) {
                mc[c] = c < splits ? cluster_read(&s_mc[r], c) : -INFINITY;
                top = fmaxf(top, mc[c]);
            }
            const float ref = top == -INFINITY ? 0.f : top;
            a0 = a1 = sum = 0.f;
#pragma unroll
            for (int c = 0; c < kFewMaxSplits; ++c)
                if (c < splits) {
                    const float w = mma_attn::fast_exp2((mc[c] - ref) * kLog2e);
                    sum = fmaf(w, cluster_read(&s_lc[r], c), sum);
                    a0 = fmaf(w, cluster_read(so + r * 64 + d, c), a0);
                    a1 = fmaf(w, cluster_read(so + r * 64 + d + 1, c), a1);
                }
        }
        const bool empty = sum == 0.f;
        const float inv = 1.f / sum;
        const int h = f.head_of(p, r);
        const int64_t t = f.s.q_start + f.query_of(r);
        *reinterpret_cast<uint32_t*>(out + t * out_tok + h * 64 + d) = empty ? 0u : mma_attn::Mma<T>::pack(a0 * inv, a1 * inv);
        if (d == 0) p.lse[h * p.lse_stride + t] = empty ? -INFINITY : fmaf(log2f(sum), kLn2, top);
    }
    if (splits > 1) cluster_sync();   // this CTA's shared memory has been read
}

// weight[h, j] = prev[h, j] + sum_i exp(s[i, j] - lse_i).  grid (splits, Hkv, B)
template <typename T, int MT, int NW>
__global__ void __launch_bounds__(32 * NW)
    bias_few_weight_kernel(const Problem p, const float* prev, float* weight, int64_t weight_stride) {
    extern __shared__ __align__(128) uint8_t few_smem[];
    __shared__ float s_p[NW][MT * 16][kFewKeys + 1];
    __shared__ float s_log_sum[MT * 16];   // of the far rows
    const int splits = gridDim.x, rank = blockIdx.x;
    Few<T, MT, NW, true> f;
    f.z = blockIdx.y;
    if (!read_pair(p, blockIdx.z, f.s) || f.s.k_len == 0 || !keys_held(f.s, weight_stride)) return;
    const int blocks = (f.s.k_len + kFewKeys - 1) / kFewKeys;
    const int per = (blocks + splits * NW - 1) / (splits * NW);
    const int begin = min(blocks, rank * per * NW), end = min(blocks, (rank + 1) * per * NW);
    if (begin >= end) return;
    const int64_t at = f.z * p.group * weight_stride + f.s.k_start;
    if (f.s.q_len == 0) {   // nothing to add
        for (int h = 0; h < p.group; ++h)
            for (int j = begin * kFewKeys + threadIdx.x; j < min(end * kFewKeys, f.s.k_len); j += (32 * NW))
                weight[at + h * weight_stride + j] = prev != nullptr ? prev[at + h * weight_stride + j] : 0.f;
        return;
    }
    f.begin(p, few_smem);
    const int first = begin + f.warp;
    // The weights so far travel with the keys: [head][16 keys] of a stage, where there are any.
    auto load = [&](int n, int blk) {
        f.load(p, n, blk * kFewKeys);
        if (prev != nullptr) {
            const float* src = prev + at + (f.lane >> 4) * weight_stride + min(blk * kFewKeys + (f.lane & 15), f.s.k_len - 1);
            uint32_t dst = f.stage(n) + kFewKeys * 128 + 4 * f.lane;
            for (int h = f.lane >> 4; h < p.group; h += 2, src += 2 * weight_stride, dst += 128) cp_async_4(dst, src, 4);
        }
    };
#pragma unroll
    for (int n = 0; n < kFewStages - 1; ++n) {
        if (first + n * NW < end) load(n, first + n * NW);
        cp_async_commit();
    }
    f.setup(p, few_smem);
    auto lse_of = [&](int r) { return r < f.rows ? __ldg(p.lse + f.head_of(p, r) * p.lse_stride + f.s.q_start + f.query_of(r)) : -INFINITY; };
    float nl[MT][2], mu[MT][2];
    bool far = false;
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float l = lse_of(t * 16 + f.g + 8 * k);
            nl[t][k] = -lse_log2(l);
            mu[t][k] = 0.f;
            far |= is_far(l);
        }
    far = __any_sync(0xffffffffu, far);   // every warp sees all rows
    if (far) {
#pragma unroll 1
        for (int r = f.warp; r < f.rows; r += NW) {
            if (!is_far(lse_of(r))) continue;
            const float ls = row_log_sum<T>(p, f.s, f.query_of(r), f.head_of(p, r));
            if (f.lane == 0) s_log_sum[r] = ls;
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = t * 16 + f.g + 8 * k;
                const float l = lse_of(r);
                if (!is_far(l)) continue;
                nl[t][k] = -s_log_sum[r] * kLog2e;
                mu[t][k] = l - s_log_sum[r];
            }
    }
    int n = 0;
    for (int blk = first; blk < end; blk += NW, ++n) {
        cp_async_wait<kFewStages - 2>();
        __syncwarp();
        const int ahead = blk + (kFewStages - 1) * NW;
        if (ahead < end) load(n + kFewStages - 1, ahead);
        cp_async_commit();
        float x[MT][2][4];
        f.scores(p, n, blk * kFewKeys, x);
        if (far) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[t][i][j] = fminf(x[t][i][j] - mu[t][j >> 1], mu[t][j >> 1] != 0.f ? 0.f : INFINITY);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s_p[f.warp][t * 16 + f.g + 8 * (j >> 1)][i * 8 + f.c2 + (j & 1)] = mma_attn::fast_exp2(fmaf(x[t][i][j], kLog2e, nl[t][j >> 1]));
        __syncwarp();
        // Key lane % 16 of heads lane / 16, + 2, ...: this block's sums over the queries, in their order.
        const int key = f.lane & 15, h0 = f.lane >> 4, j = blk * kFewKeys + key;
        if (j < f.s.k_len) {
            float* dst = weight + at + h0 * weight_stride + j;
            const float* sp = &s_p[f.warp][h0 * f.s.q_len][key];
            uint32_t old_at = f.stage(n) + kFewKeys * 128 + 4 * f.lane;
            const int skip = f.s.q_len * (kFewKeys + 1);
            for (int h = h0; h < p.group; h += 2, dst += 2 * weight_stride, sp += 2 * skip, old_at += 128) {
                float sum = sp[0];
                for (int q = 1; q < f.s.q_len; ++q) sum += sp[q * (kFewKeys + 1)];
                float old = 0.f;
                if (prev != nullptr) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(old) : "r"(old_at) : "memory");
                *dst = old + sum;
            }
        }
        __syncwarp();   // the stage and s_p may be overwritten
    }
    cp_async_wait<0>();
}

}  // namespace bias
}  // namespace ragged
