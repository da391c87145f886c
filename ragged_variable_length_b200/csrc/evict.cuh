// Eviction of tokens by the attention weight that they collected.
//
// Sequence b keeps m_b = clamp(budget[b], 0, L_b) of its tokens: the first
// `sinks` and the last `recents` ones before all others, then those with the
// largest total = fp32(sum over heads of weight[h, t], summed in fp64).  Ties
// go to the lower index, NaN ranks below every number.
#pragma once

#include "common.cuh"

namespace ragged {
namespace evict {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kCopyThreads = 256;

struct Args {
    const float* weight;      // [H, weight_stride]
    int64_t weight_stride;
    const int32_t* cu;
    const int32_t* budget;
    const int32_t* pos;       // or NULL: place within the sequence
    int B, H, max_seqlen, sinks, recents;
    int64_t capacity;         // rows of the outputs
    int32_t* cu_out;
    int32_t* src_idx;
    int32_t* pos_out;         // or NULL
    float* weight_out;        // [H, weight_out_stride] or NULL
    int64_t weight_out_stride;
    const uint4* rows;
    uint4* rows_out;
    uint32_t nvec;            // 16-byte vectors per row
};

// Unsigned order = the order of the totals: -0 folded onto +0, every NaN 0.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
// Tokens that sequence b keeps (0 for one that must be skipped).
__device__ __forceinline__ int kept_of(const Args& a, int b, bool flag) {
    const int start = __ldg(a.cu + b), len = __ldg(a.cu + b + 1) - start;
    if (start < 0 || len < 0 || len > a.max_seqlen) {
        if (flag) raise_status(RAGGED_DEV_BAD_SEQLENS);
        return 0;
    }
    return max(0, min(__ldg(a.budget + b), len));
}

// One CTA per sequence: totals, the m_b-th largest key (four 8-bit radix
// steps over keys in shared memory; integer counts, so no order enters), then
// the kept tokens in ascending order.
__global__ void __launch_bounds__(kThreads) select_kernel(Args a) {
    extern __shared__ uint32_t s_key[];
    __shared__ int s_hist[256];
    __shared__ int s_sum[kWarps], s_sum2[kWarps];
    __shared__ uint32_t s_prefix;
    __shared__ int s_need;
    const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // Output row of this sequence: what the sequences before it keep.
    int before = 0;
    for (int i = tid; i < b; i += kThreads) before += kept_of(a, i, false);
    before = warp_sum(before);
    if (lane == 0) s_sum[warp] = before;
    const int m = kept_of(a, b, tid == 0);
    __syncthreads();
    before = warp_sum(lane < kWarps ? s_sum[lane] : 0);
    if (tid == 0) {
        if (b == 0) a.cu_out[0] = 0;
        a.cu_out[b + 1] = before + m;
        if (static_cast<int64_t>(before) + m > a.capacity) raise_status(RAGGED_DEV_CAPACITY);
    }
    if (m == 0) return;
    const int start = __ldg(a.cu + b), len = __ldg(a.cu + b + 1) - start;

    uint32_t cut = 0;     // keys above it stay
    int need = len;       // and this many equal to it
    if (m < len) {
        for (int t = tid; t < len; t += kThreads) {
            uint32_t key = 0xffffffffu;
            if (t >= a.sinks && t < len - a.recents) {
                double x = 0.0;
                const float* w = a.weight + start + t;
#pragma unroll 8
                for (int h = 0; h < a.H; ++h) x += static_cast<double>(__ldg(w + h * a.weight_stride));
                key = order_key(static_cast<float>(x));
            }
            s_key[t] = key;
        }
        if (tid == 0) {
            s_prefix = 0;
            s_need = m;
        }
#pragma unroll 1
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) s_hist[tid] = 0;
            __syncthreads();
            const uint32_t prefix = s_prefix;
            const int want = s_need;
            for (int t = tid; t < len; t += kThreads) {
                const uint32_t k = s_key[t];
                if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&s_hist[(k >> shift) & 255u], 1);
            }
            __syncthreads();
            if (warp == 0) {   // the digit where the count from the top reaches `want`
                int c[8], mine = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    c[i] = s_hist[255 - (lane * 8 + i)];
                    mine += c[i];
                }
                int incl = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += y;
                }
                int above = incl - mine;
                if (above < want && want <= incl) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (above < want && want <= above + c[i]) {
                            s_prefix = prefix | (static_cast<uint32_t>(255 - (lane * 8 + i)) << shift);
                            s_need = want - above;
                        }
                        above += c[i];
                    }
                }
            }
            __syncthreads();
        }
        cut = s_prefix;
        need = s_need;
    }
    // Each warp takes a contiguous run of tokens: counts, then places.
    const int run = ((len + kWarps - 1) / kWarps + 31) & ~31;
    const int t0 = warp * run, t1 = min(len, t0 + run);
    int gt = 0, eq = 0;
    if (m < len) {
        for (int t = t0 + lane; t < t1; t += 32) {
            gt += s_key[t] > cut;
            eq += s_key[t] == cut;
        }
    } else {
        eq = max(0, t1 - t0 - lane + 31) / 32;   // every token counts as equal
    }
    gt = warp_sum(gt);
    eq = warp_sum(eq);
    __syncthreads();
    if (lane == 0) {
        s_sum[warp] = gt;
        s_sum2[warp] = eq;
    }
    __syncthreads();
    gt = warp_sum(lane < warp ? s_sum[lane] : 0);
    eq = warp_sum(lane < warp ? s_sum2[lane] : 0);
    for (int tb = t0; tb < t1; tb += 32) {
        const int t = tb + lane;
        bool is_gt = false, is_eq = false;
        if (t < t1) {
            if (m < len) {
                is_gt = s_key[t] > cut;
                is_eq = s_key[t] == cut;
            } else {
                is_eq = true;
            }
        }
        const unsigned bg = __ballot_sync(0xffffffffu, is_gt), be = __ballot_sync(0xffffffffu, is_eq);
        const unsigned lower = (1u << lane) - 1u;
        const int g = gt + __popc(bg & lower), e = eq + __popc(be & lower);
        if (is_gt || (is_eq && e < need)) {
            const int64_t o = static_cast<int64_t>(before) + g + min(e, need);
            if (o < a.capacity) {
                a.src_idx[o] = start + t;
                if (a.pos_out != nullptr) a.pos_out[o] = a.pos != nullptr ? __ldg(a.pos + start + t) : t;
            }
        }
        gt += __popc(bg);
        eq += __popc(be);
    }
}

// Gathers the kept rows (blockIdx.y = 0, one warp per row) and their weights
// (blockIdx.y = 1 + head, one thread per token).
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(Args a) {
    const int64_t total = min(static_cast<int64_t>(__ldg(a.cu_out + a.B)), a.capacity);
    if (blockIdx.y == 0) {
        if (a.rows == nullptr) return;
        const int lane = threadIdx.x & 31;
        const int64_t warps = static_cast<int64_t>(gridDim.x) * (kCopyThreads / 32);
        for (int64_t r = static_cast<int64_t>(blockIdx.x) * (kCopyThreads / 32) + (threadIdx.x >> 5); r < total; r += warps) {
            const uint4* src = a.rows + static_cast<int64_t>(__ldg(a.src_idx + r)) * a.nvec;
            uint4* dst = a.rows_out + r * a.nvec;
#pragma unroll 4
            for (uint32_t v = lane; v < a.nvec; v += 32) dst[v] = __ldcs(src + v);
        }
    } else {
        const int h = blockIdx.y - 1;
        const int64_t step = static_cast<int64_t>(gridDim.x) * kCopyThreads;
        for (int64_t r = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x; r < total; r += step)
            a.weight_out[h * a.weight_out_stride + r] = __ldg(a.weight + h * a.weight_stride + __ldg(a.src_idx + r));
    }
}

}  // namespace evict
}  // namespace ragged
