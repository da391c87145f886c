// Eviction of tokens by the attention weight that they collected.
//
// Sequence b keeps m_b = clamp(budget[b], 0, L_b) of its tokens: the first
// `sinks` and the last `recents` ones before all others, then those with the
// largest total = fp32(sum over heads of weight[h, t], summed in fp64).  Ties
// go to the lower index, NaN ranks below every number.
//
// Reading the weights and copying the kept rows is all the traffic there is;
// the selection is exact and in integers.  Measured: 32 sequences of 4,096 to
// 8,192 tokens, half of them kept, rows of 1 KB, 16 heads: keys 4.6 us,
// selection 12.5 us (one CTA per sequence, its keys in registers), copy 40.5 us
// (5.4 TB/s read and written); 4 of 79 to 197, rows of 2,304 bytes: 8.4 us in
// one launch.  A selection by bisection of the key range took 41 to 64 us, one
// shared by a cluster's CTAs no less than one CTA's.
#pragma once

#include "common.cuh"

namespace ragged {
namespace evict {

constexpr int kCopyThreads = 256;
// Sequences whose keys are in shared memory and whose places one warp scans:
// a lane per group of 32 tokens.
constexpr int kShortThreads = 256, kShortLen = RAGGED_EVICT_ONE_LAUNCH;
static_assert(kShortLen <= 32 * 32, "one lane per group of 32 tokens");
constexpr int kLongThreads = 1024, kLongKeys = RAGGED_MAX_TOKENS / kLongThreads;

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
    uint32_t* keys;           // [tokens] order keys of the long sequences' tokens
    int64_t tokens;
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
    if (start < 0 || len < 0 || len > a.max_seqlen || static_cast<int64_t>(start) + len > a.tokens) {
        if (flag) raise_status(RAGGED_DEV_BAD_SEQLENS);
        return 0;
    }
    return max(0, min(__ldg(a.budget + b), len));
}

// Order key of token t of a sequence (its first row: start).
__device__ __forceinline__ uint32_t token_key(const Args& a, int start, int len, int t) {
    if (t < a.sinks || t >= len - a.recents) return 0xffffffffu;
    double x = 0.0;
    const float* w = a.weight + start + t;
#pragma unroll 8
    for (int h = 0; h < a.H; ++h) x += static_cast<double>(__ldg(w + h * a.weight_stride));
    return order_key(static_cast<float>(x));
}
// Rows that the sequences before b keep, summed over the CTA (s_red: one int per
// warp).  Every CTA reads all sequences before its own: 57 us in all for 8,192
// sequences of 8 tokens, 1.6 ms for 65,535 of one.
template <int NT>
__device__ __forceinline__ int kept_before(const Args& a, int b, int* s_red) {
    int n = 0;
    for (int i = threadIdx.x; i < b; i += NT) n += kept_of(a, i, false);
    n = warp_sum(n);
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = n;
    __syncthreads();
    return warp_sum((threadIdx.x & 31) < NT / 32 ? s_red[threadIdx.x & 31] : 0);
}
__device__ __forceinline__ void write_bounds(const Args& a, int b, int before, int m) {
    if (b == 0) a.cu_out[0] = 0;
    a.cu_out[b + 1] = before + m;
    if (static_cast<int64_t>(before) + m > a.capacity) raise_status(RAGGED_DEV_CAPACITY);
}
__device__ __forceinline__ void write_kept(const Args& a, int64_t o, int start, int t) {
    if (o < a.capacity) {
        a.src_idx[o] = start + t;
        if (a.pos_out != nullptr) a.pos_out[o] = a.pos != nullptr ? __ldg(a.pos + start + t) : t;
    }
}

// Copies kept rows first * 4 .., + step * 4 .. of a run of `total` that begins
// at output row out0, one warp per four rows, eight vectors a lane in flight;
// row r comes from input row src(r).
template <class Src>
__device__ __forceinline__ void copy_rows(const Args& a, int64_t out0, int total, int first, int step, Src src) {
    const int lane = threadIdx.x & 31;
    total = static_cast<int>(min(static_cast<int64_t>(total), a.capacity - out0));
    for (int r0 = first * 4; r0 < total; r0 += step * 4) {
        const int n = min(4, total - r0);
        const uint4* from[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) from[i] = a.rows + static_cast<int64_t>(src(r0 + min(i, n - 1))) * a.nvec;
        uint4* to = a.rows_out + (out0 + r0) * a.nvec;
        for (uint32_t v = lane; v < a.nvec; v += 64) {
            uint4 w[2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (v + 32 * k < a.nvec) w[k][i] = __ldcs(from[i] + v + 32 * k);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (v + 32 * k < a.nvec && i < n) to[static_cast<int64_t>(i) * a.nvec + v + 32 * k] = w[k][i];
        }
    }
}

// Keys above `cut` stay, and of those equal to it the first `need` ones.
struct Cut {
    uint32_t cut;
    int need;
};

// The m-th largest of the CTA's keys (each(f) calls f(k) for every key of this
// thread, with the same number of calls in all lanes; a lane without a key
// passes in = false): three radix steps of 11, 11 and 10 bits from the top.
// Integer counts in shared memory: no order enters.  Lanes of a warp that all
// hit one bin (equal weights) add once.  1 <= m <= number of keys.
template <int NT, class Each>
__device__ __forceinline__ Cut radix_cut(int m, int* s_hist, int* s_warp, int* s_next, Each each) {
    constexpr int W = NT / 32, BINS = 2048, R = BINS / NT;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t prefix = 0;
    int want = m;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
#pragma unroll
        for (int r = 0; r < R; ++r) s_hist[tid + r * NT] = 0;
        __syncthreads();
        each([&](uint32_t k, bool in) {
            in = in && (pass == 0 || ((k ^ prefix) >> (shift + bits)) == 0);
            const unsigned who = __ballot_sync(0xffffffffu, in);
            if (!in) return;
            const int d = static_cast<int>((k >> shift) & ((1u << bits) - 1u));
            int same;
            __match_all_sync(who, d, &same);
            if (!same) atomicAdd(&s_hist[d], 1);
            else if (lane == __ffs(who) - 1) atomicAdd(&s_hist[d], __popc(who));
        });
        __syncthreads();
        // The bin, from the top, where the count reaches `want`.
        int c[R], mine = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            c[r] = s_hist[BINS - 1 - (tid * R + r)];
            mine += c[r];
        }
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) s_warp[warp] = incl;
        __syncthreads();
        int above = incl - mine + warp_sum(lane < warp && lane < W ? s_warp[lane] : 0);
        if (above < want && want <= above + mine) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (above < want && want <= above + c[r]) {
                    s_next[0] = BINS - 1 - (tid * R + r);
                    s_next[1] = want - above;
                }
                above += c[r];
            }
        }
        __syncthreads();
        prefix |= static_cast<uint32_t>(s_next[0]) << shift;
        want = s_next[1];
    }
    return Cut{prefix, want};
}

// Short sequences, one launch: grid (splits, B).  Every CTA forms the keys of
// its sequence and selects by itself, then copies its share of the rows.  Up
// to 256 tokens each thread counts the tokens ahead of its own; more go
// through the radix steps.
__global__ void __launch_bounds__(kShortThreads) short_kernel(const Args a) {
    constexpr int NT = kShortThreads, W = NT / 32;
    __shared__ __align__(16) uint32_t s_key[kShortLen];
    __shared__ int s_src[kShortLen];
    __shared__ int s_hist[2048];
    __shared__ int s_red[W], s_next[2];
    __shared__ int s_place[2][kShortLen / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, split = blockIdx.x, b = blockIdx.y;
    const int m = kept_of(a, b, tid == 0 && split == 0);
    const int start = __ldg(a.cu + b), len = __ldg(a.cu + b + 1) - start;   // valid where m > 0
    if (m > 0 && m < len)
        for (int t = tid; t < ((len + 3) & ~3); t += NT) s_key[t] = t < len ? token_key(a, start, len, t) : 0u;
    const int before = kept_before<NT>(a, b, s_red);   // a barrier inside: s_key is complete
    if (tid == 0 && split == 0) write_bounds(a, b, before, m);
    if (m == 0) return;
    auto place = [&](int r, int t) {
        s_src[r] = start + t;
        if (split == 0) write_kept(a, static_cast<int64_t>(before) + r, start, t);
    };
    if (m == len) {
        for (int t = tid; t < len; t += NT) place(t, t);
    } else if (len <= NT) {
        // Kept: fewer than m tokens rank ahead.  Places by a scan of the ballots.
        bool keep = false;
        if (tid < len) {
            const uint32_t mine = s_key[tid];
            int ahead = 0;
            for (int j = 0; j < len; j += 4) {
                const uint4 k = *reinterpret_cast<const uint4*>(s_key + j);
                ahead += (k.x > mine || (k.x == mine && j < tid)) + (k.y > mine || (k.y == mine && j + 1 < tid)) +
                         (k.z > mine || (k.z == mine && j + 2 < tid)) + (k.w > mine || (k.w == mine && j + 3 < tid));
            }
            keep = ahead < m;   // (the padding, key 0 behind the last token, is ahead of none)
        }
        const unsigned who = __ballot_sync(0xffffffffu, keep);
        if (lane == 0) s_place[0][warp] = __popc(who);
        __syncthreads();
        const int base = warp_sum(lane < warp && lane < W ? s_place[0][lane] : 0);
        if (keep) place(base + __popc(who & ((1u << lane) - 1u)), tid);
    } else {
        const Cut c = radix_cut<NT>(m, s_hist, s_red, s_next, [&](auto f) {
            for (int i = 0; i < len; i += NT) f(i + tid < len ? s_key[i + tid] : 0u, i + tid < len);
        });
        for (int i = warp * 32; i < len; i += NT) {   // ballots of every 32 tokens
            const bool in = i + lane < len;
            const unsigned gt = __ballot_sync(0xffffffffu, in && s_key[i + lane] > c.cut);
            const unsigned eq = __ballot_sync(0xffffffffu, in && s_key[i + lane] == c.cut);
            if (lane == 0) {
                s_place[0][i >> 5] = __popc(gt);
                s_place[1][i >> 5] = __popc(eq);
            }
        }
        __syncthreads();
        for (int i = warp * 32; i < len; i += NT) {
            const int before_g = warp_sum(lane < (i >> 5) ? s_place[0][lane] : 0), before_e = warp_sum(lane < (i >> 5) ? s_place[1][lane] : 0);
            const bool in = i + lane < len, is_gt = in && s_key[i + lane] > c.cut, is_eq = in && s_key[i + lane] == c.cut;
            const unsigned gt = __ballot_sync(0xffffffffu, is_gt), eq = __ballot_sync(0xffffffffu, is_eq), lower = (1u << lane) - 1u;
            const int e = before_e + __popc(eq & lower);
            if (is_gt || (is_eq && e < c.need)) place(before_g + __popc(gt & lower) + min(e, c.need), i + lane);
        }
    }
    __syncthreads();
    if (a.rows != nullptr) copy_rows(a, before, m, split * W + warp, gridDim.x * W, [&](int r) { return s_src[r]; });
    if (a.weight_out != nullptr) {
        const int end = static_cast<int>(max(int64_t(0), min(static_cast<int64_t>(m), a.capacity - before)));
        for (int h = warp + W * split; h < a.H; h += W * gridDim.x)
            for (int r = lane; r < end; r += 32)
                a.weight_out[h * a.weight_out_stride + before + r] = __ldg(a.weight + h * a.weight_stride + s_src[r]);
    }
}

// Long sequences: the keys of all tokens (grid (chunks of 256 tokens, B)), ...
__global__ void __launch_bounds__(256) keys_kernel(const Args a) {
    const int b = blockIdx.y, m = kept_of(a, b, false);
    const int start = __ldg(a.cu + b), len = __ldg(a.cu + b + 1) - start;
    const int t = blockIdx.x * 256 + threadIdx.x;
    if (m > 0 && m < len && t < len) a.keys[start + t] = token_key(a, start, len, t);
}

// ... the selection, one CTA per sequence with the keys in registers, ...
__global__ void __launch_bounds__(kLongThreads) long_kernel(const Args a) {
    constexpr int NT = kLongThreads, W = NT / 32, KEYS = kLongKeys;
    __shared__ int s_hist[2048];
    __shared__ int s_red[W], s_next[2];
    __shared__ int s_place[2][KEYS * W];
    __shared__ int s_wsum[2][W];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, b = blockIdx.x;
    const int m = kept_of(a, b, tid == 0);
    const int start = __ldg(a.cu + b), len = __ldg(a.cu + b + 1) - start;
    const int steps = (len + NT - 1) / NT;
    uint32_t key[KEYS];
    if (m > 0 && m < len) {
#pragma unroll
        for (int i = 0; i < KEYS; ++i) {
            const int t = i * NT + tid;
            key[i] = t < len ? a.keys[start + t] : 0u;
        }
    }
    const int before = kept_before<NT>(a, b, s_red);
    if (tid == 0) write_bounds(a, b, before, m);
    if (m == 0) return;
    uint32_t cut = 0;
    int need = len;
    if (m < len) {
        const Cut c = radix_cut<NT>(m, s_hist, s_red, s_next, [&](auto f) {
#pragma unroll
            for (int i = 0; i < KEYS; ++i)
                if (i < steps) f(key[i], i * NT + tid < len);
        });
        cut = c.cut;
        need = c.need;
    }
    // Places of the kept tokens: ballots per (step, warp), scanned in token order.
#pragma unroll
    for (int i = 0; i < KEYS; ++i) {
        if (i >= steps) break;
        const bool in = i * NT + tid < len;
        const unsigned gt = __ballot_sync(0xffffffffu, in && m < len && key[i] > cut);
        const unsigned eq = __ballot_sync(0xffffffffu, in && (m == len || key[i] == cut));
        if (lane == 0) {
            s_place[0][i * W + warp] = __popc(gt);
            s_place[1][i * W + warp] = __popc(eq);
        }
    }
    __syncthreads();
    static_assert(KEYS * W <= NT && W == 32, "one entry per thread, one warp total per lane");
    int v[2], incl[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        v[k] = tid < steps * W ? s_place[k][tid] : 0;
        incl[k] = v[k];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl[k], o);
            if (lane >= o) incl[k] += y;
        }
        if (lane == 31) s_wsum[k][warp] = incl[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int base = __reduce_add_sync(0xffffffffu, lane < warp ? s_wsum[k][lane] : 0);
        if (tid < KEYS * W) s_place[k][tid] = base + incl[k] - v[k];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < KEYS; ++i) {
        if (i >= steps) break;
        const int t = i * NT + tid;
        const bool in = t < len, is_gt = in && m < len && key[i] > cut, is_eq = in && (m == len || key[i] == cut);
        const unsigned gt = __ballot_sync(0xffffffffu, is_gt), eq = __ballot_sync(0xffffffffu, is_eq);
        const unsigned lower = (1u << lane) - 1u;
        const int g = s_place[0][i * W + warp] + __popc(gt & lower), e = s_place[1][i * W + warp] + __popc(eq & lower);
        if (is_gt || (is_eq && e < need)) write_kept(a, static_cast<int64_t>(before) + g + min(e, need), start, t);
    }
}

// ... and the gather of the kept rows (blockIdx.y = 0) and their weights
// (blockIdx.y = 1 + head, one thread per token).
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const Args a) {
    const int total = static_cast<int>(min(static_cast<int64_t>(__ldg(a.cu_out + a.B)), a.capacity));
    if (blockIdx.y == 0) {
        if (a.rows == nullptr) return;
        copy_rows(a, 0, total, blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5), gridDim.x * (kCopyThreads / 32),
                  [&](int r) { return __ldg(a.src_idx + r); });
    } else {
        const int h = blockIdx.y - 1;
        const int r = blockIdx.x * kCopyThreads + threadIdx.x;
        if (r < total) a.weight_out[h * a.weight_out_stride + r] = __ldg(a.weight + h * a.weight_stride + __ldg(a.src_idx + r));
    }
}

}  // namespace evict
}  // namespace ragged
