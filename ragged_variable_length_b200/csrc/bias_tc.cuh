// Attention with a learned relative position bias on the 5th-generation tensor
// cores (tcgen05.mma, TMEM accumulators), f16 / bf16, head_dim 64: what the
// forward, the two gradient kernels and the weight kernel share, and the
// forward kernel.
//
// One CTA holds 128 rows of one side (queries, or keys for the transposed
// kernels) and walks over the other side in tiles of 64 columns.  Four warps
// do the element-wise work, one thread per row (TMEM lane = row); one thread
// issues every MMA; one warp loads with cp.async, so that any strides work and
// the rows past a sequence's end are zero-filled without being read.
//
// The bias of an element needs table[bucket(p_col - p_row)].  The CTA expands
// the head's column of the table once, over every distance that its rows can
// meet, into shared memory: with rmin, rmax the extremes of its rows'
// positions and R = rmax - rmin,
//     vec[o - (p_row - rmin) + D + R],   o = clamp(p_col - rmin, -D, R + D),
// 2 (D + R) + 1 entries; clamping the column's position instead of the
// distance changes nothing, because past those ends every row's distance is
// clamped already.  So an element costs one addition and one shared-memory
// load (offsets of 4 columns come with one broadcast load), whatever holes
// pruning left between the positions.  Tiles whose columns are all past one
// end add a constant; tiles with consecutive positions read consecutive
// entries without offsets.  Rows that spread over more than `span` positions
// (strong pruning, arbitrary positions) clamp every element instead.
//
// Every mbarrier wait is bounded.  A wait that gives up sets s_fail; all later
// waits are then skipped, every role finishes its loop without work, and the
// CTA flags RAGGED_DEV_TIMEOUT and frees its TMEM.  The element-wise warps
// never leave their loops early, so their named barrier always completes.
#pragma once

#include <limits.h>

#include "attn_tc05_persist.cuh"
#include "bias_common.cuh"

namespace ragged {
namespace bias {

using namespace tc05;   // tcgen05 / mbarrier / packed-fp32 wrappers

constexpr int kThreads = 192;         // 4 element-wise warps, MMA warp, load warp
constexpr int kRowWarps = 4;
constexpr int kTcMmaWarp = 4, kTcLoadWarp = 5;
constexpr int kTile = 64;             // columns per tile
constexpr int kTileBytes = kTile * 128;
constexpr int kRowBytes = kQTile * 128;
constexpr int kChunk = 512;           // columns whose offsets are in shared memory at a time
constexpr int kChunkTiles = kChunk / kTile;
constexpr int kVecPad = 64;           // a partial tile of consecutive positions reads past its last column
constexpr int kSpan = 1024;           // largest R that the expanded table covers
constexpr uint32_t kTmemCols = 256;

enum TileKind { kGeneral = 0, kLeft = 1, kRight = 2, kConsecutive = 3, kClamped = 4 };

__host__ __device__ constexpr int vec_entries(int D, int span) { return 2 * (D + span) + 1 + kVecPad; }

__device__ __forceinline__ void row_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// The expanded table and the columns' offsets of one CTA.
struct Bias {
    float* vec;
    int* off;        // [kChunk] byte offsets into vec (kClamped: positions)
    int* kind;       // [kChunkTiles]
    float* tab;      // [kMaxBuckets] the head's column of the table, base 2
    int rmin, R, D, last;   // last: index of the last entry
    bool near;
    uint32_t row;    // byte offset of this thread's row into vec
    int p_row;
};

// Extremes of the rows' positions over the 128 row threads.
__device__ __forceinline__ void bias_rows(Bias& t, const Problem& p, int pos, bool valid, int span, int* s_red) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lo = __reduce_min_sync(0xffffffffu, valid ? pos : INT_MAX);
    const int hi = __reduce_max_sync(0xffffffffu, valid ? pos : INT_MIN);
    if (lane == 0) {
        s_red[warp] = lo;
        s_red[4 + warp] = hi;
    }
    row_barrier();
    t.rmin = min(min(s_red[0], s_red[1]), min(s_red[2], s_red[3]));
    const int rmax = max(max(s_red[4], s_red[5]), max(s_red[6], s_red[7]));
    const int64_t R = static_cast<int64_t>(rmax) - t.rmin;
    t.D = p.D;
    t.near = R <= span;
    t.R = t.near ? static_cast<int>(R) : 0;
    t.last = 2 * (t.D + t.R);
    t.p_row = pos;
    t.row = valid && t.near ? 4u * static_cast<uint32_t>(t.R - (pos - t.rmin)) : 0u;
}

// Expands head h's column of the table; SIGN = 1: rows are queries, -1: rows
// are keys.  IDS: also each entry's row of the gradient accumulator (bytes).
// All 128 row threads; barriers inside.
template <typename T, int SIGN, bool IDS>
__device__ __forceinline__ void bias_expand(const Bias& t, const Problem& p, int h, uint16_t* ids) {
    const int tid = threadIdx.x;
    row_barrier();   // the previous head's table is no longer read
    if (tid < p.num_buckets) t.tab[tid] = bias_log2<T>(__ldg(p.table + static_cast<int64_t>(tid) * p.H + h));
    row_barrier();
#pragma unroll 4
    for (int x = tid; x <= t.last; x += 128) {
        const int b = bucket_of(p, SIGN * (x - t.D - t.R));
        t.vec[x] = b < 0 ? 0.f : t.tab[b];
        if constexpr (IDS) ids[x] = static_cast<uint16_t>((b < 0 ? p.num_buckets : b) * 512);
    }
    if (tid < kVecPad) {   // read by the columns past a partial tile's end, which then count as masked
        t.vec[t.last + 1 + tid] = 0.f;
        if constexpr (IDS) ids[t.last + 1 + tid] = static_cast<uint16_t>(p.num_buckets * 512);
    }
    row_barrier();
}

// Offsets and tile kinds of columns [c0, c0 + kChunk) (positions from pos_of).
// All 128 row threads; the caller puts a barrier before and after.
template <class PosOf>
__device__ __forceinline__ void bias_columns(const Bias& t, int c0, int len, PosOf pos_of) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < kChunkTiles / kRowWarps; ++k) {
        const int tile = warp + k * kRowWarps, c = c0 + tile * kTile + lane;
        if (c0 + tile * kTile >= len) break;
        const bool v0 = c < len, v1 = c + 32 < len;
        const int p0 = v0 ? pos_of(c) : 0, p1 = v1 ? pos_of(c + 32) : 0;
        const int lo = -t.D, hi = t.R + t.D;
        auto clamped = [&](int x) {
            const int64_t d = static_cast<int64_t>(x) - t.rmin;
            return d < lo ? lo : d > hi ? hi : static_cast<int>(d);
        };
        const int o0 = clamped(p0), o1 = clamped(p1);
        const int first = __shfl_sync(0xffffffffu, o0, 0);   // column 0 of a tile that has any
        const bool left = __all_sync(0xffffffffu, (!v0 || o0 == lo) && (!v1 || o1 == lo));
        const bool right = __all_sync(0xffffffffu, (!v0 || o0 == hi) && (!v1 || o1 == hi));
        const bool run = __all_sync(0xffffffffu, (!v0 || o0 == first + lane) && (!v1 || o1 == first + 32 + lane));
        int* off = t.off + tile * kTile;
        if (t.near) {
            off[lane] = v0 ? 4 * (o0 - lo) : 0;
            off[lane + 32] = v1 ? 4 * (o1 - lo) : 0;
        } else {
            off[lane] = p0;
            off[lane + 32] = p1;
        }
        if (lane == 0) t.kind[tile] = !t.near ? kClamped : left ? kLeft : right ? kRight : run ? kConsecutive : kGeneral;
    }
}

// x = x * scale + bias for 32 columns starting at column c of the tile.
__device__ __forceinline__ void bias_add(const Bias& t, int kind, const int* off, int c, float scale_log2, float (&x)[32]) {
    const uint64_t sl2 = f2(scale_log2, scale_log2);
    const char* row = reinterpret_cast<const char*>(t.vec) + t.row;
    if (kind == kLeft || kind == kRight) {
        const float e = t.vec[kind == kLeft ? 0 : t.last];
        const uint64_t b2 = f2(e, e);
#pragma unroll
        for (int i = 0; i < 16; ++i) f2_split(f2_fma(f2(x[2 * i], x[2 * i + 1]), sl2, b2), x[2 * i], x[2 * i + 1]);
    } else if (kind == kConsecutive) {
        const float* e = reinterpret_cast<const float*>(row + off[0]) + c;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            f2_split(f2_fma(f2(x[2 * i], x[2 * i + 1]), sl2, f2(e[2 * i], e[2 * i + 1])), x[2 * i], x[2 * i + 1]);
    } else if (kind == kGeneral) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int4 o = *reinterpret_cast<const int4*>(off + c + 4 * i);
            const float e0 = *reinterpret_cast<const float*>(row + o.x), e1 = *reinterpret_cast<const float*>(row + o.y);
            const float e2 = *reinterpret_cast<const float*>(row + o.z), e3 = *reinterpret_cast<const float*>(row + o.w);
            f2_split(f2_fma(f2(x[4 * i], x[4 * i + 1]), sl2, f2(e0, e1)), x[4 * i], x[4 * i + 1]);
            f2_split(f2_fma(f2(x[4 * i + 2], x[4 * i + 3]), sl2, f2(e2, e3)), x[4 * i + 2], x[4 * i + 3]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const int d = max(-t.D, min(t.D, pos_diff(off[c + i], t.p_row)));
            x[i] = fmaf(x[i], scale_log2, t.vec[d + t.D]);
        }
    }
}

// ROWS rows of one head (base = its row 0), from row0 on, into a swizzled
// tile, by one warp; rows at or past len are zero-filled without being read.
template <int ROWS>
__device__ __forceinline__ void load_rows(uint32_t s_tile, const uint16_t* base, int64_t stride, int row0, int len, int lane) {
    const int r = lane >> 3, c = lane & 7;
    const uint32_t even = s_tile + swz(r, c), odd = s_tile + swz(r + 4, c);
    const uint16_t* src = base + static_cast<int64_t>(row0 + r) * stride + c * 8;
#pragma unroll 8
    for (int i = 0; i < ROWS / 4; ++i) {
        const bool ok = row0 + r + 4 * i < len;
        cp_async_16(((i & 1) ? odd : even) + (i >> 1) * 1024, ok ? src : base, ok ? 16 : 0);
        src += 4 * stride;
    }
}

// Bounded waits of one CTA; once one has given up, no other waits.
struct Wait {
    int* s_fail;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {   // one thread
        if (*reinterpret_cast<volatile int*>(s_fail) || !mbar_wait(bar, parity)) {
            atomicExch(s_fail, 1);
            return false;
        }
        return true;
    }
    __device__ __forceinline__ bool warp(uint32_t bar, uint32_t parity) const {   // all lanes, one answer
        return __all_sync(0xffffffffu, (*this)(bar, parity));
    }
};

__device__ __forceinline__ uint32_t tmem_alloc(uint32_t* s_tmem, uint32_t cols, int warp) {
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(s_tmem)), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    return *s_tmem;
}
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t cols, int warp, const int* s_fail) {
    fence_before_sync();
    __syncthreads();
    if (*s_fail && threadIdx.x == 0) raise_status(RAGGED_DEV_TIMEOUT);
    if (warp == 0) {
        fence_after_sync();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
    }
}

// 64 values of a row (packed pairs) to 16-bit global memory.
__device__ __forceinline__ void store_row(uint16_t* dst, const uint32_t (&w)[32]) {
    if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + c * 16), "r"(w[8 * c]),
                         "r"(w[8 * c + 1]), "r"(w[8 * c + 2]), "r"(w[8 * c + 3]), "r"(w[8 * c + 4]), "r"(w[8 * c + 5]),
                         "r"(w[8 * c + 6]), "r"(w[8 * c + 7])
                         : "memory");
    } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            *reinterpret_cast<uint4*>(dst + c * 8) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    }
}
// This thread's 64 fp32 columns at taddr, times f, rounded and stored.
template <typename T>
__device__ __forceinline__ void store_tmem_row(uint32_t taddr, float f, uint16_t* dst, bool valid) {
    uint32_t w[32];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        float v[32];
        tmem_ld32(taddr + hf * 32, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) w[hf * 16 + i] = Cvt<T>::pack(v[2 * i] * f, v[2 * i + 1] * f);
    }
    if (valid) store_row(dst, w);
}

// ---------------------------------------------------------------------------
// Forward.  grid (query tiles, H, B), two CTAs per SM.
//
// TMEM (256 columns): S of three tiles, each replaced in place by its P
// (packed 16-bit pairs, the A operand of P V), and O.  Q K^T runs three tiles
// ahead of P V: the tensor core executes one thread's MMAs in order, so
// Q K^T(g + 3), issued behind P V(g), finds P(g) read.  Softmax in one pass
// with a reference maximum that is raised, and the running sum and O
// rescaled, only when a tile exceeds it by 2^8.  P is rounded to the 16-bit
// type of V: the product's operands must have one type, and the rounding
// (half a step, independent per element) adds about as much to the result as
// its own final rounding does; the sum that divides is of the unrounded P.
// ---------------------------------------------------------------------------

constexpr int kFwdK = 3, kFwdV = 5;

__host__ __device__ constexpr int fwd_smem_bytes(int D) {
    return 1024 + kRowBytes + (kFwdK + kFwdV) * kTileBytes + 4 * (vec_entries(D, kSpan) + 3) + 4 * kChunk;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) bias_fwd_kernel(const Problem p, uint16_t* __restrict__ out, int64_t out_tok) {
    extern __shared__ uint8_t smem_raw[];
    // q_full, k_full[3], v_full[5], s_full[3], p_full[4], pv_done[5], drain
    __shared__ __align__(8) uint64_t s_bar[22];
    __shared__ float s_tab[kMaxBuckets];
    __shared__ int s_kind[kChunkTiles], s_red[8];
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;

    const int q0 = blockIdx.x * kQTile, h = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Seq s;
    if (!read_pair(p, b, s) || q0 >= s.q_len) return;
    if (s.k_len == 0) {   // a query without keys
        const int r = q0 + tid;
        if (tid < kQTile && r < s.q_len) {
            const uint32_t zero[32] = {};
            store_row(out + static_cast<int64_t>(s.q_start + r) * out_tok + h * 64, zero);
            p.lse[h * p.lse_stride + s.q_start + r] = -INFINITY;
        }
        return;
    }
    const int nt = (s.k_len + kTile - 1) / kTile;

    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t sQ = (raw + 1023u) & ~1023u;
    const uint32_t sK = sQ + kRowBytes, sV = sK + kFwdK * kTileBytes;
    uint8_t* extra = smem_raw + (sV - raw) + kFwdV * kTileBytes;

    const uint32_t bar0 = smem_addr(&s_bar[0]);
    const uint32_t q_full = bar0, drain = bar0 + 8u * 21;
    auto k_full = [&](uint32_t g) { return bar0 + 8u * (1 + g % kFwdK); };
    auto v_full = [&](uint32_t g) { return bar0 + 8u * (4 + g % kFwdV); };
    auto s_full = [&](uint32_t g) { return bar0 + 8u * (9 + g % 3); };
    // Warps without rows run up to three tiles ahead of others, so four
    // consecutive tiles have barriers of their own.
    auto p_full = [&](uint32_t g) { return bar0 + 8u * (12 + (g & 3)); };
    auto pv_done = [&](uint32_t g) { return bar0 + 8u * (16 + g % kFwdV); };
    if (tid == 0) {
        mbar_init(q_full, 32);
        for (int i = 0; i < kFwdK; ++i) mbar_init(k_full(i), 32);
        for (int i = 0; i < kFwdV; ++i) mbar_init(v_full(i), 32);
        for (int i = 0; i < 3; ++i) mbar_init(s_full(i), 1);
        for (int i = 0; i < 4; ++i) mbar_init(p_full(i), 128);
        for (int i = 0; i < kFwdV; ++i) mbar_init(pv_done(i), 1);
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        s_fail = 0;
    }
    const uint32_t tmem = tmem_alloc(&s_tmem, kTmemCols, warp);
    const uint32_t o_col = 3 * kTile;
    const Wait wait{&s_fail};

    if (warp == kTcLoadWarp) {
        const int64_t z = static_cast<int64_t>(h / p.group) * p.kv_head;
        const uint16_t* qb = p.q + s.q_start * p.q_tok + h * p.q_head;
        const uint16_t* kb = p.k + s.k_start * p.kv_tok + z;
        const uint16_t* vb = p.v + s.k_start * p.kv_tok + z;
        load_rows<kQTile>(sQ, qb, p.q_tok, q0, s.q_len, lane);
        cp_async_arrive_noinc(q_full);
        bool ok = !test_hook(1);
        for (uint32_t g = 0; ok && g < static_cast<uint32_t>(nt); ++g) {
            // K stage g % 3 is free once Q K^T of tile g - 3 has finished, V
            // stage g % 5 once P V of tile g - 5 has.
            if (g >= kFwdK) ok = wait.warp(s_full(g), ((g - kFwdK) / 3) & 1);
            if (!ok) break;
            load_rows<kTile>(sK + (g % kFwdK) * kTileBytes, kb, p.kv_tok, g * kTile, s.k_len, lane);
            cp_async_arrive_noinc(k_full(g));
            if (g >= kFwdV) ok = wait.warp(pv_done(g), ((g - kFwdV) / kFwdV) & 1);
            if (!ok) break;
            load_rows<kTile>(sV + (g % kFwdV) * kTileBytes, vb, p.kv_tok, g * kTile, s.k_len, lane);
            cp_async_arrive_noinc(v_full(g));
        }
        cp_async_wait_all();
    } else if (warp == kTcMmaWarp) {
        if (lane == 0) {
            const uint32_t idesc_qk = make_idesc(Cvt<T>::kFormat, 0, kTile);
            const uint32_t idesc_pv = make_idesc(Cvt<T>::kFormat, 1, 64);
            auto issue_qk = [&](uint32_t g) {
                if (!wait(k_full(g), (g / kFwdK) & 1)) return false;
                fence_async_smem();   // cp.async wrote through the generic proxy
                fence_after_sync();
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_f16(tmem + (g % 3) * kTile, make_sdesc(sQ + ks * 32),
                            make_sdesc(sK + (g % kFwdK) * kTileBytes + ks * 32), idesc_qk, ks > 0);
                mma_commit(s_full(g));
                return true;
            };
            bool ok = wait(q_full, 0);
            const uint32_t n = nt;
            for (uint32_t g = 0; ok && g < 3 && g < n; ++g) ok = issue_qk(g);
            for (uint32_t g = 0; ok && g < n; ++g) {
                ok = wait(p_full(g), (g >> 2) & 1) && wait(v_full(g), (g / kFwdV) & 1);
                if (!ok) break;
                fence_async_smem();
                fence_after_sync();
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_f16_ts(tmem + o_col, tmem + (g % 3) * kTile + ks * 8,
                               make_sdesc(sV + (g % kFwdV) * kTileBytes + ks * 2048), idesc_pv, (g > 0 || ks > 0) ? 1u : 0u);
                mma_commit(pv_done(g));
                if (g + 3 < n) ok = issue_qk(g + 3);
            }
            mma_commit(drain);   // every MMA has finished before TMEM is freed
            mbar_wait(drain, 0);
        }
    } else {
        const int row = q0 + tid;
        const bool valid = row < s.q_len, warp_rows = q0 + warp * 32 < s.q_len;
        Bias t;
        t.vec = reinterpret_cast<float*>(extra);
        t.off = reinterpret_cast<int*>(extra + 4 * ((vec_entries(p.D, kSpan) + 3) & ~3));
        t.kind = s_kind;
        t.tab = s_tab;
        bias_rows(t, p, valid ? query_pos(p, s, row) : 0, valid, kSpan, s_red);
        bias_expand<T, 1, false>(t, p, h, nullptr);

        const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        bool ok = true;
        int pv_seen = -1;   // pv_done phases are waited for one by one, in order
        auto confirm_pv = [&](int x) {
            while (pv_seen < x) {
                ++pv_seen;
                ok = ok && wait.warp(pv_done(pv_seen), (pv_seen / kFwdV) & 1);
            }
        };
        float m_ref = -INFINITY, l0 = 0.f, l1 = 0.f;
        for (int g = 0; g < nt; ++g) {
            if (g % kChunkTiles == 0) {
                if (g) row_barrier();
                bias_columns(t, g * kTile, s.k_len, [&](int c) { return key_pos(p, s, c); });
                row_barrier();
            }
            ok = ok && wait.warp(s_full(g), (g / 3) & 1);
            if (ok && warp_rows) {
                fence_after_sync();
                const uint32_t s_buf = t_lane + static_cast<uint32_t>((g % 3) * kTile);
                const int kind = t.kind[g % kChunkTiles];
                const int* off = t.off + (g % kChunkTiles) * kTile;
                float x[2][32];
                tmem_ld32(s_buf, x[0]);
                tmem_ld32(s_buf + 32, x[1]);
                bias_add(t, kind, off, 0, p.scale_log2, x[0]);
                bias_add(t, kind, off, 32, p.scale_log2, x[1]);
                const int cols = s.k_len - g * kTile;
                if (cols < kTile) {
#pragma unroll
                    for (int i = 0; i < 64; ++i)
                        if (i >= cols) x[i >> 5][i & 31] = -INFINITY;
                }
                float mt = -INFINITY;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    float m0 = fmax3(x[hf][0], x[hf][1], x[hf][2]), m1 = fmax3(x[hf][16], x[hf][17], x[hf][18]);
#pragma unroll
                    for (int i = 3; i < 15; i += 2) {
                        m0 = fmax3(m0, x[hf][i], x[hf][i + 1]);
                        m1 = fmax3(m1, x[hf][16 + i], x[hf][17 + i]);
                    }
                    mt = fmax3(mt, fmaxf(m0, x[hf][15]), fmaxf(m1, x[hf][31]));
                }
                const bool grow = mt > m_ref + kRescaleThreshold;
                float alpha = 1.f;
                if (grow) {
                    alpha = mma_attn::fast_exp2(m_ref - mt);
                    l0 *= alpha;
                    l1 *= alpha;
                    m_ref = mt;
                }
                if (g > 0 && __any_sync(0xffffffffu, grow)) {
                    confirm_pv(g - 1);   // O holds the finished products so far
                    if (ok) {
                        fence_after_sync();
                        const uint64_t a2 = f2(alpha, alpha);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            float part[16];
                            tmem_ld16(t_lane + o_col + q * 16, part);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                f2_split(f2_mul(f2(part[2 * i], part[2 * i + 1]), a2), part[2 * i], part[2 * i + 1]);
                            tmem_st16(t_lane + o_col + q * 16, part);
                        }
                    }
                }
                // A row without a finite score so far has no reference: -inf - 0 gives p = 0.
                const float ref = m_ref == -INFINITY ? 0.f : -m_ref;
                const uint64_t nm = f2(ref, ref);
                uint64_t sum = f2(l0, l1);
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float a, c;
                        f2_split(f2_add(f2(x[hf][2 * i], x[hf][2 * i + 1]), nm), a, c);
                        a = mma_attn::fast_exp2(a);
                        c = mma_attn::fast_exp2(c);
                        sum = f2_add(sum, f2(a, c));
                        w[i] = Cvt<T>::pack(a, c);
                    }
                    tmem_st16_u(s_buf + hf * 16, w);
                }
                f2_split(sum, l0, l1);
                tmem_wait_st();
            }
            if (g >= 2) confirm_pv(g - 2);
            fence_before_sync();
            mbar_arrive(p_full(g));
        }
        confirm_pv(nt - 1);
        if (ok && warp_rows) {
            fence_after_sync();
            const float l = l0 + l1;
            const bool empty = l == 0.f;   // every score is -inf
            uint32_t w[32];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                float v[32];
                tmem_ld32(t_lane + o_col + hf * 32, v);
                const float inv = 1.f / l;
#pragma unroll
                for (int i = 0; i < 16; ++i) w[hf * 16 + i] = empty ? 0u : Cvt<T>::pack(v[2 * i] * inv, v[2 * i + 1] * inv);
            }
            if (valid) {
                store_row(out + static_cast<int64_t>(s.q_start + row) * out_tok + h * 64, w);
                p.lse[h * p.lse_stride + s.q_start + row] = empty ? -INFINITY : (m_ref + log2f(l)) * kLn2;
            }
        }
    }
    tmem_free(tmem, kTmemCols, warp, &s_fail);
}

}  // namespace bias
}  // namespace ragged
