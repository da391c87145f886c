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
constexpr int kTcMmaWarp = 4, kTcLoadWarp = 5;
constexpr int kTile = 64;             // columns per tile
constexpr int kTileBytes = kTile * 128;
constexpr int kRowBytes = kQTile * 128;
constexpr int kChunk = 512;           // columns whose offsets are in shared memory at a time
constexpr int kChunkTiles = kChunk / kTile;
constexpr int kVecPad = 64;           // a partial tile of consecutive positions reads past its last column
constexpr int kSpan = 1024;           // largest R that the expanded table covers
constexpr uint32_t kTmemCols = 256;

enum TileKind { kGeneral = 0, kLeft = 1, kRight = 2, kConsecutive = 3, kClamped = 4, kFarKind = 5 };

__host__ __device__ constexpr int vec_entries(int D, int span) { return 2 * (D + span) + 1 + kVecPad; }

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

// A waiting thread sleeps for up to kWaitNs before it looks again: without the
// hint the polls of the MMA and load warps took more issue slots than the
// element-wise work (60 % of all instructions).
constexpr uint32_t kWaitNs = 4000;
// A wait gives up by time, because the hint is an upper limit: a poll may come
// back at once.  2^18 full sleeps are about a second; the polls have a limit
// too, which is past that even at 20 cycles each.
constexpr uint32_t kWaitLimit = 1u << 18;
constexpr uint32_t kWaitPolls = 1u << 28;

__device__ __forceinline__ bool mbar_try(uint32_t mbar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done)
        : "r"(mbar), "r"(parity), "r"(kWaitNs)
        : "memory");
    return done != 0;
}
// Bounded waits of one CTA; once one has given up, the others soon do.
struct Wait {
    int* s_fail;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {   // one thread
        if (mbar_try(bar, parity)) return true;
        const int64_t limit = static_cast<int64_t>(min(spin_limit(), kWaitLimit)) * (2 * kWaitNs);   // cycles, at up to 2 GHz
        const int64_t start = clock64();
        for (uint32_t i = 0; i < kWaitPolls; ++i) {
            if (mbar_try(bar, parity)) return true;
            if (*reinterpret_cast<volatile int*>(s_fail)) return false;
            if (clock64() - start > limit) break;
        }
        atomicExch(s_fail, 1);
        return false;
    }
    __device__ __forceinline__ bool warp(uint32_t bar, uint32_t parity) const {   // all lanes, one answer
        return __all_sync(0xffffffffu, (*this)(bar, parity));
    }
};

// 32 values of a row (packed pairs) to 16-bit global memory.
__device__ __forceinline__ void store_half_row(uint16_t* dst, const uint32_t (&w)[16]) {
    if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + c * 16), "r"(w[8 * c]),
                         "r"(w[8 * c + 1]), "r"(w[8 * c + 2]), "r"(w[8 * c + 3]), "r"(w[8 * c + 4]), "r"(w[8 * c + 5]),
                         "r"(w[8 * c + 6]), "r"(w[8 * c + 7])
                         : "memory");
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4*>(dst + c * 8) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
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
// ---------------------------------------------------------------------------
// The bias of a group of 128 row threads in 16 bits: the entries are the
// table's own values, so nothing is lost, and 32 rows that spread over 64
// positions read 32 words, one per bank, where fp32 entries would take two or
// three passes.  Scores are formed in base e, x = s * scale + bias, and the
// factor log2 e goes into the exponent's multiply-add.
// ---------------------------------------------------------------------------

// What a tile of columns is for the rows of one warp.
struct TileInfo {
    int lo, hi;   // extremes of the columns' positions
    int kind;     // kConsecutive, kGeneral or kClamped
    int unused;
};

struct Bias16 {
    uint16_t* vec;    // [2 (D + span) + 1 + pad], one head's entries
    int* off;         // [kChunk] byte offsets into vec (kClamped: positions)
    TileInfo* tiles;  // [kChunkTiles]
    int rmin, R, D, last;
    int wlo, whi;     // extremes of the positions of this warp's rows
    bool near;
    uint32_t row;     // byte offset of this thread's row
    int p_row;
};

// Barrier of the NR (128 or 256) row threads.
template <int NR>
__device__ __forceinline__ void rows_barrier() {
    asm volatile("bar.sync 1, %0;" ::"n"(NR) : "memory");
}

// The same, and whether any of the threads has x.
template <int NR>
__device__ __forceinline__ bool rows_any(bool x) {
    int any;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbar.red.or.pred q, 1, %2, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
                 : "=r"(any)
                 : "r"(static_cast<int>(x)), "n"(NR)
                 : "memory");
    return any != 0;
}

// The bucket map as bytes in shared memory (none: an entry outside the table).
template <int NR>
__device__ __forceinline__ void bias_map(const Problem& p, uint8_t* map, int none) {
#pragma unroll 2
    for (int x = threadIdx.x; x <= 2 * p.D; x += NR) {
        const int b = bucket_of(p, x - p.D);
        map[x] = static_cast<uint8_t>(b < 0 ? none : b);
    }
}
// Extremes of the row positions (s_red: 2 * NR / 32 ints; a barrier inside,
// which also completes the map).  With 256 threads each half holds all rows.
template <int NR>
__device__ __forceinline__ void bias_rows(Bias16& t, const Problem& p, int pos, bool valid, int span, int* s_red) {
    constexpr int W = NR / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    t.wlo = __reduce_min_sync(0xffffffffu, valid ? pos : INT_MAX);
    t.whi = __reduce_max_sync(0xffffffffu, valid ? pos : INT_MIN);
    if (lane == 0) {
        s_red[warp] = t.wlo;
        s_red[W + warp] = t.whi;
    }
    rows_barrier<NR>();
    t.rmin = min(min(s_red[0], s_red[1]), min(s_red[2], s_red[3]));
    const int rmax = max(max(s_red[W], s_red[W + 1]), max(s_red[W + 2], s_red[W + 3]));
    const int64_t R = static_cast<int64_t>(rmax) - t.rmin;
    t.D = p.D;
    t.near = R <= span;
    t.R = t.near ? static_cast<int>(R) : 0;
    t.last = 2 * (t.D + t.R);
    t.p_row = pos;
    t.row = valid && t.near ? 2u * static_cast<uint32_t>(t.R - (pos - t.rmin)) : 0u;
}
// The bucket of every entry, once per CTA.  SIGN = 1: rows are queries, -1: keys.
template <int SIGN, int NR>
__device__ __forceinline__ void bias_ids(const Bias16& t, const uint8_t* map, uint8_t* ids, int none) {
#pragma unroll 4
    for (int x = threadIdx.x; x <= t.last; x += NR)
        ids[x] = map[max(-t.D, min(t.D, SIGN * (x - t.D - t.R))) + t.D];
    for (int x = t.last + 1 + threadIdx.x; x <= t.last + kVecPad; x += NR) ids[x] = static_cast<uint8_t>(none);   // past a partial tile's end
}
// One head's entries from its column of the table; tab[none] = 0.
template <int NR>
__device__ __forceinline__ void bias_fill(const Bias16& t, const uint8_t* ids, const uint16_t* tab) {
#pragma unroll 4
    for (int x = threadIdx.x; x <= t.last + kVecPad; x += NR) t.vec[x] = tab[ids[x]];
}
// Positions of columns [c0, c0 + kChunk), loaded ahead of what needs them.
template <int NR>
struct Columns {
    static constexpr int K = kChunkTiles / (NR / 32);   // tiles of a warp
    int pos[K][2];
    template <class PosOf>
    __device__ __forceinline__ void load(int c0, int len, PosOf pos_of) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = c0 + (warp + k * (NR / 32)) * kTile + lane;
            pos[k][0] = c < len ? pos_of(c) : 0;
            pos[k][1] = c + 32 < len ? pos_of(c + 32) : 0;
        }
    }
    // Offsets and kinds; barriers around it are the caller's.  Places past the last
    // column: with REPEAT they get its bias, so that an entry of the table that
    // no pair uses, which may be anything, stays out of sight of kernels that
    // only add -inf there; without, the caller masks them.
    template <bool REPEAT = false>
    __device__ __forceinline__ void store(const Bias16& t, int c0, int len) const {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const int lo = -t.D, hi = t.R + t.D;
        auto clamped = [&](int x) {
            const int64_t d = static_cast<int64_t>(x) - t.rmin;
            return d < lo ? lo : d > hi ? hi : static_cast<int>(d);
        };
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int tile = warp + k * (NR / 32), c = c0 + tile * kTile + lane;
            if (c0 + tile * kTile >= len) break;   // the whole warp
            const bool v0 = c < len, v1 = c + 32 < len;
            int p0 = pos[k][0], p1 = pos[k][1];
            if constexpr (REPEAT) {
                const int end = min(len - c0 - tile * kTile, kTile) - 1;
                const int p_end = __shfl_sync(0xffffffffu, end < 32 ? p0 : p1, end & 31);
                if (!v0) p0 = p_end;
                if (!v1) p1 = p_end;
            }
            const int o0 = clamped(p0), o1 = clamped(p1);
            const int first = __shfl_sync(0xffffffffu, o0, 0);
            const bool any0 = !REPEAT && !v0, any1 = !REPEAT && !v1;   // places whose bias does not matter
            const bool run = __all_sync(0xffffffffu, (any0 || o0 == first + lane) && (any1 || o1 == first + 32 + lane));
            const int pmin = __reduce_min_sync(0xffffffffu, min(v0 ? p0 : INT_MAX, v1 ? p1 : INT_MAX));
            const int pmax = __reduce_max_sync(0xffffffffu, max(v0 ? p0 : INT_MIN, v1 ? p1 : INT_MIN));
            int* off = t.off + tile * kTile;
            off[lane] = !t.near ? p0 : !any0 ? 2 * (o0 - lo) : 0;
            off[lane + 32] = !t.near ? p1 : !any1 ? 2 * (o1 - lo) : 0;
            if (lane == 0) t.tiles[tile] = TileInfo{pmin, pmax, !t.near ? kClamped : run ? kConsecutive : kGeneral, 0};
        }
    }
};
// The kind of a tile for this warp: all its distances past one end of the map
// (one bias for all), or what the columns allow.
__device__ __forceinline__ int tile_kind(const Bias16& t, int tile) {
    const int4 i = *reinterpret_cast<const int4*>(t.tiles + tile);
    return pos_diff(i.y, t.wlo) <= -t.D ? kLeft : pos_diff(i.x, t.whi) >= t.D ? kRight : i.z;
}
// x = x * scale + bias for 32 columns from column c of a tile (not for kLeft,
// kRight).  kFarKind (with FAR), whatever the columns' positions: the largest
// score of the far rows or columns is taken off, mu or mu_cols (0: not far).
template <typename T, bool FAR = false>
__device__ __forceinline__ void bias_add(const Bias16& t, int kind, const int* off, int c, float scale, float (&x)[32],
                                         const float* mu_cols = nullptr, float mu = 0.f) {
    const uint64_t sc2 = f2(scale, scale);
    const char* row = reinterpret_cast<const char*>(t.vec) + t.row;
    auto at = [&](int o) { return to_float<T>(*reinterpret_cast<const uint16_t*>(row + o)); };
    if (kind == kConsecutive) {
        const char* e = row + off[0] + 2 * c;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float e0 = to_float<T>(*reinterpret_cast<const uint16_t*>(e + 4 * i)), e1 = to_float<T>(*reinterpret_cast<const uint16_t*>(e + 4 * i + 2));
            f2_split(f2_fma(f2(x[2 * i], x[2 * i + 1]), sc2, f2(e0, e1)), x[2 * i], x[2 * i + 1]);
        }
    } else if (kind == kGeneral) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int4 o = *reinterpret_cast<const int4*>(off + c + 4 * i);
            f2_split(f2_fma(f2(x[4 * i], x[4 * i + 1]), sc2, f2(at(o.x), at(o.y))), x[4 * i], x[4 * i + 1]);
            f2_split(f2_fma(f2(x[4 * i + 2], x[4 * i + 3]), sc2, f2(at(o.z), at(o.w))), x[4 * i + 2], x[4 * i + 3]);
        }
    } else if (!FAR || kind == kClamped) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const int d = max(-t.D, min(t.D, pos_diff(off[c + i], t.p_row)));
            x[i] = fmaf(x[i], scale, to_float<T>(t.vec[d + t.D]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const int o = off[c + i];   // of a place past both ends of the map it is that end's
            const float e = t.near ? at(o) : to_float<T>(t.vec[max(-t.D, min(t.D, pos_diff(o, t.p_row))) + t.D]);
            const float m = mu_cols != nullptr ? mu_cols[c + i] : mu;
            x[i] = fminf(fmaf(x[i], scale, e) - m, m != 0.f ? 0.f : INFINITY);
        }
    }
}

// ---------------------------------------------------------------------------
// Forward.  grid (query tiles, groups of heads, B), two CTAs per SM.
//
// A CTA holds the positions of its 128 queries and walks over its heads; the
// tile counter runs on from head to head, so the loads and the first scores of
// a head are under way while the one before it finishes.  TMEM (256 columns): S of
// three tiles, each replaced in place by its P (packed 16-bit pairs, the A
// operand of P V), and O.  Q K^T runs three tiles ahead of P V: the tensor
// core executes one thread's MMAs in order, so Q K^T(g + 3), issued behind
// P V(g), finds P(g) read.  A head's result is read out of O when the first P
// of the next head is ready, before it is handed over (its product overwrites
// O).
//
// Softmax in one pass with a reference maximum that is raised, and the running
// sum and O rescaled, only when a tile exceeds it by 2^8.  P is rounded to the
// 16-bit type of V: the product's operands must have one type, and the
// rounding (half a step, independent per element) adds about as much to the
// result as its own final rounding does (bf16: 0.0023 of the result's norm
// instead of 0.0017); the sum that divides is of the unrounded P.  A second
// operand for the residual, as the kernels for few rows have it, costs 23 and
// 18 % in bf16 (121 instead of 98 us, 680 instead of 576, for the first two
// shapes below), because the row warps form it.
//
// Bound by the latency of the row warps' work, not by the tensor core or memory
// (issue slots a third busy): per element one table entry is read from shared
// memory.  With all places taken, a tile of 128 x 64 costs a CTA 1.3 us where
// every distance is past one end of the map and 1.6 where the entries are
// gathered, a head 2.3 us besides; the last CTAs of a grid end later than an even
// split would (four waves: some 20 %).
// Measured: 64 sequences of 173 to 403 tokens, 12 heads, bf16, positions with
// gaps: 98 us, the least that memory and products allow is 18; 2 of 4,914 to
// 8,191, 12 over 4 heads: 576 us, 433 TFLOP/s; 4 of 79 to 118, 6 heads, f16:
// 8.0 us, of which most is the launch and one chain of dependent reads.
//
// Tried against an earlier state of this (104 and 580 us for the first two): eight
// row warps that share each tile (half the columns each): 112 and 651 us; two
// groups of row warps on two heads with registers moved between roles: 220 and
// 1,069 us; waits without the sleep hint: 110 and 573 us.
// ---------------------------------------------------------------------------

constexpr int kFwdK = 3, kFwdV = 5;

__host__ __device__ constexpr int fwd_fixed_bytes() { return 1024 + 2 * kRowBytes + (kFwdK + kFwdV) * kTileBytes + 4 * kChunk; }
__host__ __device__ constexpr int vec16_bytes(int D, int span) { return 2 * ((vec_entries(D, span) + 7) & ~7); }
__host__ __device__ constexpr int ids_bytes(int D, int span) {   // and the bucket map
    return ((vec_entries(D, span) + 15) & ~15) + ((2 * D + 1 + 15) & ~15);
}
__host__ __device__ constexpr int fwd_smem_bytes(int D, int span) {
    return fwd_fixed_bytes() + 2 * vec16_bytes(D, span) + ids_bytes(D, span);
}

// One lane of a converged warp, chosen by the hardware: the compiler then knows
// that the branch holds one thread, and keeps the MMAs' descriptors, which are
// the same in all lanes, in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// The start of a CTA: the load warp sets up the barriers and begins at once,
// the MMA warp takes the TMEM and waits for the barriers, the row threads join
// when they have prepared the bias.
__device__ __forceinline__ void start_loads() { asm volatile("bar.arrive 2, 64;" ::: "memory"); }
__device__ __forceinline__ uint32_t start_mma(uint32_t* s_tmem, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(s_tmem)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    fence_before_sync();
    asm volatile("bar.sync 2, 64;" ::: "memory");
    asm volatile("bar.arrive 3, 160;" ::: "memory");
    fence_after_sync();
    return *s_tmem;
}
__device__ __forceinline__ uint32_t start_rows(const uint32_t* s_tmem) {
    asm volatile("bar.sync 3, 160;" ::: "memory");
    fence_after_sync();
    return *s_tmem;
}
// The end: all roles meet, and the MMA warp frees the TMEM.
__device__ __forceinline__ void finish_cta(const uint32_t* s_tmem, uint32_t cols, int warp, const int* s_fail) {
    fence_before_sync();
    __syncthreads();
    if (*s_fail && threadIdx.x == 0) raise_status(RAGGED_DEV_TIMEOUT);
    if (warp == kTcMmaWarp) {
        fence_after_sync();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(*s_tmem), "r"(cols) : "memory");
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
    bias_fwd_kernel(const Problem p, uint16_t* __restrict__ out, int64_t out_tok, int heads_per_cta, int span) {
    extern __shared__ uint8_t smem_raw[];
    // q_full[2], q_empty[2], k_full[3], v_full[5], s_full[3], p_full[4], pv_done[5], done
    constexpr int kBars = 25;
    __shared__ __align__(8) uint64_t s_bar[kBars];
    __shared__ uint16_t s_tab[2][kMaxBuckets + 1];
    __shared__ __align__(16) TileInfo s_tiles[kChunkTiles];
    __shared__ int s_red[8];
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;

    const int q0 = blockIdx.x * kQTile, h0 = blockIdx.y * heads_per_cta, b = blockIdx.z;
    const int nh = min(heads_per_cta, p.H - h0);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Seq s;
    if (!read_pair(p, b, s) || q0 >= s.q_len) return;
    if (s.k_len == 0) {   // queries without keys
        for (int i = tid; i < nh * kQTile; i += kThreads) {
            const int h = h0 + i / kQTile, r = q0 + i % kQTile;
            if (r >= s.q_len) continue;
            const uint32_t zero[32] = {};
            store_row(out + static_cast<int64_t>(s.q_start + r) * out_tok + h * 64, zero);
            p.lse[h * p.lse_stride + s.q_start + r] = -INFINITY;
        }
        return;
    }
    const int nt = (s.k_len + kTile - 1) / kTile;
    const uint32_t total = static_cast<uint32_t>(nt) * nh;   // tiles of all heads

    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t sQ = (raw + 1023u) & ~1023u;   // two buffers, by head
    const uint32_t sK = sQ + 2 * kRowBytes, sV = sK + kFwdK * kTileBytes;
    uint8_t* extra = smem_raw + (sV - raw) + kFwdV * kTileBytes;
    const uint32_t bar0 = smem_addr(&s_bar[0]);
    auto q_full = [&](uint32_t i) { return bar0 + 8u * (i & 1); };
    auto q_empty = [&](uint32_t i) { return bar0 + 8u * (2 + (i & 1)); };
    auto k_full = [&](uint32_t g) { return bar0 + 8u * (4 + g % kFwdK); };
    auto v_full = [&](uint32_t g) { return bar0 + 8u * (7 + g % kFwdV); };
    auto s_full = [&](uint32_t g) { return bar0 + 8u * (12 + g % 3); };
    // Warps without rows run up to three tiles ahead of others, so four
    // consecutive tiles have barriers of their own.
    auto p_full = [&](uint32_t g) { return bar0 + 8u * (15 + (g & 3)); };
    auto pv_done = [&](uint32_t g) { return bar0 + 8u * (19 + g % kFwdV); };
    const uint32_t done = bar0 + 8u * 24;
    constexpr uint32_t o_col = 3 * kTile;
    const Wait wait{&s_fail};

    if (warp == kTcLoadWarp) {
        // ---------------- loads ----------------
        if (lane < kBars) mbar_init(bar0 + 8 * lane, lane < 2 || (lane >= 4 && lane < 12) ? 32 : lane >= 15 && lane < 19 ? 128 : 1);
        if (lane == 0) s_fail = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        __syncwarp();
        start_loads();
        bool ok = !test_hook(1);
        uint32_t g = 0;
        for (int i = 0; ok && i < nh; ++i) {
            const int h = h0 + i;
            const int64_t z = static_cast<int64_t>(h / p.group) * p.kv_head;
            const uint16_t* kb = p.k + s.k_start * p.kv_tok + z;
            const uint16_t* vb = p.v + s.k_start * p.kv_tok + z;
            if (i >= 2) ok = wait.warp(q_empty(i), ((i >> 1) - 1) & 1);
            if (!ok) break;
            load_rows<kQTile>(sQ + (i & 1) * kRowBytes, p.q + s.q_start * p.q_tok + h * p.q_head, p.q_tok, q0, s.q_len, lane);
            cp_async_arrive_noinc(q_full(i));
            for (int t = 0; t < nt; ++t, ++g) {
                // K stage g % 3 is free once Q K^T of tile g - 3 has finished, V
                // stage g % 5 once P V of tile g - 5 has.
                if (g >= kFwdK) ok = wait.warp(s_full(g), (g / 3 - 1) & 1);
                if (!ok) break;
                load_rows<kTile>(sK + (g % kFwdK) * kTileBytes, kb, p.kv_tok, t * kTile, s.k_len, lane);
                cp_async_arrive_noinc(k_full(g));
                if (g >= kFwdV) ok = wait.warp(pv_done(g), (g / kFwdV - 1) & 1);
                if (!ok) break;
                load_rows<kTile>(sV + (g % kFwdV) * kTileBytes, vb, p.kv_tok, t * kTile, s.k_len, lane);
                cp_async_arrive_noinc(v_full(g));
            }
        }
        cp_async_wait_all();
    } else if (warp == kTcMmaWarp) {
        // ---------------- MMA issue (one elected thread; the warp waits as one) ----------------
        const uint32_t tmem = uniform(start_mma(&s_tmem, kTmemCols));
        const uint32_t n = uniform(total), per_head = uniform(nt);
        const uint32_t idesc_qk = make_idesc(Cvt<T>::kFormat, 0, kTile), idesc_pv = make_idesc(Cvt<T>::kFormat, 1, 64);
        const bool leader = elect_one();
        uint32_t qi = 0, qt = 0;   // head and tile of the next scores
        auto issue_qk = [&](uint32_t g) {
            if (qt == 0 && !wait.warp(q_full(qi), (qi >> 1) & 1)) return false;
            if (!wait.warp(k_full(g), (g / kFwdK) & 1)) return false;
            fence_async_smem();   // cp.async wrote through the generic proxy
            fence_after_sync();
            const uint32_t sq = sQ + (qi & 1) * kRowBytes, sk = sK + (g % kFwdK) * kTileBytes, d = tmem + (g % 3) * kTile;
            if (leader) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_f16(d, make_sdesc(sq + ks * 32), make_sdesc(sk + ks * 32), idesc_qk, ks > 0);
                mma_commit(s_full(g));
                if (qt + 1 == per_head) mma_commit(q_empty(qi));
            }
            __syncwarp();
            if (++qt == per_head) {
                qt = 0;
                ++qi;
            }
            return true;
        };
        bool ok = true;
        for (uint32_t g = 0; ok && g < 3 && g < n; ++g) ok = issue_qk(g);
        uint32_t t = 0;
        for (uint32_t g = 0; ok && g < n; ++g) {
            ok = wait.warp(v_full(g), (g / kFwdV) & 1) && wait.warp(p_full(g), (g >> 2) & 1);
            if (!ok) break;
            fence_async_smem();
            fence_after_sync();
            const uint32_t pa = tmem + (g % 3) * kTile, sv = sV + (g % kFwdV) * kTileBytes;
            if (leader) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_f16_ts(tmem + o_col, pa + ks * 8, make_sdesc(sv + ks * 2048), idesc_pv, (t > 0 || ks > 0) ? 1u : 0u);
                mma_commit(pv_done(g));
            }
            __syncwarp();
            if (g + 3 < n) ok = issue_qk(g + 3);
            if (++t == per_head) t = 0;
        }
        if (leader) {
            mma_commit(done);   // every MMA has finished before TMEM is freed
            mbar_wait(done, 0);
        }
        __syncwarp();
    } else {
        // ---------------- softmax and results (one thread per query) ----------------
        const int row = q0 + tid;
        const bool valid = row < s.q_len, warp_rows = q0 + warp * 32 < s.q_len;
        const int64_t t_row = s.q_start + row;
        Bias16 t;
        uint16_t* const vec0 = reinterpret_cast<uint16_t*>(extra);
        const int vec_step = vec16_bytes(p.D, span) / 2;
        uint8_t* ids = extra + 2 * vec16_bytes(p.D, span);
        t.vec = vec0;
        t.off = reinterpret_cast<int*>(ids + ids_bytes(p.D, span));
        t.tiles = s_tiles;
        uint8_t* map = ids + ((vec_entries(p.D, span) + 15) & ~15);
        const bool has_entry = tid < p.num_buckets;   // of the table's column of a head
        const uint16_t* column = p.table + static_cast<int64_t>(has_entry ? tid : 0) * p.H + h0;
        // What the set-up needs of global memory, all under way at once.
        const uint16_t entry = __ldg(column);
        const int pos = valid ? query_pos(p, s, row) : 0;
        auto key_at = [&](int c) { return key_pos(p, s, c); };
        Columns<128> cols;
        cols.load(0, s.k_len, key_at);
        bias_map<128>(p, map, p.num_buckets);
        if (has_entry) s_tab[0][tid] = entry;
        if (tid == p.num_buckets) s_tab[0][tid] = s_tab[1][tid] = 0;
        bias_rows<128>(t, p, pos, valid, span, s_red);
        bias_ids<1, 128>(t, map, ids, p.num_buckets);
        cols.store(t, 0, s.k_len);
        rows_barrier<128>();
        bias_fill<128>(t, ids, s_tab[0]);
        const uint32_t tmem = start_rows(&s_tmem);

        const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        const uint32_t o_lane = t_lane + o_col;
        bool ok = true;
        uint32_t g = 0;
        // Products up to tile x have finished.  Called when the scores of tile
        // x + 1 or later have been seen, which were issued behind P V(x - 2): the
        // barrier's earlier phases are over, so the parity is exact.
        auto confirm_pv = [&](uint32_t x) { ok = ok && wait.warp(pv_done(x), (x / kFwdV) & 1); };
        float l_done = 0.f, m_done = 0.f;   // of the head before
        // Result of head h, whose last product was tile x's.
        auto finish = [&](int h, uint32_t x, float m, float l) {
            confirm_pv(x);
            if (!ok || !warp_rows) return;
            fence_after_sync();
            const bool empty = l == 0.f;   // every score is -inf
            const float inv = 1.f / l;
            uint16_t* dst = out + t_row * out_tok + h * 64;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                float v[32];
                tmem_ld32(o_lane + hf * 32, v);
                uint32_t pk[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) pk[j] = empty ? 0u : Cvt<T>::pack(v[2 * j] * inv, v[2 * j + 1] * inv);
                if (valid) store_half_row(dst + hf * 32, pk);
            }
            if (valid) p.lse[h * p.lse_stride + t_row] = empty ? -INFINITY : fmaf(log2f(l), kLn2, m);
        };
        for (int i = 0; i < nh; ++i) {
            // This head's entries are complete and the last head's no longer read after
            // this barrier; the next head's are filled in behind it.
            if (i + 1 < nh && has_entry) s_tab[(i + 1) & 1][tid] = __ldg(column + i + 1);
            rows_barrier<128>();
            if (i + 1 < nh) {
                t.vec = vec0 + ((i + 1) & 1) * vec_step;
                bias_fill<128>(t, ids, s_tab[(i + 1) & 1]);
            }
            t.vec = vec0 + (i & 1) * vec_step;
            float m_ref = -INFINITY, neg_ref = 0.f, l0 = 0.f, l1 = 0.f;   // neg_ref: -m_ref in base 2, or 0
            bool far = false;                                              // some row of the warp is
            for (int tile = 0; tile < nt; ++tile, ++g) {
                if (tile % kChunkTiles == 0 && (tile > 0 || (i > 0 && nt > kChunkTiles))) {
                    cols.load(tile * kTile, s.k_len, key_at);
                    if (tile > 0) rows_barrier<128>();
                    cols.store(t, tile * kTile, s.k_len);
                    rows_barrier<128>();
                }
                const int kind = tile_kind(t, tile % kChunkTiles);
                const int* off = t.off + (tile % kChunkTiles) * kTile;
                ok = ok && wait.warp(s_full(g), (g / 3) & 1);
                if (ok && warp_rows) {
                    fence_after_sync();
                    const uint32_t s_buf = t_lane + static_cast<uint32_t>((g % 3) * kTile);
                    float x[2][32];
                    tmem_ld32(s_buf, x[0]);
                    tmem_ld32(s_buf + 32, x[1]);
                    // Scores in base 2 are x * scale + add; one bias for the whole tile goes into `add`.
                    const bool flat = kind == kLeft || kind == kRight;
                    float scale = kLog2e, add = 0.f, entry = 0.f;
                    if (flat) {
                        scale = p.scale_log2;
                        entry = to_float<T>(t.vec[kind == kLeft ? 0 : t.last]);
                        add = entry * kLog2e;
                    } else {
                        bias_add<T>(t, kind, off, 0, p.scale, x[0]);
                        bias_add<T>(t, kind, off, 32, p.scale, x[1]);
                    }
                    const int cols = s.k_len - tile * kTile;
                    if (cols < kTile) {
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            if (c >= cols) x[c >> 5][c & 31] = -INFINITY;
                    }
                    float mt = -INFINITY;
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        float a = fmax3(x[hf][0], x[hf][1], x[hf][2]), c = fmax3(x[hf][16], x[hf][17], x[hf][18]);
#pragma unroll
                        for (int j = 3; j < 15; j += 2) {
                            a = fmax3(a, x[hf][j], x[hf][j + 1]);
                            c = fmax3(c, x[hf][16 + j], x[hf][17 + j]);
                        }
                        mt = fmax3(mt, fmaxf(a, x[hf][15]), fmaxf(c, x[hf][31]));
                    }
                    if (flat) mt = fmaf(mt, p.scale, entry);
                    const bool grow = mt > m_ref + kRescaleThreshold * kLn2;
                    if (__any_sync(0xffffffffu, grow)) {
                        float alpha = 1.f;
                        if (grow) {
                            alpha = mma_attn::fast_exp2((m_ref - mt) * kLog2e);
                            l0 *= alpha;
                            l1 *= alpha;
                            m_ref = mt;
                            neg_ref = -mt * kLog2e;
                        }
                        far = __any_sync(0xffffffffu, is_far(m_ref));
                        if (tile > 0) {   // O holds the head's products so far
                            confirm_pv(g - 1);
                            fence_after_sync();
                            if (ok) {
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    float part[16];
                                    tmem_ld16(o_lane + q * 16, part);
#pragma unroll
                                    for (int j = 0; j < 16; ++j) part[j] *= alpha;
                                    tmem_st16(o_lane + q * 16, part);
                                }
                            }
                        }
                    }
                    // A row without a finite score so far has no reference: p = 2^-inf = 0.
                    const float ref = add + neg_ref;
                    const uint64_t sc2 = f2(scale, scale), ref2 = f2(ref, ref);
                    uint64_t sum = f2(l0, l1);
                    if (__builtin_expect(far, false)) {   // (a change of x ahead of one loop for both costs 10 % of the time)
                        const float mu = m_ref == -INFINITY ? 0.f : m_ref;
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            uint32_t pk[16];
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                float a = x[hf][2 * j], c = x[hf][2 * j + 1];
                                if (flat) {
                                    a = fmaf(a, p.scale, entry);
                                    c = fmaf(c, p.scale, entry);
                                }
                                a = mma_attn::fast_exp2((a - mu) * kLog2e);
                                c = mma_attn::fast_exp2((c - mu) * kLog2e);
                                sum = f2_add(sum, f2(a, c));
                                pk[j] = Cvt<T>::pack(a, c);
                            }
                            tmem_st16_u(s_buf + hf * 16, pk);
                        }
                    } else {
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            uint32_t pk[16];
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                float a, c;
                                f2_split(f2_fma(f2(x[hf][2 * j], x[hf][2 * j + 1]), sc2, ref2), a, c);
                                a = mma_attn::fast_exp2(a);
                                c = mma_attn::fast_exp2(c);
                                sum = f2_add(sum, f2(a, c));
                                pk[j] = Cvt<T>::pack(a, c);
                            }
                            tmem_st16_u(s_buf + hf * 16, pk);
                        }
                    }
                    f2_split(sum, l0, l1);
                    tmem_wait_st();
                }
                if (tile == 0 && i > 0) finish(h0 + i - 1, g - 1, m_done, l_done);
                fence_before_sync();
                mbar_arrive(p_full(g));
            }
            m_done = m_ref;
            l_done = l0 + l1;
        }
        finish(h0 + nh - 1, g - 1, m_done, l_done);
    }
    finish_cta(&s_tmem, kTmemCols, warp, &s_fail);
}

}  // namespace bias
}  // namespace ragged
