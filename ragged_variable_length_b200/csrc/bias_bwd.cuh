// Gradients of the attention with a learned relative position bias, and the
// attention weight that each key collects, on the tensor cores (see
// bias_tc.cuh for the roles and the expanded bias table).
//
//   P = exp(s - lse),  dP = dO V^T,  delta = rowsum(dO O),  dS = P (dP - delta)
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO,  dtable = sum of dS by bucket
//
// Two kernels, so that every sum has a fixed order and no sum needs atomics:
// one with query rows (dQ, delta, the table), one with key rows (dK, dV,
// transposed scores).  Each recomputes S and dP, 7 products instead of 5.  In
// f16 a small kernel before them reads the size of V (below).
//
// delta is formed from O as it was stored, so it is off by dO . err O, which
// where V lies far from 0 is many times u of dS (values of mean 4 and 4,000
// keys: the table's gradient off by 190 u of its norm, dQ by 8, dK by 2; u is
// half a step of the type).  A row's dS add up to 0, so what they add up to is
// what delta was off by: the query kernel adds them up, hands the exact delta to
// the key kernel, and takes the difference out of the table's sums of flat
// tiles, whose probabilities it adds up too (dK 0.6 u, the table 5 u; values of
// mean 0: 0.6 and 0.4 u).  dQ keeps it: its products are done by then.  Where a
// row's keys are one tile, delta is sum P dP from the start, and nothing is off.
// The two sums cost 3 % of the gradients.
//
// Measured, both kernels and the sums: 64 sequences of 173 to 403 tokens, 12
// heads, bf16, positions with gaps: 374 us (memory and products allow 40); 2
// of 3,279 to 4,099, 8 over 2 heads, f16: 457 us (117); 4 of 79 to 197, 6
// heads, f16: 30 us.
//
// Both have eight row warps: two threads share a row, one for each half of a
// tile's 64 columns (nothing is reduced along a row but the table's sums, which
// have a column per thread).
//
// dS and P are rounded to the 16-bit type to be operands of the next product.
// In f16 they would lose what lies below 2^-14: probabilities of long rows,
// and gradients far below 1; and a large V would push dS past 65504.  Both are
// therefore scaled by powers of two, which the accumulators undo exactly: P by
// 2^14, dS by 2^(14 - e - f).  2^e is above the norm of the row's dO (dQ), or
// of every dO that a key meets (dK), 2^f above the norm of every row of V:
// |dP| and |delta| are below 2^(e + f), so |dS| stays below 2^15.
#pragma once

#include "bias_tc.cuh"

namespace ragged {
namespace bias {

constexpr int kBwdRows = 256;                   // row threads
constexpr int kBwdThreads = kBwdRows + 64;      // and the MMA and load warps
constexpr int kBwdMmaWarp = 8, kBwdLoadWarp = 9;
constexpr int kBwdQStages = 2, kBwdStages = 3;   // of the kernels below; three for the first were no faster
constexpr int kNoExp = -1000;                   // of rows that are zero, or not finite

template <typename T>
constexpr bool kScaled = std::is_same<T, __half>::value;
constexpr int kPExp = 14, kSExp = 14;

// 2^e for |e| up to 126.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// e with |x| < 2^e for a row x whose squares add up to ss.
__device__ __forceinline__ int norm_exp(float ss) { return ss > 0.f && ss < INFINITY ? (ilogbf(ss) >> 1) + 1 : kNoExp; }

// Where the table's gradient is summed up: by a launch of its own, or by CTAs
// of the key-row kernel beyond the last key tile, or beyond the last sequence.
enum TableIn { kOwnLaunch = 0, kColumn = 1, kSlice = 2 };

struct BwdArgs {
    const uint16_t* out;
    const uint16_t* dout;
    int64_t out_tok, dout_tok;
    uint16_t* dq;
    uint16_t* dk;
    uint16_t* dv;
    int64_t dq_tok, dq_head, dkv_tok, dkv_head;
    float* delta;     // [H, lse_stride]
    float* log_sum;   // [H, lse_stride]: row_log_sum of the far rows, nothing elsewhere
    int* tile_exp;    // [B][H][query tiles][4 warps]: exponent e of the rows of dO, plus f (f16)
    int* v_exp;       // [B][Hkv][key tiles]: exponent f of the rows of V (f16)
    float* partial;   // [H][num_buckets][B][query tiles]
    uint16_t* dtable;
    int q_tiles, k_tiles;
    int span, heads;  // of a launch: positions of its expanded table, heads per CTA
    // Key rows in parts (where the grid would not fill the GPU): queries of a
    // part, and the parts' fp32 sums [part][B * key rows][Hkv][dK, dV][64].
    int parts;
    int table_in;        // the key-row kernel's CTAs for the table, if any
    float* part_sums;
    int64_t part_rows;   // key rows per sequence, a multiple of 128
};

__device__ __forceinline__ uint32_t start_rows256(const uint32_t* s_tmem) {
    asm volatile("bar.sync 3, 288;" ::: "memory");
    fence_after_sync();
    return *s_tmem;
}
__device__ __forceinline__ uint32_t start_mma256(uint32_t* s_tmem, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(s_tmem)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    fence_before_sync();
    asm volatile("bar.sync 2, 64;" ::: "memory");
    asm volatile("bar.arrive 3, 288;" ::: "memory");
    fence_after_sync();
    return *s_tmem;
}
__device__ __forceinline__ void finish_cta256(const uint32_t* s_tmem, uint32_t cols, int warp, const int* s_fail) {
    fence_before_sync();
    __syncthreads();
    if (*s_fail && threadIdx.x == 0) raise_status(RAGGED_DEV_TIMEOUT);
    if (warp == kBwdMmaWarp) {
        fence_after_sync();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(*s_tmem), "r"(cols) : "memory");
    }
}
// The key-row kernel is launched while the query-row kernel still runs: its
// CTAs come up as the other's last ones leave, prepare what does not depend on
// it, and wait here for its end before they read delta, the exponents or the
// tiles' sums.  The load and MMA warps wait here as well before their first
// bounded wait for the row warps: that limit is for this kernel's own work, and
// the other kernel may run for longer.  So for the value kernel.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// 32 of a row's 64 fp32 columns at taddr, times f, rounded and stored.
template <typename T>
__device__ __forceinline__ void store_tmem_half(uint32_t taddr, float f, uint16_t* dst, bool valid) {
    float v[32];
    tmem_ld32(taddr, v);
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = Cvt<T>::pack(v[2 * i] * f, v[2 * i + 1] * f);
    if (valid) store_half_row(dst, w);
}

// p = exp(s - lse) of the 32 columns from column c of a tile (x: scores before
// scale and bias).  The negated lse in base 2 is a row's (nl) or the tile's
// columns' (neg_lse); of far ones it is the logarithm of their sum only, and
// the tile is of kFarKind, which takes off their largest scores (mu, mu_cols).
// (As a kind of tile that costs no other tile anything; a step between the bias
// and the exponentials cost 3 to 10 % of the kernels.)
template <typename T>
__device__ __forceinline__ void probabilities(const Bias16& t, const Problem& p, int kind, const int* off, int c,
                                              const float* neg_lse, float nl, const float* mu_cols, float mu, float (&x)[32]) {
    const bool flat = kind == kLeft || kind == kRight;
    const float scale = flat ? p.scale_log2 : kLog2e;
    const float add = flat ? to_float<T>(t.vec[kind == kLeft ? 0 : t.last]) * kLog2e : 0.f;
    if (!flat) bias_add<T, true>(t, kind, off, c, p.scale, x, mu_cols, mu);
    const uint64_t sc2 = f2(scale, scale), add2 = f2(add, add);
    if (neg_lse == nullptr) {
        const uint64_t c2 = f2(add + nl, add + nl);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float a, b;
            f2_split(f2_fma(f2(x[2 * i], x[2 * i + 1]), sc2, c2), a, b);
            x[2 * i] = mma_attn::fast_exp2(a);
            x[2 * i + 1] = mma_attn::fast_exp2(b);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 l = *reinterpret_cast<const float4*>(neg_lse + c + 4 * i);
            float a, b;
            f2_split(f2_fma(f2(x[4 * i], x[4 * i + 1]), sc2, f2_add(f2(l.x, l.y), add2)), a, b);
            x[4 * i] = mma_attn::fast_exp2(a);
            x[4 * i + 1] = mma_attn::fast_exp2(b);
            f2_split(f2_fma(f2(x[4 * i + 2], x[4 * i + 3]), sc2, f2_add(f2(l.z, l.w), add2)), a, b);
            x[4 * i + 2] = mma_attn::fast_exp2(a);
            x[4 * i + 3] = mma_attn::fast_exp2(b);
        }
    }
}

__device__ __forceinline__ float sum32(const float (&x)[32]) {
    uint64_t sum[4];   // chains of their own
#pragma unroll
    for (int c = 0; c < 16; ++c) sum[c & 3] = c < 4 ? f2(x[2 * c], x[2 * c + 1]) : f2_add(sum[c & 3], f2(x[2 * c], x[2 * c + 1]));
    float u, v;
    f2_split(f2_add(f2_add(sum[0], sum[1]), f2_add(sum[2], sum[3])), u, v);
    return u + v;
}

__host__ __device__ constexpr int bwd_q_fixed_bytes(int num_buckets) {
    return 1024 + kBwdQStages * 2 * kTileBytes + (num_buckets + 1) * 4 * kBwdRows + 4 * kChunk;
}
__host__ __device__ constexpr int bwd_q_smem_bytes(int D, int num_buckets, int span) {
    return bwd_q_fixed_bytes(num_buckets) + vec16_bytes(D, span) + ids_bytes(D, span);
}

// Exponent f of each tile of 128 rows of V (f16 only).  grid (key tiles, Hkv, B);
// eight threads per row.  Bound by that one read of V (2.7 us for 2 MB, 30 us
// for 190 MB), of which the next kernel finds in L2 what fits there.
template <typename T>
__global__ void __launch_bounds__(256) bias_bwd_value_kernel(const Problem p, const BwdArgs a) {
    __shared__ int s_top[8];
    let_next_start();
    const int k0 = blockIdx.x * kQTile, z = blockIdx.y, b = blockIdx.z;
    Seq s;
    if (!read_pair(p, b, s) || k0 >= s.k_len) return;
    const int r0 = k0 + (threadIdx.x >> 3), lane = threadIdx.x & 31;
    const uint16_t* src = p.v + (s.k_start + r0) * p.kv_tok + z * p.kv_head + (threadIdx.x & 7) * 8;
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = r0 + 32 * i < s.k_len ? __ldg(reinterpret_cast<const uint4*>(src + 32 * i * p.kv_tok)) : make_uint4(0, 0, 0, 0);
    int top = kNoExp;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t xs[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float x0 = to_float<T>(static_cast<uint16_t>(xs[k])), x1 = to_float<T>(static_cast<uint16_t>(xs[k] >> 16));
            ss = fmaf(x0, x0, fmaf(x1, x1, ss));
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        top = max(top, norm_exp(ss));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) s_top[threadIdx.x >> 5] = top;
    __syncthreads();
    if (threadIdx.x != 0) return;
#pragma unroll
    for (int k = 1; k < 8; ++k) top = max(top, s_top[k]);
    a.v_exp[(static_cast<int64_t>(b) * p.Hkv + z) * a.k_tiles + blockIdx.x] = top;
}
// Of every row of V of a sequence and key head, by one warp.
__device__ __forceinline__ int value_exp(const Problem& p, const BwdArgs& a, int b, int z, int k_len) {
    const int* src = a.v_exp + (static_cast<int64_t>(b) * p.Hkv + z) * a.k_tiles;
    int top = kNoExp;
    for (int i = threadIdx.x & 31; i < (k_len + kQTile - 1) / kQTile; i += 32) top = max(top, __ldcg(src + i));
    top = __reduce_max_sync(0xffffffffu, top);
    return top == kNoExp ? 0 : top;
}

// Query rows: dQ, delta, and each tile's sums for the table's gradient.  ONE:
// no sequence has more keys than a tile.
//
// The table's sums have a column of shared memory per thread, so that no two
// threads meet and the order is fixed; each element is one read-modify-write
// there, after the read of its bucket.  With all places taken a tile costs a CTA
// 3.1 us where the distances are inside the map, most of it these sums, and 1.8
// where one sum in a register serves the whole tile; a head costs 11.5 us besides,
// because its change waits for the products, sums up the table, stores dQ and
// brings Q and dO before the next head's first product: seven heads of 80 us in
// all, next to 37 tiles, for 64 sequences of 173 to 403 tokens (238 us).
// grid (query tiles, groups of heads, B), two CTAs per SM where the table is small.
//
// TMEM (256 columns): S, dP (each half replaced in place by its dS), dQ, and
// the rows of Q and dO as packed A operands: an MMA with A in TMEM takes half
// the time of one with A in shared memory, and the room goes to the table's
// sums.  S of the next tile is computed while dS of this one is, dP of the
// next one while its probabilities are.
template <typename T, bool ONE>
__global__ void __launch_bounds__(kBwdThreads, 2) bias_bwd_q_kernel(const Problem p, const BwdArgs a) {
    extern __shared__ uint8_t smem_raw[];
    // kv_full[2], kv_done[2] from 3, delta_full, qd_full, s_full, dp_full, a_full, b_full, dq_full, done
    constexpr int kBars = 13;
    __shared__ __align__(8) uint64_t s_bar[kBars];
    __shared__ uint16_t s_tab[kMaxBuckets + 1];
    __shared__ float s_delta[2][kQTile], s_norm[2][kQTile], s_undo[kQTile];
    __shared__ __align__(16) TileInfo s_tiles[kChunkTiles];
    __shared__ int s_red[16];
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;

    let_next_start();
    const int q0 = blockIdx.x * kQTile, h0 = blockIdx.y * a.heads, b = blockIdx.z;
    const int nh = min(a.heads, p.H - h0);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t item0 = (static_cast<int64_t>(b) * p.H + h0) * a.q_tiles + blockIdx.x;   // + i * q_tiles
    const int64_t sums = static_cast<int64_t>(p.B) * a.q_tiles, sum0 = static_cast<int64_t>(b) * a.q_tiles + blockIdx.x;
    Seq s;
    const bool any = read_pair(p, b, s) && q0 < s.q_len;
    if (kScaled<T> && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) wait_for_last();   // never ends before the value kernel
    if (!any || s.k_len == 0) {   // nothing for the table; queries without keys get no gradient
        for (int i = tid; i < nh * p.num_buckets; i += kBwdThreads) a.partial[(h0 * p.num_buckets + i) * sums + sum0] = 0.f;
        if (any)
            for (int i = tid; i < nh * kQTile; i += kBwdThreads) {
                const int r = q0 + i % kQTile;
                const uint32_t zero[32] = {};
                if (r < s.q_len) store_row(a.dq + static_cast<int64_t>(s.q_start + r) * a.dq_tok + (h0 + i / kQTile) * a.dq_head, zero);
            }
        return;
    }
    const int nt = (s.k_len + kTile - 1) / kTile;

    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t sRing = (raw + 1023u) & ~1023u;   // stage: K, then V
    float* acc = reinterpret_cast<float*>(smem_raw + (sRing - raw) + kBwdQStages * 2 * kTileBytes);   // [buckets + 1][256]
    auto stage = [&](uint32_t g) { return sRing + (g % kBwdQStages) * 2 * kTileBytes; };
    const uint32_t bar0 = smem_addr(&s_bar[0]);
    auto kv_full = [&](uint32_t g) { return bar0 + 8u * (g % kBwdQStages); };
    auto kv_done = [&](uint32_t g) { return bar0 + 8u * (3 + g % kBwdQStages); };
    const uint32_t delta_full = bar0 + 40, qd_full = bar0 + 48, s_full = bar0 + 56, dp_full = bar0 + 64, a_full = bar0 + 72, b_full = bar0 + 80, dq_full = bar0 + 88, done = bar0 + 96;
    constexpr uint32_t dp_col = kTile, dq_col = 2 * kTile, q_col = 3 * kTile, do_col = 3 * kTile + 32;
    const Wait wait{&s_fail};

    if (warp == kBwdLoadWarp) {
        if (lane < kBars) mbar_init(bar0 + 8 * lane, lane < 3 ? 32 : lane == 5 || lane == 6 || lane == 9 || lane == 10 ? kBwdRows : 1);
        if (lane == 0) s_fail = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        __syncwarp();
        start_loads();
        bool ok = !test_hook(1);
        uint32_t g = 0;
        for (int i = 0; ok && i < nh; ++i) {
            const int64_t z = static_cast<int64_t>((h0 + i) / p.group) * p.kv_head;
            const uint16_t* kb = p.k + s.k_start * p.kv_tok + z;
            const uint16_t* vb = p.v + s.k_start * p.kv_tok + z;
            for (int t = 0; t < nt; ++t, ++g) {
                if (kScaled<T> && g == kBwdQStages) wait_for_last();
                if (g >= kBwdQStages) ok = wait.warp(kv_done(g), (g / kBwdQStages - 1) & 1);
                if (!ok) break;
                load_rows<kTile>(stage(g), kb, p.kv_tok, t * kTile, s.k_len, lane);
                load_rows<kTile>(stage(g) + kTileBytes, vb, p.kv_tok, t * kTile, s.k_len, lane);
                cp_async_arrive_noinc(kv_full(g));
            }
        }
        cp_async_wait_all();
    } else if (warp == kBwdMmaWarp) {
        const uint32_t tmem = start_mma256(&s_tmem, kTmemCols);
        if (lane == 0) {
            const uint32_t idesc_s = make_idesc(Cvt<T>::kFormat, 0, kTile), idesc_g = make_idesc(Cvt<T>::kFormat, 1, 64);
            auto product = [&](uint32_t col, uint32_t from, uint32_t sb) {   // [128, 64] = A B^T over the head dimension
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_f16_ts(tmem + col, tmem + from + ks * 8, make_sdesc(sb + ks * 32), idesc_s, ks > 0);
            };
            bool ok = true;
            uint32_t g = 0;
            for (int i = 0; ok && i < nh; ++i) {
                ok = wait(qd_full, i & 1) && wait(kv_full(g), (g / kBwdQStages) & 1);
                if (!ok) break;
                fence_async_smem();
                fence_after_sync();
                product(0, q_col, stage(g));
                mma_commit(s_full);
                product(dp_col, do_col, stage(g) + kTileBytes);
                mma_commit(dp_full);
                if (kScaled<T> && i == 0) wait_for_last();
                for (int t = 0; t < nt; ++t, ++g) {
                    const bool more = t + 1 < nt;
                    if (more) {
                        ok = wait(kv_full(g + 1), ((g + 1) / kBwdQStages) & 1);
                        if (!ok) break;
                        fence_async_smem();
                    }
                    ok = wait(a_full, g & 1);   // S has been read
                    if (!ok) break;
                    if (more) {
                        fence_after_sync();
                        product(0, q_col, stage(g + 1));
                        mma_commit(s_full);
                    }
                    ok = wait(b_full, g & 1);   // dS is there
                    if (!ok) break;
                    fence_after_sync();
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)   // dS of columns 0-31 at dP + 0, of 32-63 at dP + 32
                        mma_f16_ts(tmem + dq_col, tmem + dp_col + (ks >> 1) * 32 + (ks & 1) * 8, make_sdesc(stage(g) + ks * 2048), idesc_g,
                                   (t > 0 || ks > 0) ? 1u : 0u);
                    mma_commit(kv_done(g));
                    if (more) {
                        product(dp_col, do_col, stage(g + 1) + kTileBytes);
                        mma_commit(dp_full);
                    } else {
                        mma_commit(dq_full);
                    }
                }
            }
            mma_commit(done);
            mbar_wait(done, 0);
        }
        __syncwarp();
    } else {
        const int half = warp >> 2, r = tid & 127, row = q0 + r;
        const bool valid = row < s.q_len, warp_rows = q0 + (warp & 3) * 32 < s.q_len;
        const int64_t t_row = s.q_start + (valid ? row : 0);
        Bias16 t;
        uint8_t* extra = reinterpret_cast<uint8_t*>(acc + (p.num_buckets + 1) * kBwdRows);
        t.vec = reinterpret_cast<uint16_t*>(extra);
        uint8_t* ids = extra + vec16_bytes(p.D, a.span);
        t.off = reinterpret_cast<int*>(ids + ids_bytes(p.D, a.span));
        t.tiles = s_tiles;
        uint8_t* map = ids + ((vec_entries(p.D, a.span) + 15) & ~15);
        const bool has_entry = tid < p.num_buckets;
        const uint16_t* column = p.table + static_cast<int64_t>(has_entry ? tid : 0) * p.H + h0;
        // What the set-up needs of global memory, all under way at once.
        uint16_t entry = __ldg(column);
        const int pos = valid ? query_pos(p, s, row) : 0;
        auto key_at = [&](int c) { return key_pos(p, s, c); };
        Columns<kBwdRows> cols;
        cols.load(0, s.k_len, key_at);
        // This thread's halves of a head's rows of Q, dO and O, and the row's lse.
        uint4 qw[4], dw[4], ow[4];
        float lse = -INFINITY;
        auto load_row = [&](int h) {
            const uint4* qp = reinterpret_cast<const uint4*>(p.q + t_row * p.q_tok + h * p.q_head) + half * 4;
            const uint4* dp = reinterpret_cast<const uint4*>(a.dout + t_row * a.dout_tok + h * 64) + half * 4;
            const uint4* op = reinterpret_cast<const uint4*>(a.out + t_row * a.out_tok + h * 64) + half * 4;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                qw[c] = valid ? __ldg(qp + c) : make_uint4(0, 0, 0, 0);
                dw[c] = valid ? __ldg(dp + c) : make_uint4(0, 0, 0, 0);
                if constexpr (!ONE) ow[c] = valid ? __ldg(op + c) : make_uint4(0, 0, 0, 0);
            }
            if (valid) lse = p.lse[h * p.lse_stride + t_row];
        };
        load_row(h0);
        bias_map<kBwdRows>(p, map, p.num_buckets);
        if (has_entry) s_tab[tid] = entry;
        if (tid == p.num_buckets) s_tab[tid] = 0;
        for (int n = 0; n <= p.num_buckets; ++n) acc[n * kBwdRows + tid] = 0.f;
        bias_rows<kBwdRows>(t, p, pos, valid, a.span, s_red);
        bias_ids<1, kBwdRows>(t, map, ids, p.num_buckets);
        cols.store(t, 0, s.k_len);
        rows_barrier<kBwdRows>();
        const uint32_t tmem = start_rows256(&s_tmem);
        const uint32_t t_lane = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        char* acc_row = reinterpret_cast<char*>(acc + tid);
        const uint8_t* id_row = ids + (t.row >> 1);
        bool ok = true;
        uint32_t g = 0;
        float undo = 1.f, delta = 0.f, far_left = 0.f, far_right = 0.f, p_left = 0.f, p_right = 0.f, near_sum = 0.f;
        // From head i to the next: the table's sums of head i, its dQ once its last product has
        // finished, and the next head's bias and rows.
        auto change = [&](int i, bool more) {
            if (i >= 0) {
                if (more) {
                    load_row(h0 + i + 1);
                    if (has_entry) entry = __ldg(column + i + 1);
                }
                if constexpr (!ONE) {   // what delta was short of: dS of a row adds up to 0
                    if (nt == 1) rows_barrier<kBwdRows>();   // the deltas have been read (else some tile's products waited for that)
                    s_delta[half][r] = far_left + far_right + near_sum;
                    rows_barrier<kBwdRows>();
                    const float sum = s_delta[0][r] + s_delta[1][r];
                    if (p_left != 0.f) far_left = fmaf(-sum, p_left, far_left);   // (a row's NaN keeps to the buckets of its pairs)
                    if (p_right != 0.f) far_right = fmaf(-sum, p_right, far_right);
                    delta = fmaf(sum, undo, delta);
                }
                if (half == 0 && valid) a.delta[(h0 + i) * p.lse_stride + t_row] = delta;
                *reinterpret_cast<float*>(acc_row + ids[0] * (4 * kBwdRows)) += far_left;
                *reinterpret_cast<float*>(acc_row + ids[t.last] * (4 * kBwdRows)) += far_right;
                if (half == 0) s_undo[r] = valid ? undo : 0.f;
                if (more && has_entry) s_tab[tid] = entry;
                rows_barrier<kBwdRows>();   // sums complete, the last head's entries no longer read
                for (int n = warp; n < p.num_buckets; n += 8) {   // each thread's sums, unscaled, in a fixed order
                    float sum = 0.f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int u = lane + 32 * k;
                        sum += q0 + (u & 127) < s.q_len ? acc[n * kBwdRows + u] * s_undo[u & 127] : 0.f;
                        acc[n * kBwdRows + u] = 0.f;
                    }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    if (lane == 0) a.partial[((h0 + i) * p.num_buckets + n) * sums + sum0] = sum;
                }
            }
            if (more) bias_fill<kBwdRows>(t, ids, s_tab);
            if (i >= 0) {
                ok = ok && wait.warp(dq_full, i & 1);
                if (ok && warp_rows) {
                    fence_after_sync();
                    store_tmem_half<T>(t_lane + dq_col + half * 32, p.scale * undo, a.dq + t_row * a.dq_tok + (h0 + i) * a.dq_head + half * 32, valid);
                }
            }
            if (!more) return;
            // Q and dO to TMEM: every product of the head before has finished.
            uint32_t w[16];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                w[4 * c] = qw[c].x;
                w[4 * c + 1] = qw[c].y;
                w[4 * c + 2] = qw[c].z;
                w[4 * c + 3] = qw[c].w;
            }
            tmem_st16_u(t_lane + q_col + half * 16, w);
            float d = 0.f, ss = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t ys[4] = {dw[c].x, dw[c].y, dw[c].z, dw[c].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    w[4 * c + k] = ys[k];
                    const float d0 = to_float<T>(static_cast<uint16_t>(ys[k])), d1 = to_float<T>(static_cast<uint16_t>(ys[k] >> 16));
                    if constexpr (!ONE) {
                        const uint32_t xs[4] = {ow[c].x, ow[c].y, ow[c].z, ow[c].w};
                        d = fmaf(to_float<T>(static_cast<uint16_t>(xs[k])), d0, d);
                        d = fmaf(to_float<T>(static_cast<uint16_t>(xs[k] >> 16)), d1, d);
                    }
                    if constexpr (kScaled<T>) ss = fmaf(d0, d0, fmaf(d1, d1, ss));
                }
            }
            tmem_st16_u(t_lane + do_col + half * 16, w);
            tmem_wait_st();
            fence_before_sync();
            mbar_arrive(qd_full);
            if constexpr (!ONE) s_delta[half][r] = d;
            if constexpr (kScaled<T>) s_norm[half][r] = ss;
            rows_barrier<kBwdRows>();   // entries, deltas and cleared sums are there
        };
        change(-1, true);
        if constexpr (kScaled<T>) wait_for_last();   // the value kernel's exponents
        for (int i = 0; i < nh; ++i) {
            const int h = h0 + i;
            if constexpr (!ONE) delta = s_delta[0][r] + s_delta[1][r];
            float rs = 1.f;   // dS is kept times rs
            undo = 1.f;
            if constexpr (kScaled<T>) {
                int e = norm_exp(s_norm[0][r] + s_norm[1][r]);
                const int f = value_exp(p, a, b, h / p.group, s.k_len);
                if (e != kNoExp) {
                    e += f;
                    rs = pow2(kSExp - e);
                    undo = pow2(e - kSExp);
                }
                const int top = __reduce_max_sync(0xffffffffu, e);
                if (half == 0 && lane == 0) a.tile_exp[(item0 + static_cast<int64_t>(i) * a.q_tiles) * 4 + warp] = top;
            }
            float nl = valid ? -lse_log2(lse) : -INFINITY, mu = 0.f;
            uint32_t todo = __ballot_sync(0xffffffffu, valid && is_far(lse));
            const bool far = todo != 0;
            for (; todo != 0; todo &= todo - 1) {
                const int src = __ffs(todo) - 1;
                const float ls = row_log_sum<T>(p, s, q0 + (warp & 3) * 32 + src, h);
                if (lane == src) {
                    mu = lse - ls;
                    nl = -ls * kLog2e;
                    if (half == 0) a.log_sum[h * p.lse_stride + t_row] = ls;
                }
            }
            const uint64_t r2 = f2(rs, rs);
            uint64_t nd2 = f2(-delta * rs, -delta * rs);
            far_left = far_right = p_left = p_right = near_sum = 0.f;
            for (int tile = 0; tile < nt; ++tile, ++g) {
                if (tile % kChunkTiles == 0 && (tile > 0 || (i > 0 && nt > kChunkTiles))) {
                    cols.load(tile * kTile, s.k_len, key_at);
                    if (tile > 0) rows_barrier<kBwdRows>();
                    cols.store(t, tile * kTile, s.k_len);
                    rows_barrier<kBwdRows>();
                }
                const int kind = far ? kFarKind : tile_kind(t, tile % kChunkTiles);
                const int* off = t.off + (tile % kChunkTiles) * kTile;
                const int left = s.k_len - tile * kTile - half * 32;   // columns of this half
                float x[32];
                ok = ok && wait.warp(s_full, g & 1);
                if (ok && warp_rows) {
                    fence_after_sync();
                    tmem_ld32(t_lane + half * 32, x);
                }
                fence_before_sync();
                mbar_arrive(a_full);
                if (ok && warp_rows) {
                    probabilities<T>(t, p, kind, off, half * 32, nullptr, nl, nullptr, mu, x);
                    if (left < 32) {
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (c >= left) x[c] = 0.f;
                    }
                    if constexpr (!ONE) {
                        if (kind == kLeft) p_left += sum32(x);
                        else if (kind == kRight) p_right += sum32(x);
                    }
                }
                ok = ok && wait.warp(dp_full, g & 1);
                if constexpr (ONE) {   // the whole row is here: delta = sum P dP
                    float sum = 0.f;
                    if (ok && warp_rows) {
                        fence_after_sync();
                        float y[32];
                        tmem_ld32(t_lane + dp_col + half * 32, y);
                        uint64_t two = f2(0.f, 0.f);
#pragma unroll
                        for (int c = 0; c < 16; ++c) two = f2_fma(f2(x[2 * c], x[2 * c + 1]), f2(y[2 * c], y[2 * c + 1]), two);
                        float u, v;
                        f2_split(two, u, v);
                        sum = u + v;
                    }
                    s_delta[half][r] = sum;
                    mbar_arrive(delta_full);
                    ok = ok && wait.warp(delta_full, i & 1);
                    delta = s_delta[0][r] + s_delta[1][r];
                    nd2 = f2(-delta * rs, -delta * rs);
                }
                if (ok && warp_rows) {
                    fence_after_sync();
                    float y[32];
                    tmem_ld32(t_lane + dp_col + half * 32, y);
                    uint32_t w[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        f2_split(f2_mul(f2(x[2 * c], x[2 * c + 1]), f2_fma(f2(y[2 * c], y[2 * c + 1]), r2, nd2)), x[2 * c], x[2 * c + 1]);
                        w[c] = Cvt<T>::pack(x[2 * c], x[2 * c + 1]);
                    }
                    tmem_st16_u(t_lane + dp_col + half * 32, w);
                    tmem_wait_st();
                }
                fence_before_sync();
                mbar_arrive(b_full);
                if (ok && warp_rows) {   // the table's share, behind the hand-over
                    const float sum = sum32(x);
                    if (kind == kLeft) {
                        far_left += sum;
                    } else if (kind == kRight) {
                        far_right += sum;
                    } else {
                        near_sum += sum;
                        // Addresses first: a load of the next one could not pass a store to the sums.
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            if (left <= q * 16) break;   // no columns left
                            uint32_t at[16];
                            if (kind == kConsecutive) {
                                const uint8_t* id = id_row + (off[0] >> 1) + half * 32 + q * 16;
#pragma unroll
                                for (int c = 0; c < 16; ++c) at[c] = id[c];
                            } else if (kind == kGeneral || (kind == kFarKind && t.near)) {
#pragma unroll
                                for (int c = 0; c < 4; ++c) {
                                    const int4 o = *reinterpret_cast<const int4*>(off + half * 32 + q * 16 + 4 * c);
                                    at[4 * c] = id_row[o.x >> 1];
                                    at[4 * c + 1] = id_row[o.y >> 1];
                                    at[4 * c + 2] = id_row[o.z >> 1];
                                    at[4 * c + 3] = id_row[o.w >> 1];
                                }
                            } else {
#pragma unroll
                                for (int c = 0; c < 16; ++c) at[c] = ids[max(-t.D, min(t.D, pos_diff(off[half * 32 + q * 16 + c], t.p_row))) + t.D];
                            }
#pragma unroll
                            for (int c = 0; c < 16; ++c) *reinterpret_cast<float*>(acc_row + at[c] * (4 * kBwdRows)) += x[q * 16 + c];
                        }
                    }
                }
            }
            change(i, i + 1 < nh);
        }
    }
    finish_cta256(&s_tmem, kTmemCols, warp, &s_fail);
}

__host__ __device__ constexpr int bwd_kv_fixed_bytes() { return 1024 + 2 * kRowBytes + kBwdStages * 2 * kTileBytes + 16 * kChunk; }
__host__ __device__ constexpr int bwd_kv_smem_bytes(int D, int span) {
    return bwd_kv_fixed_bytes() + vec16_bytes(D, span) + ids_bytes(D, span);
}

// dtable[n, h] = sum of the tiles' sums, in a fixed order: entries id, id + n_ids,
// ... by the CTA's warps.
template <typename T>
__device__ __forceinline__ void table_gradient(const Problem& p, const BwdArgs& a, int id, int n_ids) {
    const int lane = threadIdx.x & 31, warps = blockDim.x / 32, n = p.B * a.q_tiles, all = p.num_buckets * p.H;
    for (int e = id * warps + (threadIdx.x >> 5); e < all; e += n_ids * warps) {
        const float* src = a.partial + static_cast<int64_t>(e) * n;
        float x = 0.f;
#pragma unroll 4
        for (int i = lane; i < n; i += 32) x += __ldcg(src + i);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        const int h = e / p.num_buckets;
        if (lane == 0) a.dtable[static_cast<int64_t>(e - h * p.num_buckets) * p.H + h] = from_float<T>(x);
    }
}
template <typename T>
__global__ void __launch_bounds__(256) bias_bwd_table_kernel(const Problem p, const BwdArgs a) {
    table_gradient<T>(p, a, blockIdx.x, gridDim.x);
}

// Key rows: dK and dV, over the query tiles of every query head of a key head.
// grid (key tiles * parts, groups of key heads, B), two CTAs per SM, and a
// column or a slice of CTAs that sums up the table's gradient.
//
// TMEM (256 columns): S^T and dP^T (each half replaced in place by its P^T,
// dS^T), dK and dV.  Bound by the row warps' instructions, as the forward pass.
// A table column of shared memory less, so three stages of Q and dO fit.
template <typename T>
__global__ void __launch_bounds__(kBwdThreads, 2) bias_bwd_kv_kernel(const Problem p, const BwdArgs a) {
    extern __shared__ uint8_t smem_raw[];
    // kv_full, kv_empty, q_full[3], q_done[3], s_full, dp_full, a_full, b_full, acc_full, done
    constexpr int kBars = 14;
    __shared__ __align__(8) uint64_t s_bar[kBars];
    __shared__ uint16_t s_tab[kMaxBuckets + 1];
    __shared__ __align__(16) TileInfo s_tiles[kChunkTiles];
    __shared__ int s_red[16];
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;

    // One column, or one slice, of CTAs more: the table's gradient.
    if (a.table_in == kColumn ? blockIdx.x == gridDim.x - 1 : a.table_in == kSlice && blockIdx.z == gridDim.z - 1) {
        wait_for_last();
        const int other = a.table_in == kSlice ? blockIdx.x : blockIdx.z, others = a.table_in == kSlice ? gridDim.x : gridDim.z;
        table_gradient<T>(p, a, blockIdx.y + gridDim.y * other, gridDim.y * others);
        return;
    }
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) wait_for_last();   // this grid never ends before the other
    const int part = blockIdx.x % a.parts, k0 = (blockIdx.x / a.parts) * kQTile, z0 = blockIdx.y * a.heads, b = blockIdx.z;
    const int nz = min(a.heads, p.Hkv - z0);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Seq s;
    if (!read_pair(p, b, s) || k0 >= s.k_len) return;
    if (s.q_len == 0) {   // keys without queries
        if (part == 0)
            for (int i = tid; i < nz * kQTile; i += kBwdThreads) {
                const int r = k0 + i % kQTile;
                if (r >= s.k_len) continue;
                const uint32_t zero[32] = {};
                const int64_t at = static_cast<int64_t>(s.k_start + r) * a.dkv_tok + (z0 + i / kQTile) * a.dkv_head;
                store_row(a.dk + at, zero);
                store_row(a.dv + at, zero);
            }
        return;
    }
    // This part's query tiles [t0, t1) of every head; a part without any still writes zeros.
    const int nt_all = (s.q_len + kTile - 1) / kTile, per = (nt_all + a.parts - 1) / a.parts;
    const int t0 = min(nt_all, part * per), t1 = min(nt_all, t0 + per), nt = t1 - t0;

    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t sK = (raw + 1023u) & ~1023u;
    const uint32_t sV = sK + kRowBytes, sRing = sV + kRowBytes;   // stage: Q, then dO
    uint8_t* extra = smem_raw + (sRing - raw) + kBwdStages * 2 * kTileBytes;
    auto stage = [&](uint32_t g) { return sRing + (g % kBwdStages) * 2 * kTileBytes; };
    const uint32_t bar0 = smem_addr(&s_bar[0]);
    const uint32_t kv_full = bar0, kv_empty = bar0 + 8, s_full = bar0 + 64, dp_full = bar0 + 72, a_full = bar0 + 80, b_full = bar0 + 88, acc_full = bar0 + 96, done = bar0 + 104;
    auto q_full = [&](uint32_t g) { return bar0 + 8u * (2 + g % kBwdStages); };
    auto q_done = [&](uint32_t g) { return bar0 + 8u * (5 + g % kBwdStages); };
    constexpr uint32_t dp_col = kTile, dk_col = 2 * kTile, dv_col = 3 * kTile;
    const Wait wait{&s_fail};
    const uint32_t per_head = static_cast<uint32_t>(nt) * p.group;   // tiles of a key head

    if (warp == kBwdLoadWarp) {
        if (lane < kBars) mbar_init(bar0 + 8 * lane, lane == 0 || (lane >= 2 && lane < 5) ? 32 : lane == 10 || lane == 11 ? kBwdRows : 1);
        if (lane == 0) s_fail = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        __syncwarp();
        start_loads();
        bool ok = !test_hook(1);
        uint32_t g = 0;
        for (int i = 0; ok && i < nz && nt > 0; ++i) {
            const int z = z0 + i;
            if (i == 1) wait_for_last();
            if (i > 0) ok = wait.warp(kv_empty, (i - 1) & 1);
            if (!ok) break;
            const int64_t at = s.k_start * p.kv_tok + z * p.kv_head;
            load_rows<kQTile>(sK, p.k + at, p.kv_tok, k0, s.k_len, lane);
            load_rows<kQTile>(sV, p.v + at, p.kv_tok, k0, s.k_len, lane);
            cp_async_arrive_noinc(kv_full);
            for (int h = z * p.group; ok && h < (z + 1) * p.group; ++h) {
                const uint16_t* qb = p.q + s.q_start * p.q_tok + h * p.q_head;
                const uint16_t* db = a.dout + s.q_start * a.dout_tok + h * 64;
                for (int t = t0; t < t1; ++t, ++g) {
                    if (g == kBwdStages) wait_for_last();
                    if (g >= kBwdStages) ok = wait.warp(q_done(g), (g / kBwdStages - 1) & 1);
                    if (!ok) break;
                    load_rows<kTile>(stage(g), qb, p.q_tok, t * kTile, s.q_len, lane);
                    load_rows<kTile>(stage(g) + kTileBytes, db, a.dout_tok, t * kTile, s.q_len, lane);
                    cp_async_arrive_noinc(q_full(g));
                }
            }
        }
        cp_async_wait_all();
    } else if (warp == kBwdMmaWarp) {
        const uint32_t tmem = start_mma256(&s_tmem, kTmemCols);
        if (lane == 0) {
            const uint32_t idesc_s = make_idesc(Cvt<T>::kFormat, 0, kTile), idesc_g = make_idesc(Cvt<T>::kFormat, 1, 64);
            auto product = [&](uint32_t col, uint32_t sa, uint32_t sb) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_f16(tmem + col, make_sdesc(sa + ks * 32), make_sdesc(sb + ks * 32), idesc_s, ks > 0);
            };
            auto gradient = [&](uint32_t col, uint32_t from, uint32_t sb, bool first) {   // += A (TMEM, two halves) B
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_f16_ts(tmem + col, tmem + from + (ks >> 1) * 32 + (ks & 1) * 8, make_sdesc(sb + ks * 2048), idesc_g, (!first || ks > 0) ? 1u : 0u);
            };
            bool ok = true;
            uint32_t g = 0;
            for (int i = 0; ok && i < nz && nt > 0; ++i) {
                ok = wait(kv_full, i & 1) && wait(q_full(g), (g / kBwdStages) & 1);
                if (!ok) break;
                fence_async_smem();
                fence_after_sync();
                product(0, sK, stage(g));
                mma_commit(s_full);
                product(dp_col, sV, stage(g) + kTileBytes);
                mma_commit(dp_full);
                if (per_head == 1) mma_commit(kv_empty);   // the head's last product with K and V
                if (i == 0) wait_for_last();
                for (uint32_t n = 0; n < per_head; ++n, ++g) {
                    const bool more = n + 1 < per_head;
                    if (more) {
                        ok = wait(q_full(g + 1), ((g + 1) / kBwdStages) & 1);
                        if (!ok) break;
                        fence_async_smem();
                    }
                    ok = wait(a_full, g & 1);   // P^T is there
                    if (!ok) break;
                    fence_after_sync();
                    gradient(dv_col, 0, stage(g) + kTileBytes, n == 0);
                    if (more) {
                        product(0, sK, stage(g + 1));
                        mma_commit(s_full);
                    }
                    ok = wait(b_full, g & 1);   // dS^T is there
                    if (!ok) break;
                    fence_after_sync();
                    gradient(dk_col, dp_col, stage(g), n == 0);
                    mma_commit(q_done(g));
                    if (more) {
                        product(dp_col, sV, stage(g + 1) + kTileBytes);
                        mma_commit(dp_full);
                        if (n + 2 == per_head) mma_commit(kv_empty);
                    } else {
                        mma_commit(acc_full);
                    }
                }
            }
            mma_commit(done);
            mbar_wait(done, 0);
        }
        __syncwarp();
    } else {
        const int half = warp >> 2, r = tid & 127, row = k0 + r;
        const bool valid = row < s.k_len, warp_rows = k0 + (warp & 3) * 32 < s.k_len;
        const int64_t t_row = s.k_start + (valid ? row : 0);
        Bias16 t;
        t.vec = reinterpret_cast<uint16_t*>(extra);
        uint8_t* ids = extra + vec16_bytes(p.D, a.span);
        t.off = reinterpret_cast<int*>(ids + ids_bytes(p.D, a.span));
        float* s_lse = reinterpret_cast<float*>(t.off + kChunk);   // negated
        float* s_delta = s_lse + kChunk;
        float* s_mu = s_delta + kChunk;
        t.tiles = s_tiles;
        uint8_t* map = ids + ((vec_entries(p.D, a.span) + 15) & ~15);
        const bool has_entry = tid < p.num_buckets;
        const uint16_t* column = p.table + static_cast<int64_t>(has_entry ? tid : 0) * p.H;
        // What the set-up needs of global memory, all under way at once.
        const uint16_t entry = __ldg(column + z0 * p.group);
        const int pos = valid ? key_pos(p, s, row) : 0;
        auto query_at = [&](int c) { return query_pos(p, s, c); };
        Columns<kBwdRows> cols;
        cols.load(t0 * kTile, s.q_len, query_at);
        bias_map<kBwdRows>(p, map, p.num_buckets);
        if (has_entry) s_tab[tid] = entry;
        if (tid == p.num_buckets) s_tab[tid] = 0;
        bias_rows<kBwdRows>(t, p, pos, valid, a.span, s_red);
        bias_ids<-1, kBwdRows>(t, map, ids, p.num_buckets);
        cols.store<true>(t, t0 * kTile, s.q_len);
        const uint32_t tmem = start_rows256(&s_tmem);
        const uint32_t t_lane = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        wait_for_last();   // delta and the exponents
        bool ok = true;
        uint32_t g = 0;
        const float shift = kScaled<T> ? static_cast<float>(kPExp) : 0.f;
        // dK and dV of key head z0 + i, half of the columns each (fp32 where the parts are summed up).
        auto finish = [&](int i, int e) {
            if (nt > 0) ok = ok && wait.warp(acc_full, i & 1);
            if (!ok || !warp_rows) return;
            fence_after_sync();
            const float fk = kScaled<T> ? p.scale * pow2(e - kSExp) : p.scale, fv = kScaled<T> ? pow2(-kPExp) : 1.f;
            const int z = z0 + i;
            if (a.parts == 1) {
                const int64_t at = t_row * a.dkv_tok + z * a.dkv_head + half * 32;
                store_tmem_half<T>(t_lane + dk_col + half * 32, fk, a.dk + at, valid);
                store_tmem_half<T>(t_lane + dv_col + half * 32, fv, a.dv + at, valid);
                return;
            }
            float* dst = a.part_sums + (((static_cast<int64_t>(part) * p.B + b) * a.part_rows + row) * p.Hkv + z) * 128 + half * 32;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                float v[32];
                if (nt > 0) tmem_ld32(t_lane + (m ? dv_col : dk_col) + half * 32, v);
                const float f = m ? fv : fk;
                if (valid)
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        reinterpret_cast<float4*>(dst + m * 64)[c] =
                            nt > 0 ? make_float4(v[4 * c] * f, v[4 * c + 1] * f, v[4 * c + 2] * f, v[4 * c + 3] * f) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        };
        int e_done = 0;
        for (int i = 0; i < nz; ++i) {
            const int z = z0 + i;
            // One scale for everything that a key sums: the largest |dO| of its queries.
            int e = 0;
            if constexpr (kScaled<T>) {
                int top = kNoExp;
                const int n = (s.q_len + kQTile - 1) / kQTile * 4;   // warps of queries per head
                for (int k = tid; k < n * p.group; k += kBwdRows) {
                    const int hh = k / n;
                    top = max(top, a.tile_exp[(static_cast<int64_t>(b) * p.H + z * p.group + hh) * a.q_tiles * 4 + (k - hh * n)]);
                }
                top = __reduce_max_sync(0xffffffffu, top);
                rows_barrier<kBwdRows>();   // s_red's last values are no longer read
                if (lane == 0) s_red[warp] = top;
                rows_barrier<kBwdRows>();
#pragma unroll
                for (int k = 0; k < 8; ++k) top = max(top, s_red[k]);
                e = top == kNoExp ? 0 : top;
            }
            const float rs = kScaled<T> ? pow2(kSExp - e - kPExp) : 1.f;
            const uint64_t r2 = f2(rs, rs);
            bool first = i > 0;   // the head before is finished when this one's first P is ready
            for (int h = z * p.group; h < (z + 1) * p.group; ++h) {
                const float* lse = p.lse + h * p.lse_stride + s.q_start;
                const float* delta = a.delta + h * p.lse_stride + s.q_start;
                // lse and delta of the first columns are on their way under the barriers and the fill.
                float l_next[kChunk / kBwdRows], d_next[kChunk / kBwdRows];
                auto load_stats = [&](int c0) {
#pragma unroll
                    for (int k = 0; k < kChunk / kBwdRows; ++k) {
                        const int c = c0 + tid + k * kBwdRows;
                        l_next[k] = c < s.q_len ? lse[c] : 0.f;
                        d_next[k] = c < s.q_len ? delta[c] : 0.f;
                    }
                };
                auto store_stats = [&](int c0) {   // whether one of them is far
                    bool any = false;
#pragma unroll
                    for (int k = 0; k < kChunk / kBwdRows; ++k) {
                        const int c = tid + k * kBwdRows;
                        const bool in = c0 + c < s.q_len, far = in && is_far(l_next[k]);   // no such query: p = 0
                        const float ls = far ? a.log_sum[h * p.lse_stride + s.q_start + c0 + c] : 0.f;
                        s_lse[c] = !in ? -INFINITY : shift - (far ? ls * kLog2e : lse_log2(l_next[k]));
                        s_mu[c] = far ? l_next[k] - ls : 0.f;
                        s_delta[c] = in ? -d_next[k] * rs : 0.f;
                        any |= far;
                    }
                    return any;
                };
                load_stats(t0 * kTile);
                const bool start = h == z0 * p.group;   // the first head's entries are in s_tab, its columns stored
                const uint16_t next = start ? uint16_t(0) : __ldg(column + h);
                rows_barrier<kBwdRows>();   // the last head's entries and columns are no longer read
                if (!start) {
                    if (has_entry) s_tab[tid] = next;
                    rows_barrier<kBwdRows>();
                }
                bias_fill<kBwdRows>(t, ids, s_tab);
                bool far = false;
                for (int tile = 0; tile < nt; ++tile, ++g) {
                    if (tile % kChunkTiles == 0) {
                        const int c0 = (t0 + tile) * kTile;
                        const bool again = nt > kChunkTiles && (tile > 0 || !start);
                        if (tile > 0) load_stats(c0);
                        if (again) cols.load(c0, s.q_len, query_at);
                        if (tile > 0) rows_barrier<kBwdRows>();
                        if (again) cols.store<true>(t, c0, s.q_len);
                        far = rows_any<kBwdRows>(store_stats(c0));
                    }
                    const int kind = far ? kFarKind : tile_kind(t, tile % kChunkTiles), c0 = (tile % kChunkTiles) * kTile;
                    float x[32];
                    ok = ok && wait.warp(s_full, g & 1);
                    if (ok && warp_rows) {
                        fence_after_sync();
                        tmem_ld32(t_lane + half * 32, x);
                        probabilities<T>(t, p, kind, t.off + c0, half * 32, s_lse + c0, 0.f, s_mu + c0, 0.f, x);
                        uint32_t w[16];
#pragma unroll
                        for (int c = 0; c < 16; ++c) w[c] = Cvt<T>::pack(x[2 * c], x[2 * c + 1]);
                        tmem_st16_u(t_lane + half * 32, w);
                        tmem_wait_st();
                    }
                    if (first) {
                        finish(i - 1, e_done);
                        first = false;
                    }
                    fence_before_sync();
                    mbar_arrive(a_full);
                    ok = ok && wait.warp(dp_full, g & 1);
                    if (ok && warp_rows) {
                        fence_after_sync();
                        float y[32];
                        tmem_ld32(t_lane + dp_col + half * 32, y);
                        uint32_t w[16];
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const float4 d = *reinterpret_cast<const float4*>(s_delta + c0 + half * 32 + 4 * c);
                            float u, v;
                            f2_split(f2_mul(f2(x[4 * c], x[4 * c + 1]), f2_fma(f2(y[4 * c], y[4 * c + 1]), r2, f2(d.x, d.y))), u, v);
                            w[2 * c] = Cvt<T>::pack(u, v);
                            f2_split(f2_mul(f2(x[4 * c + 2], x[4 * c + 3]), f2_fma(f2(y[4 * c + 2], y[4 * c + 3]), r2, f2(d.z, d.w))), u, v);
                            w[2 * c + 1] = Cvt<T>::pack(u, v);
                        }
                        tmem_st16_u(t_lane + dp_col + half * 32, w);
                        tmem_wait_st();
                    }
                    fence_before_sync();
                    mbar_arrive(b_full);
                }
            }
            if (nt == 0) finish(i, e);
            e_done = e;
        }
        if (nt > 0) finish(nz - 1, e_done);
    }
    finish_cta256(&s_tmem, kTmemCols, warp, &s_fail);
}

// dK and dV from the parts' sums, in their order.  One thread per 8 values;
// grid (chunks of a sequence's rows, B).
template <typename T>
__global__ void __launch_bounds__(256) bias_bwd_parts_kernel(const Problem p, const BwdArgs a) {
    const int b = blockIdx.y;
    Seq s;
    if (!read_pair(p, b, s) || s.q_len == 0) return;
    const int64_t n = static_cast<int64_t>(s.k_len) * p.Hkv * 16, step = static_cast<int64_t>(gridDim.x) * 256;
    const int64_t part_step = static_cast<int64_t>(p.B) * a.part_rows * p.Hkv * 128;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += step) {
        const int c = static_cast<int>(i & 15);   // eight values of dK (0-7) or dV
        const int64_t rz = i >> 4, row = rz / p.Hkv, z = rz - row * p.Hkv;
        const float* src = a.part_sums + ((b * a.part_rows + row) * p.Hkv + z) * 128 + c * 8;
        float v[8] = {};
        for (int k = 0; k < a.parts; ++k) {
            const float4 x = __ldcs(reinterpret_cast<const float4*>(src + k * part_step)), y = __ldcs(reinterpret_cast<const float4*>(src + k * part_step) + 1);
            v[0] += x.x;
            v[1] += x.y;
            v[2] += x.z;
            v[3] += x.w;
            v[4] += y.x;
            v[5] += y.y;
            v[6] += y.z;
            v[7] += y.w;
        }
        uint16_t* dst = (c < 8 ? a.dk : a.dv) + (s.k_start + row) * a.dkv_tok + z * a.dkv_head + (c & 7) * 8;
        *reinterpret_cast<uint4*>(dst) = make_uint4(Cvt<T>::pack(v[0], v[1]), Cvt<T>::pack(v[2], v[3]), Cvt<T>::pack(v[4], v[5]), Cvt<T>::pack(v[6], v[7]));
    }
}

// ---------------------------------------------------------------------------
// weight[h, j] = prev[h, j] + sum_i exp(s[i, j] - lse_i): key rows, transposed
// scores, summed along each thread's row.  grid (key tiles, groups of heads,
// B), three CTAs per SM; TMEM: two score buffers.  Bound by the row warps'
// instructions.  512 sequences of 79 to 118 tokens, 6 heads, f16: 58 us, 352 of
// up to 36, 12 heads: 37; with two CTAs and more registers (an earlier state,
// 60 and 39 us with three) 53 and 48.  The reads alone are 12 us of the first.
// ---------------------------------------------------------------------------

constexpr int kWeightStages = 3;
constexpr uint32_t kWeightTmem = 128;

__host__ __device__ constexpr int weight_smem_bytes(int D, int span) {
    return 1024 + kRowBytes + kWeightStages * kTileBytes + 12 * kChunk + vec16_bytes(D, span) + ids_bytes(D, span);
}

// The statistics of a chunk's far queries, each warp those of its own threads'
// columns.  Every key tile forms them again: there is no place to keep them.
template <typename T>
__device__ __forceinline__ void far_columns(const Problem& p, const Seq& s, int h, int c0, float* s_lse, float* s_mu) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int c = threadIdx.x; c < kChunk; c += 128) {
        const float l = c0 + c < s.q_len ? p.lse[h * p.lse_stride + s.q_start + c0 + c] : 0.f;
        for (uint32_t todo = __ballot_sync(0xffffffffu, is_far(l)); todo != 0; todo &= todo - 1) {
            const int src = __ffs(todo) - 1;
            const float ls = row_log_sum<T>(p, s, c0 + c - lane + src, h);
            if (lane == src) {
                s_lse[c] = -ls * kLog2e;
                s_mu[c] = l - ls;
            }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 3)
    bias_weight_kernel(const Problem p, const float* prev, float* weight, int64_t weight_stride, int heads_per_cta, int span) {
    extern __shared__ uint8_t smem_raw[];
    // k_full, k_empty, q_full[3], s_full[3], a_full[2], done
    constexpr int kBars = 11;
    __shared__ __align__(8) uint64_t s_bar[kBars];
    __shared__ uint16_t s_tab[kMaxBuckets + 1];
    __shared__ __align__(16) TileInfo s_tiles[kChunkTiles];
    __shared__ int s_red[8];
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;

    const int k0 = blockIdx.x * kQTile, h0 = blockIdx.y * heads_per_cta, b = blockIdx.z;
    const int nh = min(heads_per_cta, p.H - h0);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Seq s;
    if (!read_pair(p, b, s) || k0 >= s.k_len || !keys_held(s, weight_stride)) return;
    if (s.q_len == 0) {   // nothing to add
        for (int i = tid; i < nh * kQTile; i += kThreads) {
            const int r = k0 + i % kQTile;
            const int64_t at = (h0 + i / kQTile) * weight_stride + s.k_start + r;
            if (r < s.k_len) weight[at] = prev != nullptr ? prev[at] : 0.f;
        }
        return;
    }
    const int nt = (s.q_len + kTile - 1) / kTile;

    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t sK = (raw + 1023u) & ~1023u;
    const uint32_t sRing = sK + kRowBytes;
    uint8_t* extra = smem_raw + (sRing - raw) + kWeightStages * kTileBytes;
    const uint32_t bar0 = smem_addr(&s_bar[0]);
    const uint32_t k_full = bar0, k_empty = bar0 + 8, done = bar0 + 80;
    auto q_full = [&](uint32_t g) { return bar0 + 8u * (2 + g % 3); };
    auto s_full = [&](uint32_t g) { return bar0 + 8u * (5 + g % 3); };
    auto a_full = [&](uint32_t g) { return bar0 + 8u * (8 + (g & 1)); };
    const Wait wait{&s_fail};

    if (warp == kTcLoadWarp) {
        if (lane < kBars) mbar_init(bar0 + 8 * lane, lane == 0 || (lane >= 2 && lane < 5) ? 32 : lane == 8 || lane == 9 ? 128 : 1);
        if (lane == 0) s_fail = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        __syncwarp();
        start_loads();
        bool ok = !test_hook(1);
        uint32_t g = 0;
        for (int i = 0; ok && i < nh; ++i) {
            const int h = h0 + i;
            if (i > 0) ok = wait.warp(k_empty, (i - 1) & 1);
            if (!ok) break;
            load_rows<kQTile>(sK, p.k + s.k_start * p.kv_tok + (h / p.group) * p.kv_head, p.kv_tok, k0, s.k_len, lane);
            cp_async_arrive_noinc(k_full);
            const uint16_t* qb = p.q + s.q_start * p.q_tok + h * p.q_head;
            for (int t = 0; t < nt; ++t, ++g) {
                if (g >= kWeightStages) ok = wait.warp(s_full(g), (g / 3 - 1) & 1);
                if (!ok) break;
                load_rows<kTile>(sRing + (g % 3) * kTileBytes, qb, p.q_tok, t * kTile, s.q_len, lane);
                cp_async_arrive_noinc(q_full(g));
            }
        }
        cp_async_wait_all();
    } else if (warp == kTcMmaWarp) {
        const uint32_t tmem = start_mma(&s_tmem, kWeightTmem);
        if (lane == 0) {
            const uint32_t idesc = make_idesc(Cvt<T>::kFormat, 0, kTile);
            bool ok = true;
            uint32_t g = 0;
            for (int i = 0; ok && i < nh; ++i) {
                ok = wait(k_full, i & 1);
                for (int t = 0; ok && t < nt; ++t, ++g) {
                    ok = wait(q_full(g), (g / 3) & 1);
                    if (ok && g >= 2) ok = wait(a_full(g), (g / 2 - 1) & 1);   // scores of tile g - 2 have been read
                    if (!ok) break;
                    fence_async_smem();
                    fence_after_sync();
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_f16(tmem + (g & 1) * kTile, make_sdesc(sK + ks * 32), make_sdesc(sRing + (g % 3) * kTileBytes + ks * 32), idesc, ks > 0);
                    mma_commit(s_full(g));
                }
                mma_commit(k_empty);
            }
            mma_commit(done);
            mbar_wait(done, 0);
        }
        __syncwarp();
    } else {
        const int row = k0 + tid;
        const bool valid = row < s.k_len, warp_rows = k0 + warp * 32 < s.k_len;
        Bias16 t;
        t.vec = reinterpret_cast<uint16_t*>(extra);
        uint8_t* ids = extra + vec16_bytes(p.D, span);
        t.off = reinterpret_cast<int*>(ids + ids_bytes(p.D, span));
        float* s_lse = reinterpret_cast<float*>(t.off + kChunk);   // negated
        float* s_mu = s_lse + kChunk;
        t.tiles = s_tiles;
        uint8_t* map = ids + ((vec_entries(p.D, span) + 15) & ~15);
        const bool has_entry = tid < p.num_buckets;
        const uint16_t* column = p.table + static_cast<int64_t>(has_entry ? tid : 0) * p.H + h0;
        // What the set-up needs of global memory, all under way at once.
        const uint16_t entry = __ldg(column);
        const int pos = valid ? key_pos(p, s, row) : 0;
        auto query_at = [&](int c) { return query_pos(p, s, c); };
        Columns<128> cols;
        cols.load(0, s.q_len, query_at);
        bias_map<128>(p, map, p.num_buckets);
        if (has_entry) s_tab[tid] = entry;
        if (tid == p.num_buckets) s_tab[tid] = 0;
        bias_rows<128>(t, p, pos, valid, span, s_red);
        bias_ids<-1, 128>(t, map, ids, p.num_buckets);
        cols.store<true>(t, 0, s.q_len);
        const uint32_t tmem = start_rows(&s_tmem);
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        bool ok = true;
        uint32_t g = 0;
        for (int i = 0; i < nh; ++i) {
            const int h = h0 + i;
            const float* lse = p.lse + h * p.lse_stride + s.q_start;
            const int64_t at = h * weight_stride + s.k_start + row;
            const float old = valid && prev != nullptr ? prev[at] : 0.f;
            float l_next[kChunk / 128];   // on their way under the barriers and the fill
            auto load_lse = [&](int c0) {
#pragma unroll
                for (int k = 0; k < kChunk / 128; ++k) l_next[k] = c0 + tid + k * 128 < s.q_len ? lse[c0 + tid + k * 128] : 0.f;
            };
            load_lse(0);
            const uint16_t next = i == 0 ? uint16_t(0) : __ldg(column + i);
            rows_barrier<128>();   // the last head's entries and columns are no longer read
            if (i > 0) {
                if (has_entry) s_tab[tid] = next;
                rows_barrier<128>();
            }
            bias_fill<128>(t, ids, s_tab);
            float sum_all = 0.f;
            bool far = false;
            for (int tile = 0; tile < nt; ++tile, ++g) {
                if (tile % kChunkTiles == 0) {
                    const int c0 = tile * kTile;
                    const bool again = nt > kChunkTiles && (tile > 0 || i > 0);
                    if (tile > 0) load_lse(c0);
                    if (again) cols.load(c0, s.q_len, query_at);
                    if (tile > 0) rows_barrier<128>();
                    if (again) cols.store<true>(t, c0, s.q_len);
                    bool mine = false;
#pragma unroll
                    for (int k = 0; k < kChunk / 128; ++k) {
                        const int c = tid + k * 128;
                        s_lse[c] = c0 + c < s.q_len ? -lse_log2(l_next[k]) : -INFINITY;
                        s_mu[c] = 0.f;
                        mine |= c0 + c < s.q_len && is_far(l_next[k]);
                    }
                    if (__any_sync(0xffffffffu, mine)) far_columns<T>(p, s, h, c0, s_lse, s_mu);
                    far = rows_any<128>(mine);
                }
                const int kind = far ? kFarKind : tile_kind(t, tile % kChunkTiles), c0 = (tile % kChunkTiles) * kTile;
                ok = ok && wait.warp(s_full(g), (g / 3) & 1);
                if (ok && warp_rows) {
                    fence_after_sync();
                    uint64_t sum = f2(0.f, 0.f);
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        float x[32];
                        tmem_ld32(t_lane + (g & 1) * kTile + hf * 32, x);
                        if (hf == 1) {
                            fence_before_sync();
                            mbar_arrive(a_full(g));
                        }
                        probabilities<T>(t, p, kind, t.off + c0, hf * 32, s_lse + c0, 0.f, s_mu + c0, 0.f, x);
#pragma unroll
                        for (int c = 0; c < 16; ++c) sum = f2_add(sum, f2(x[2 * c], x[2 * c + 1]));
                    }
                    float u, v;
                    f2_split(sum, u, v);
                    sum_all += u + v;
                } else {
                    mbar_arrive(a_full(g));
                }
            }
            if (ok && valid) weight[at] = old + sum_all;
        }
    }
    finish_cta(&s_tmem, kWeightTmem, warp, &s_fail);
}

}  // namespace bias
}  // namespace ragged
