// Gradients of the attention with a learned relative position bias, and the
// attention weight that each key collects, on the tensor cores (see
// bias_tc.cuh for the roles and the expanded bias table).
//
//   P = exp(s - lse),  dP = dO V^T,  delta = rowsum(dO O),  dS = P (dP - delta)
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO,  dtable = sum of dS by bucket
//
// Two kernels, so that every sum has a fixed order and no sum needs atomics:
// one with query rows (dQ, delta, the table), one with key rows (dK, dV,
// transposed scores).  Each recomputes S and dP, 7 products instead of 5.
//
// dS and P are rounded to the 16-bit type to be operands of the next product.
// In f16 they would lose what lies below 2^-14: probabilities of long rows,
// and gradients far below 1.  Both are therefore scaled by powers of two, which
// the accumulators undo exactly: P by 2^14, dS by 2^(6 - e) with e the exponent
// of the largest |dO| of the row (dQ), or of all rows that a key meets (dK).
#pragma once

#include "bias_tc.cuh"

namespace ragged {
namespace bias {

constexpr int kBwdStages = 3;
constexpr int kNoExp = -1000;       // a row (or tile) of zero gradients

template <typename T>
constexpr bool kScaled = std::is_same<T, __half>::value;
constexpr int kPExp = 14, kSExp = 6;

// 2^e for |e| up to 126.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

struct BwdArgs {
    const uint16_t* out;
    const uint16_t* dout;
    int64_t out_tok, dout_tok;
    uint16_t* dq;
    uint16_t* dk;
    uint16_t* dv;
    int64_t dq_tok, dq_head, dkv_tok, dkv_head;
    float* delta;     // [H, lse_stride]
    int* tile_exp;    // [B][H][query tiles]: exponent of the largest |dO|
    float* partial;   // [B][H][query tiles][num_buckets]
    uint16_t* dtable;
    int q_tiles;
    int span;         // of the query kernel's expanded table
};

__host__ __device__ constexpr int bwd_q_fixed_bytes(int num_buckets) {
    return 1024 + 2 * kRowBytes + kBwdStages * 2 * kTileBytes + (num_buckets + 1) * 512 + 4 * kChunk;
}
__host__ __device__ constexpr int bwd_q_smem_bytes(int D, int num_buckets, int span) {
    return bwd_q_fixed_bytes(num_buckets) + 4 * ((vec_entries(D, span) + 3) & ~3) + 2 * ((vec_entries(D, span) + 7) & ~7);
}

// Query rows: dQ, delta, and this tile's sums for the table's gradient.
// grid (query tiles, H, B), two CTAs per SM where the table is small.
//
// TMEM: S, dP (replaced in place by dS) and dQ, 64 columns each.  S of the next
// tile is computed while dS of this one is, and dP of the next one while its
// probabilities are.
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) bias_bwd_q_kernel(const Problem p, const BwdArgs a) {
    extern __shared__ uint8_t smem_raw[];
    // stat_full, tile_full[3], s_full, dp_full[2], a_full, b_full, done
    __shared__ __align__(8) uint64_t s_bar[10];
    __shared__ float s_tab[kMaxBuckets], s_rowscale[kQTile];
    __shared__ int s_kind[kChunkTiles], s_red[8];
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;

    const int q0 = blockIdx.x * kQTile, h = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t item = (static_cast<int64_t>(b) * p.H + h) * a.q_tiles + blockIdx.x;
    Seq s;
    const bool any = read_pair(p, b, s) && q0 < s.q_len;
    if (!any || s.k_len == 0) {   // nothing for the table; queries without keys get no gradient
        if (tid < p.num_buckets) a.partial[item * p.num_buckets + tid] = 0.f;
        if (any && tid < kQTile && q0 + tid < s.q_len) {
            const uint32_t zero[32] = {};
            store_row(a.dq + static_cast<int64_t>(s.q_start + q0 + tid) * a.dq_tok + h * a.dq_head, zero);
        }
        return;
    }
    const int nt = (s.k_len + kTile - 1) / kTile;

    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t sQ = (raw + 1023u) & ~1023u;
    const uint32_t sdO = sQ + kRowBytes, sRing = sdO + kRowBytes;   // stage: K, then V
    float* acc = reinterpret_cast<float*>(smem_raw + (sRing - raw) + kBwdStages * 2 * kTileBytes);   // [buckets + 1][128]
    auto stage = [&](uint32_t g) { return sRing + (g % kBwdStages) * 2 * kTileBytes; };

    const uint32_t bar0 = smem_addr(&s_bar[0]);
    const uint32_t stat_full = bar0, s_full = bar0 + 8u * 4, a_full = bar0 + 8u * 7, b_full = bar0 + 8u * 8, done = bar0 + 8u * 9;
    auto tile_full = [&](uint32_t g) { return bar0 + 8u * (1 + g % kBwdStages); };
    // Two barriers, so that the load warp's wait for tile g - 2 is exact: that
    // barrier's next phase needs tile g, which it has yet to load.
    auto dp_full = [&](uint32_t g) { return bar0 + 8u * (5 + (g & 1)); };
    if (tid == 0) {
        mbar_init(stat_full, 32);
        for (int i = 0; i < kBwdStages; ++i) mbar_init(tile_full(i), 32);
        mbar_init(s_full, 1);
        mbar_init(dp_full(0), 1);
        mbar_init(dp_full(1), 1);
        mbar_init(a_full, 128);
        mbar_init(b_full, 128);
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        s_fail = 0;
    }
    const uint32_t tmem = tmem_alloc(&s_tmem, kTmemCols, warp);
    const uint32_t dp_col = kTile, dq_col = 2 * kTile;
    const Wait wait{&s_fail};

    if (warp == kTcLoadWarp) {
        const int64_t z = static_cast<int64_t>(h / p.group) * p.kv_head;
        const uint16_t* kb = p.k + s.k_start * p.kv_tok + z;
        const uint16_t* vb = p.v + s.k_start * p.kv_tok + z;
        load_rows<kQTile>(sQ, p.q + s.q_start * p.q_tok + h * p.q_head, p.q_tok, q0, s.q_len, lane);
        load_rows<kQTile>(sdO, a.dout + s.q_start * a.dout_tok + h * 64, a.dout_tok, q0, s.q_len, lane);
        cp_async_arrive_noinc(stat_full);
        bool ok = true;
        for (uint32_t g = 0; g < static_cast<uint32_t>(nt); ++g) {
            // dP(g - 2) was issued behind dQ(g - 3), the last product of the stage's previous tile.
            if (g >= kBwdStages) ok = wait.warp(dp_full(g), ((g - 2) >> 1) & 1);
            if (!ok) break;
            load_rows<kTile>(stage(g), kb, p.kv_tok, g * kTile, s.k_len, lane);
            load_rows<kTile>(stage(g) + kTileBytes, vb, p.kv_tok, g * kTile, s.k_len, lane);
            cp_async_arrive_noinc(tile_full(g));
        }
        cp_async_wait_all();
    } else if (warp == kTcMmaWarp) {
        if (lane == 0) {
            const uint32_t idesc_s = make_idesc(Cvt<T>::kFormat, 0, kTile), idesc_g = make_idesc(Cvt<T>::kFormat, 1, 64);
            const uint32_t n = nt;
            auto product = [&](uint32_t col, uint32_t sa, uint32_t sb) {   // [128, 64] = A B^T over the head dimension
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_f16(tmem + col, make_sdesc(sa + ks * 32), make_sdesc(sb + ks * 32), idesc_s, ks > 0);
            };
            bool ok = wait(stat_full, 0) && wait(tile_full(0), 0);
            if (ok) {
                fence_async_smem();
                fence_after_sync();
                product(0, sQ, stage(0));
                mma_commit(s_full);
                product(dp_col, sdO, stage(0) + kTileBytes);
                mma_commit(dp_full(0));
            }
            for (uint32_t g = 0; ok && g < n; ++g) {
                ok = wait(a_full, g & 1);
                if (ok && g + 1 < n) {
                    ok = wait(tile_full(g + 1), ((g + 1) / kBwdStages) & 1);
                    if (!ok) break;
                    fence_async_smem();
                    fence_after_sync();
                    product(0, sQ, stage(g + 1));
                    mma_commit(s_full);
                }
                ok = ok && wait(b_full, g & 1);
                if (!ok) break;
                fence_after_sync();
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_f16_ts(tmem + dq_col, tmem + dp_col + ks * 8, make_sdesc(stage(g) + ks * 2048), idesc_g,
                               (g > 0 || ks > 0) ? 1u : 0u);
                if (g + 1 < n) {
                    product(dp_col, sdO, stage(g + 1) + kTileBytes);
                    mma_commit(dp_full(g + 1));
                }
            }
            mma_commit(done);
            mbar_wait(done, 0);
        }
    } else {
        const int row = q0 + tid;
        const bool valid = row < s.q_len, warp_rows = q0 + warp * 32 < s.q_len;
        const int64_t t_row = s.q_start + (valid ? row : 0);
        Bias t;
        uint8_t* extra = reinterpret_cast<uint8_t*>(acc + (p.num_buckets + 1) * kQTile);
        t.vec = reinterpret_cast<float*>(extra);
        uint16_t* ids = reinterpret_cast<uint16_t*>(extra + 4 * ((vec_entries(p.D, a.span) + 3) & ~3));
        t.off = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(ids) + 2 * ((vec_entries(p.D, a.span) + 7) & ~7));
        t.kind = s_kind;
        t.tab = s_tab;
        // delta, and the exponent of the row's largest |dO|
        float delta = 0.f, big = 0.f;
        if (valid) {
            const uint4* o = reinterpret_cast<const uint4*>(a.out + t_row * a.out_tok + h * 64);
            const uint4* d = reinterpret_cast<const uint4*>(a.dout + t_row * a.dout_tok + h * 64);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const uint4 x = __ldg(o + c), y = __ldg(d + c);
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float d0 = to_float<T>(static_cast<uint16_t>(ys[i])), d1 = to_float<T>(static_cast<uint16_t>(ys[i] >> 16));
                    delta = fmaf(to_float<T>(static_cast<uint16_t>(xs[i])), d0, delta);
                    delta = fmaf(to_float<T>(static_cast<uint16_t>(xs[i] >> 16)), d1, delta);
                    if constexpr (kScaled<T>) big = fmaxf(big, fmaxf(fabsf(d0), fabsf(d1)));
                }
            }
            a.delta[h * p.lse_stride + t_row] = delta;
        }
        int e = kNoExp;
        float r = 1.f, undo = 1.f;   // dS is kept times r
        if constexpr (kScaled<T>) {
            if (big > 0.f && big < INFINITY) {
                e = ilogbf(big) + 1;
                r = pow2(kSExp - e);
                undo = pow2(e - kSExp);
            }
            const int top = __reduce_max_sync(0xffffffffu, e);
            if (lane == 0) s_red[warp] = top;
            row_barrier();
            if (tid == 0) a.tile_exp[item] = max(max(s_red[0], s_red[1]), max(s_red[2], s_red[3]));
            row_barrier();
        }
        const float lse = valid ? lse_log2(p.lse[h * p.lse_stride + t_row]) : INFINITY;
        for (int n = 0; n <= p.num_buckets; ++n) acc[n * kQTile + tid] = 0.f;
        bias_rows(t, p, valid ? query_pos(p, s, row) : 0, valid, a.span, s_red);
        bias_expand<T, 1, true>(t, p, h, ids);

        const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        const uint64_t nl2 = f2(-lse, -lse), r2 = f2(r, r), nd2 = f2(-delta * r, -delta * r);
        const char* id_row = reinterpret_cast<const char*>(ids) + (t.row >> 1);
        char* acc_row = reinterpret_cast<char*>(acc + tid);
        float far_left = 0.f, far_right = 0.f;   // dS of the tiles past either end of the table
        bool ok = true;
        for (int g = 0; g < nt; ++g) {
            if (g % kChunkTiles == 0) {
                if (g) row_barrier();
                bias_columns(t, g * kTile, s.k_len, [&](int c) { return key_pos(p, s, c); });
                row_barrier();
            }
            const int kind = t.kind[g % kChunkTiles];
            const int* off = t.off + (g % kChunkTiles) * kTile;
            const int cols = s.k_len - g * kTile;
            float x[2][32];
            ok = ok && wait.warp(s_full, g & 1);
            if (ok && warp_rows) {
                fence_after_sync();
                tmem_ld32(t_lane, x[0]);
                tmem_ld32(t_lane + 32, x[1]);
            }
            fence_before_sync();
            mbar_arrive(a_full);
            if (ok && warp_rows) {
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    bias_add(t, kind, off, hf * 32, p.scale_log2, x[hf]);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float u, v;
                        f2_split(f2_add(f2(x[hf][2 * i], x[hf][2 * i + 1]), nl2), u, v);
                        x[hf][2 * i] = mma_attn::fast_exp2(u);
                        x[hf][2 * i + 1] = mma_attn::fast_exp2(v);
                    }
                }
                if (cols < kTile) {
#pragma unroll
                    for (int i = 0; i < 64; ++i)
                        if (i >= cols) x[i >> 5][i & 31] = 0.f;
                }
            }
            ok = ok && wait.warp(dp_full(g), (g >> 1) & 1);
            if (ok && warp_rows) {
                fence_after_sync();
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    float y[32];
                    tmem_ld32(t_lane + dp_col + hf * 32, y);
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint64_t d = f2_mul(f2(x[hf][2 * i], x[hf][2 * i + 1]), f2_fma(f2(y[2 * i], y[2 * i + 1]), r2, nd2));
                        f2_split(d, x[hf][2 * i], x[hf][2 * i + 1]);
                        w[i] = Cvt<T>::pack(x[hf][2 * i], x[hf][2 * i + 1]);
                    }
                    tmem_st16_u(t_lane + dp_col + hf * 16, w);
                }
                tmem_wait_st();
            }
            fence_before_sync();
            mbar_arrive(b_full);
            if (ok && warp_rows) {   // the table's share, behind the hand-over
                if (kind == kLeft || kind == kRight) {
                    float sum = 0.f;
#pragma unroll
                    for (int i = 0; i < 32; ++i) sum += x[0][i] + x[1][i];
                    if (kind == kLeft) far_left += sum;
                    else far_right += sum;
                } else if (kind == kClamped) {
#pragma unroll
                    for (int i = 0; i < 64; ++i) {
                        const int d = max(-t.D, min(t.D, pos_diff(off[i], t.p_row)));
                        *reinterpret_cast<float*>(acc_row + ids[d + t.D]) += x[i >> 5][i & 31];
                    }
                } else if (kind == kConsecutive) {
                    const uint16_t* id = reinterpret_cast<const uint16_t*>(id_row + (off[0] >> 1));
#pragma unroll
                    for (int i = 0; i < 64; ++i) *reinterpret_cast<float*>(acc_row + id[i]) += x[i >> 5][i & 31];
                } else {
#pragma unroll
                    for (int i = 0; i < 64; ++i)
                        *reinterpret_cast<float*>(acc_row + *reinterpret_cast<const uint16_t*>(id_row + (off[i] >> 1))) += x[i >> 5][i & 31];
                }
            }
        }
        ok = ok && wait.warp(done, 0);
        if (ok && warp_rows) {
            fence_after_sync();
            store_tmem_row<T>(t_lane + dq_col, p.scale * undo, a.dq + t_row * a.dq_tok + h * a.dq_head, valid);
        }
        // This tile's share of the table's gradient: each thread's sums, unscaled, in a fixed order.
        if (t.last >= 0) {
            *reinterpret_cast<float*>(acc_row + ids[0]) += far_left;
            *reinterpret_cast<float*>(acc_row + ids[t.last]) += far_right;
        }
        s_rowscale[tid] = valid ? undo : 0.f;
        row_barrier();
        for (int n = warp; n < p.num_buckets; n += kRowWarps) {
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int u = lane + 32 * k;
                sum += q0 + u < s.q_len ? acc[n * kQTile + u] * s_rowscale[u] : 0.f;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) a.partial[item * p.num_buckets + n] = sum;
        }
    }
    tmem_free(tmem, kTmemCols, warp, &s_fail);
}

__host__ __device__ constexpr int bwd_kv_smem_bytes(int D) {
    return 1024 + 2 * kRowBytes + kBwdStages * 2 * kTileBytes + 4 * ((vec_entries(D, kSpan) + 3) & ~3) + 12 * kChunk;
}

// Key rows: dK and dV, over the query tiles of every query head of the key's
// head.  grid (key tiles, Hkv, B), two CTAs per SM.
//
// TMEM: S^T (replaced by P^T), dP^T (replaced by dS^T), dK and dV.
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) bias_bwd_kv_kernel(const Problem p, const BwdArgs a) {
    extern __shared__ uint8_t smem_raw[];
    // stat_full, tile_full[3], s_full, dp_full[2], a_full, b_full, done
    __shared__ __align__(8) uint64_t s_bar[10];
    __shared__ float s_tab[kMaxBuckets];
    __shared__ int s_kind[kChunkTiles], s_red[8];
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;

    const int k0 = blockIdx.x * kQTile, z = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Seq s;
    if (!read_pair(p, b, s) || k0 >= s.k_len) return;
    if (s.q_len == 0) {   // keys without queries
        if (tid < kQTile && k0 + tid < s.k_len) {
            const uint32_t zero[32] = {};
            const int64_t at = static_cast<int64_t>(s.k_start + k0 + tid) * a.dkv_tok + z * a.dkv_head;
            store_row(a.dk + at, zero);
            store_row(a.dv + at, zero);
        }
        return;
    }
    const int nt = (s.q_len + kTile - 1) / kTile;   // per query head
    const uint32_t n = static_cast<uint32_t>(nt) * p.group;

    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t sK = (raw + 1023u) & ~1023u;
    const uint32_t sV = sK + kRowBytes, sRing = sV + kRowBytes;   // stage: Q, then dO
    uint8_t* extra = smem_raw + (sRing - raw) + kBwdStages * 2 * kTileBytes;
    auto stage = [&](uint32_t g) { return sRing + (g % kBwdStages) * 2 * kTileBytes; };

    const uint32_t bar0 = smem_addr(&s_bar[0]);
    const uint32_t stat_full = bar0, s_full = bar0 + 8u * 4, a_full = bar0 + 8u * 7, b_full = bar0 + 8u * 8, done = bar0 + 8u * 9;
    auto tile_full = [&](uint32_t g) { return bar0 + 8u * (1 + g % kBwdStages); };
    auto dp_full = [&](uint32_t g) { return bar0 + 8u * (5 + (g & 1)); };
    if (tid == 0) {
        mbar_init(stat_full, 32);
        for (int i = 0; i < kBwdStages; ++i) mbar_init(tile_full(i), 32);
        mbar_init(s_full, 1);
        mbar_init(dp_full(0), 1);
        mbar_init(dp_full(1), 1);
        mbar_init(a_full, 128);
        mbar_init(b_full, 128);
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        s_fail = 0;
    }
    const uint32_t tmem = tmem_alloc(&s_tmem, kTmemCols, warp);
    const uint32_t dp_col = kTile, dk_col = 2 * kTile, dv_col = 3 * kTile;
    const Wait wait{&s_fail};

    if (warp == kTcLoadWarp) {
        const int64_t at = s.k_start * p.kv_tok + z * p.kv_head;
        load_rows<kQTile>(sK, p.k + at, p.kv_tok, k0, s.k_len, lane);
        load_rows<kQTile>(sV, p.v + at, p.kv_tok, k0, s.k_len, lane);
        cp_async_arrive_noinc(stat_full);
        bool ok = true;
        uint32_t g = 0;
        for (int h = z * p.group; ok && h < (z + 1) * p.group; ++h) {
            const uint16_t* qb = p.q + s.q_start * p.q_tok + h * p.q_head;
            const uint16_t* db = a.dout + s.q_start * a.dout_tok + h * 64;
            for (int i = 0; i < nt; ++i, ++g) {
                if (g >= kBwdStages) ok = wait.warp(dp_full(g), ((g - 2) >> 1) & 1);
                if (!ok) break;
                load_rows<kTile>(stage(g), qb, p.q_tok, i * kTile, s.q_len, lane);
                load_rows<kTile>(stage(g) + kTileBytes, db, a.dout_tok, i * kTile, s.q_len, lane);
                cp_async_arrive_noinc(tile_full(g));
            }
        }
        cp_async_wait_all();
    } else if (warp == kTcMmaWarp) {
        if (lane == 0) {
            const uint32_t idesc_s = make_idesc(Cvt<T>::kFormat, 0, kTile), idesc_g = make_idesc(Cvt<T>::kFormat, 1, 64);
            auto product = [&](uint32_t col, uint32_t sa, uint32_t sb) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_f16(tmem + col, make_sdesc(sa + ks * 32), make_sdesc(sb + ks * 32), idesc_s, ks > 0);
            };
            auto gradient = [&](uint32_t col, uint32_t from, uint32_t sb, bool first) {   // += A (TMEM) B
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_f16_ts(tmem + col, tmem + from + ks * 8, make_sdesc(sb + ks * 2048), idesc_g, (!first || ks > 0) ? 1u : 0u);
            };
            bool ok = wait(stat_full, 0) && wait(tile_full(0), 0);
            if (ok) {
                fence_async_smem();
                fence_after_sync();
                product(0, sK, stage(0));
                mma_commit(s_full);
                product(dp_col, sV, stage(0) + kTileBytes);
                mma_commit(dp_full(0));
            }
            for (uint32_t g = 0; ok && g < n; ++g) {
                ok = wait(a_full, g & 1);
                if (!ok) break;
                fence_after_sync();
                gradient(dv_col, 0, stage(g) + kTileBytes, g == 0);
                if (g + 1 < n) {
                    ok = wait(tile_full(g + 1), ((g + 1) / kBwdStages) & 1);
                    if (!ok) break;
                    fence_async_smem();
                    fence_after_sync();
                    product(0, sK, stage(g + 1));
                    mma_commit(s_full);
                }
                ok = wait(b_full, g & 1);
                if (!ok) break;
                fence_after_sync();
                gradient(dk_col, dp_col, stage(g), g == 0);
                if (g + 1 < n) {
                    product(dp_col, sV, stage(g + 1) + kTileBytes);
                    mma_commit(dp_full(g + 1));
                }
            }
            mma_commit(done);
            mbar_wait(done, 0);
        }
    } else {
        const int row = k0 + tid;
        const bool valid = row < s.k_len, warp_rows = k0 + warp * 32 < s.k_len;
        Bias t;
        t.vec = reinterpret_cast<float*>(extra);
        t.off = reinterpret_cast<int*>(extra + 4 * ((vec_entries(p.D, kSpan) + 3) & ~3));
        float* s_lse = reinterpret_cast<float*>(t.off + kChunk);
        float* s_delta = s_lse + kChunk;
        t.kind = s_kind;
        t.tab = s_tab;
        bias_rows(t, p, valid ? key_pos(p, s, row) : 0, valid, kSpan, s_red);
        // One scale for everything that this key sums: the largest |dO| of its queries.
        int e = 0;
        if constexpr (kScaled<T>) {
            int top = kNoExp;
            const int tiles = (s.q_len + kQTile - 1) / kQTile;
            for (int i = tid; i < tiles * p.group; i += 128) {
                const int hh = i / tiles;
                top = max(top, a.tile_exp[(static_cast<int64_t>(b) * p.H + z * p.group + hh) * a.q_tiles + (i - hh * tiles)]);
            }
            top = __reduce_max_sync(0xffffffffu, top);
            row_barrier();   // bias_rows' extremes are no longer read
            if (lane == 0) s_red[warp] = top;
            row_barrier();
            top = max(max(s_red[0], s_red[1]), max(s_red[2], s_red[3]));
            e = top == kNoExp ? 0 : top;
        }
        const float shift = kScaled<T> ? static_cast<float>(kPExp) : 0.f;
        const float r = kScaled<T> ? pow2(kSExp - e - kPExp) : 1.f;

        const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        const uint64_t r2 = f2(r, r);
        bool ok = true;
        uint32_t g = 0;
        for (int h = z * p.group; h < (z + 1) * p.group; ++h) {
            bias_expand<T, -1, false>(t, p, h, nullptr);
            const float* lse = p.lse + h * p.lse_stride + s.q_start;
            const float* delta = a.delta + h * p.lse_stride + s.q_start;
            for (int i0 = 0; i0 < nt; ++i0, ++g) {
                if (i0 % kChunkTiles == 0) {
                    if (i0) row_barrier();
                    const int c0 = i0 * kTile;
                    bias_columns(t, c0, s.q_len, [&](int c) { return query_pos(p, s, c); });
                    for (int c = tid; c < kChunk && c0 + c < ((s.q_len + kTile - 1) & ~(kTile - 1)); c += 128) {
                        const bool in = c0 + c < s.q_len;
                        s_lse[c] = in ? lse_log2(lse[c0 + c]) - shift : INFINITY;   // no such query: p = 0
                        s_delta[c] = in ? -delta[c0 + c] * r : 0.f;
                    }
                    row_barrier();
                }
                const int kind = t.kind[i0 % kChunkTiles], c0 = (i0 % kChunkTiles) * kTile;
                const int* off = t.off + c0;
                float x[2][32];
                ok = ok && wait.warp(s_full, g & 1);
                if (ok && warp_rows) {
                    fence_after_sync();
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        tmem_ld32(t_lane + hf * 32, x[hf]);
                        bias_add(t, kind, off, hf * 32, p.scale_log2, x[hf]);
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 l = *reinterpret_cast<const float4*>(s_lse + c0 + hf * 32 + 4 * i);
                            float u[4];
                            f2_split(f2_sub(f2(x[hf][4 * i], x[hf][4 * i + 1]), f2(l.x, l.y)), u[0], u[1]);
                            f2_split(f2_sub(f2(x[hf][4 * i + 2], x[hf][4 * i + 3]), f2(l.z, l.w)), u[2], u[3]);
#pragma unroll
                            for (int j = 0; j < 4; ++j) x[hf][4 * i + j] = mma_attn::fast_exp2(u[j]);
                            w[2 * i] = Cvt<T>::pack(x[hf][4 * i], x[hf][4 * i + 1]);
                            w[2 * i + 1] = Cvt<T>::pack(x[hf][4 * i + 2], x[hf][4 * i + 3]);
                        }
                        tmem_st16_u(t_lane + hf * 16, w);
                    }
                    tmem_wait_st();
                }
                fence_before_sync();
                mbar_arrive(a_full);
                ok = ok && wait.warp(dp_full(g), (g >> 1) & 1);
                if (ok && warp_rows) {
                    fence_after_sync();
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        float y[32];
                        tmem_ld32(t_lane + dp_col + hf * 32, y);
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 d = *reinterpret_cast<const float4*>(s_delta + c0 + hf * 32 + 4 * i);
                            float u[4];
                            f2_split(f2_mul(f2(x[hf][4 * i], x[hf][4 * i + 1]), f2_fma(f2(y[4 * i], y[4 * i + 1]), r2, f2(d.x, d.y))), u[0], u[1]);
                            f2_split(f2_mul(f2(x[hf][4 * i + 2], x[hf][4 * i + 3]), f2_fma(f2(y[4 * i + 2], y[4 * i + 3]), r2, f2(d.z, d.w))), u[2], u[3]);
                            w[2 * i] = Cvt<T>::pack(u[0], u[1]);
                            w[2 * i + 1] = Cvt<T>::pack(u[2], u[3]);
                        }
                        tmem_st16_u(t_lane + dp_col + hf * 16, w);
                    }
                    tmem_wait_st();
                }
                fence_before_sync();
                mbar_arrive(b_full);
            }
        }
        ok = ok && wait.warp(done, 0);
        if (ok && warp_rows) {
            fence_after_sync();
            const int64_t at = static_cast<int64_t>(s.k_start + (valid ? row : 0)) * a.dkv_tok + z * a.dkv_head;
            store_tmem_row<T>(t_lane + dk_col, kScaled<T> ? p.scale * pow2(e - kSExp) : p.scale, a.dk + at, valid);
            store_tmem_row<T>(t_lane + dv_col, kScaled<T> ? pow2(-kPExp) : 1.f, a.dv + at, valid);
        }
    }
    tmem_free(tmem, kTmemCols, warp, &s_fail);
}

// dtable[n, h] = sum of the tiles' sums, in a fixed order.  grid (num_buckets, H)
template <typename T>
__global__ void __launch_bounds__(256) bias_bwd_table_kernel(const Problem p, const BwdArgs a) {
    __shared__ float s_sum[8];
    const int n = blockIdx.x, h = blockIdx.y, tiles = a.q_tiles;
    float x = 0.f;
    for (int i = threadIdx.x; i < p.B * tiles; i += 256) {
        const int b = i / tiles, t = i - b * tiles;
        x += a.partial[((static_cast<int64_t>(b) * p.H + h) * tiles + t) * p.num_buckets + n];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = x;
    __syncthreads();
    if (threadIdx.x == 0) {
        x = 0.f;
        for (int w = 0; w < 8; ++w) x += s_sum[w];
        a.dtable[static_cast<int64_t>(n) * p.H + h] = from_float<T>(x);
    }
}

// ---------------------------------------------------------------------------
// weight[h, j] = prev[h, j] + sum_i exp(s[i, j] - lse_i): key rows, transposed
// scores, summed along each thread's row.  grid (key tiles, H, B).
// ---------------------------------------------------------------------------

constexpr int kWeightStages = 3;
constexpr uint32_t kWeightTmem = 128;

__host__ __device__ constexpr int weight_smem_bytes(int D) {
    return 1024 + kRowBytes + kWeightStages * kTileBytes + 4 * ((vec_entries(D, kSpan) + 3) & ~3) + 8 * kChunk;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 3)
    bias_weight_kernel(const Problem p, const float* prev, float* weight, int64_t weight_stride) {
    extern __shared__ uint8_t smem_raw[];
    // k_full, tile_full[3], s_full[3], a_full[2], done
    __shared__ __align__(8) uint64_t s_bar[10];
    __shared__ float s_tab[kMaxBuckets];
    __shared__ int s_kind[kChunkTiles], s_red[8];
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;

    const int k0 = blockIdx.x * kQTile, h = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Seq s;
    if (!read_pair(p, b, s) || k0 >= s.k_len) return;
    const int64_t at = h * weight_stride + s.k_start + k0 + tid;
    if (s.q_len == 0) {
        if (tid < kQTile && k0 + tid < s.k_len) weight[at] = prev != nullptr ? prev[at] : 0.f;
        return;
    }
    const int nt = (s.q_len + kTile - 1) / kTile;

    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t sK = (raw + 1023u) & ~1023u;
    const uint32_t sRing = sK + kRowBytes;
    uint8_t* extra = smem_raw + (sRing - raw) + kWeightStages * kTileBytes;
    const uint32_t bar0 = smem_addr(&s_bar[0]);
    const uint32_t k_full = bar0, done = bar0 + 8u * 9;
    auto tile_full = [&](uint32_t g) { return bar0 + 8u * (1 + g % 3); };
    auto s_full = [&](uint32_t g) { return bar0 + 8u * (4 + g % 3); };
    auto a_full = [&](uint32_t g) { return bar0 + 8u * (7 + (g & 1)); };
    if (tid == 0) {
        mbar_init(k_full, 32);
        for (int i = 0; i < 3; ++i) {
            mbar_init(tile_full(i), 32);
            mbar_init(s_full(i), 1);
        }
        mbar_init(a_full(0), 128);
        mbar_init(a_full(1), 128);
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        s_fail = 0;
    }
    const uint32_t tmem = tmem_alloc(&s_tmem, kWeightTmem, warp);
    const Wait wait{&s_fail};

    if (warp == kTcLoadWarp) {
        const uint16_t* qb = p.q + s.q_start * p.q_tok + h * p.q_head;
        load_rows<kQTile>(sK, p.k + s.k_start * p.kv_tok + (h / p.group) * p.kv_head, p.kv_tok, k0, s.k_len, lane);
        cp_async_arrive_noinc(k_full);
        bool ok = true;
        for (uint32_t g = 0; g < static_cast<uint32_t>(nt); ++g) {
            if (g >= kWeightStages) ok = wait.warp(s_full(g), ((g - 3) / 3) & 1);
            if (!ok) break;
            load_rows<kTile>(sRing + (g % 3) * kTileBytes, qb, p.q_tok, g * kTile, s.q_len, lane);
            cp_async_arrive_noinc(tile_full(g));
        }
        cp_async_wait_all();
    } else if (warp == kTcMmaWarp) {
        if (lane == 0) {
            const uint32_t idesc = make_idesc(Cvt<T>::kFormat, 0, kTile);
            bool ok = wait(k_full, 0);
            for (uint32_t g = 0; ok && g < static_cast<uint32_t>(nt); ++g) {
                ok = wait(tile_full(g), (g / 3) & 1);
                if (ok && g >= 2) ok = wait(a_full(g), ((g - 2) >> 1) & 1);   // scores of tile g - 2 have been read
                if (!ok) break;
                fence_async_smem();
                fence_after_sync();
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_f16(tmem + (g & 1) * kTile, make_sdesc(sK + ks * 32), make_sdesc(sRing + (g % 3) * kTileBytes + ks * 32),
                            idesc, ks > 0);
                mma_commit(s_full(g));
            }
            mma_commit(done);
            mbar_wait(done, 0);
        }
    } else {
        const int row = k0 + tid;
        const bool valid = row < s.k_len, warp_rows = k0 + warp * 32 < s.k_len;
        Bias t;
        t.vec = reinterpret_cast<float*>(extra);
        t.off = reinterpret_cast<int*>(extra + 4 * ((vec_entries(p.D, kSpan) + 3) & ~3));
        float* s_lse = reinterpret_cast<float*>(t.off + kChunk);
        t.kind = s_kind;
        t.tab = s_tab;
        bias_rows(t, p, valid ? key_pos(p, s, row) : 0, valid, kSpan, s_red);
        bias_expand<T, -1, false>(t, p, h, nullptr);
        const float* lse = p.lse + h * p.lse_stride + s.q_start;
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        float total = 0.f;
        bool ok = true;
        for (int g = 0; g < nt; ++g) {
            if (g % kChunkTiles == 0) {
                if (g) row_barrier();
                const int c0 = g * kTile;
                bias_columns(t, c0, s.q_len, [&](int c) { return query_pos(p, s, c); });
                for (int c = tid; c < kChunk && c0 + c < ((s.q_len + kTile - 1) & ~(kTile - 1)); c += 128)
                    s_lse[c] = c0 + c < s.q_len ? lse_log2(lse[c0 + c]) : INFINITY;
                row_barrier();
            }
            const int kind = t.kind[g % kChunkTiles], c0 = (g % kChunkTiles) * kTile;
            ok = ok && wait.warp(s_full(g), (g / 3) & 1);
            if (ok && warp_rows) {
                fence_after_sync();
                float x[2][32];
                tmem_ld32(t_lane + (g & 1) * kTile, x[0]);
                tmem_ld32(t_lane + (g & 1) * kTile + 32, x[1]);
                fence_before_sync();
                mbar_arrive(a_full(g));
                uint64_t sum = f2(0.f, 0.f);
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    bias_add(t, kind, t.off + c0, hf * 32, p.scale_log2, x[hf]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 l = *reinterpret_cast<const float4*>(s_lse + c0 + hf * 32 + 4 * i);
                        float u[4];
                        f2_split(f2_sub(f2(x[hf][4 * i], x[hf][4 * i + 1]), f2(l.x, l.y)), u[0], u[1]);
                        f2_split(f2_sub(f2(x[hf][4 * i + 2], x[hf][4 * i + 3]), f2(l.z, l.w)), u[2], u[3]);
                        sum = f2_add(sum, f2(mma_attn::fast_exp2(u[0]), mma_attn::fast_exp2(u[1])));
                        sum = f2_add(sum, f2(mma_attn::fast_exp2(u[2]), mma_attn::fast_exp2(u[3])));
                    }
                }
                float a, c;
                f2_split(sum, a, c);
                total += a + c;
            } else {
                mbar_arrive(a_full(g));
            }
        }
        if (ok && valid) weight[at] = (prev != nullptr ? prev[at] : 0.f) + total;
    }
    tmem_free(tmem, kWeightTmem, warp, &s_fail);
}

}  // namespace bias
}  // namespace ragged
