// Host side of the operators with a learned relative position bias and of the
// eviction (declared in ragged.h).  Included by ragged_api.cu, whose argument
// helpers (fail, cuda_check, aligned16, ensure_smem) it uses.
#pragma once

#include "bias_bwd.cuh"
#include "bias_few.cuh"
#include "evict.cuh"

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

ragged_status check_stride16(int64_t elements, const char* what) {
    if (elements <= 0 || elements % 8)
        return fail(RAGGED_ERR_INVALID_ARG, "%s = %lld must be a positive multiple of 16 bytes", what, (long long)elements);
    return RAGGED_OK;
}

// Argument checks shared by the three operators; fills the kernels' view.
ragged_status check_bias_problem(const ragged_bias_attn* a, bool need_v, ragged::bias::Problem* p) {
    if (a == nullptr) return fail(RAGGED_ERR_INVALID_ARG, "the problem is NULL");
    if (a->B < 0) return fail(RAGGED_ERR_INVALID_ARG, "B = %lld is negative", (long long)a->B);
    if (a->B > 65535) return fail(RAGGED_ERR_UNSUPPORTED, "B = %lld exceeds 65535", (long long)a->B);
    if (a->dtype != RAGGED_F16 && a->dtype != RAGGED_BF16 && a->dtype != RAGGED_F32)
        return fail(RAGGED_ERR_INVALID_ARG, "unknown dtype %d", (int)a->dtype);
    if (a->dtype == RAGGED_F32) return fail(RAGGED_ERR_UNSUPPORTED, "the attention with a position bias takes f16 and bf16");
    if (a->head_dim != 64)
        return fail(RAGGED_ERR_UNSUPPORTED, "head_dim = %lld (only 64 is implemented)", (long long)a->head_dim);
    if (a->H < 1 || a->H > 65534) return fail(RAGGED_ERR_INVALID_ARG, "H = %lld outside [1, 65534]", (long long)a->H);
    if (a->Hkv < 1 || a->H % a->Hkv)
        return fail(RAGGED_ERR_INVALID_ARG, "H = %lld is not a multiple of Hkv = %lld", (long long)a->H, (long long)a->Hkv);
    const int64_t longest[2] = {a->max_seqlen_q, a->max_seqlen_k};
    for (int64_t n : longest)
        if (n < 1 || n > RAGGED_MAX_TOKENS)
            return fail(RAGGED_ERR_INVALID_ARG, "max_seqlen = %lld outside [1, %d]", (long long)n, RAGGED_MAX_TOKENS);
    if (!(a->scale > 0.f) || a->scale > 1.0e38f)   // times log2 e it stays finite
        return fail(RAGGED_ERR_INVALID_ARG, "scale must be positive and at most 1e38");
    if (a->num_buckets < 1 || a->num_buckets > ragged::bias::kMaxBuckets)
        return fail(RAGGED_ERR_UNSUPPORTED, "num_buckets = %lld outside [1, %d]", (long long)a->num_buckets,
                    ragged::bias::kMaxBuckets);
    if (a->max_distance < 0 || a->max_distance > ragged::bias::kMaxDistance)
        return fail(RAGGED_ERR_UNSUPPORTED, "max_distance = %lld outside [0, %d]", (long long)a->max_distance,
                    ragged::bias::kMaxDistance);
    if (a->B > 0) {
        if (!a->q || !a->k || (need_v && !a->v) || !a->cu_seqlens_q || !a->cu_seqlens_k || !a->table || !a->buckets || !a->lse)
            return fail(RAGGED_ERR_INVALID_ARG, "q, k, v, cu_seqlens, table, buckets and lse must not be NULL");
        if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->v))
            return fail(RAGGED_ERR_INVALID_ARG, "q, k and v must be 16-byte aligned");
        if (!aligned4(a->cu_seqlens_q) || !aligned4(a->cu_seqlens_k) || !aligned4(a->pos_q) || !aligned4(a->pos_k) ||
            !aligned4(a->buckets) || !aligned4(a->lse))
            return fail(RAGGED_ERR_INVALID_ARG, "cu_seqlens, positions, buckets and lse must be 4-byte aligned");
        if (reinterpret_cast<uintptr_t>(a->table) & 1u)
            return fail(RAGGED_ERR_INVALID_ARG, "table must be 2-byte aligned");
        ragged_status st = check_stride16(a->q_tok_stride, "q_tok_stride");
        if (st == RAGGED_OK) st = check_stride16(a->kv_tok_stride, "kv_tok_stride");
        if (st == RAGGED_OK && a->H > 1) st = check_stride16(a->q_head_stride, "q_head_stride");
        if (st == RAGGED_OK && a->Hkv > 1) st = check_stride16(a->kv_head_stride, "kv_head_stride");
        if (st != RAGGED_OK) return st;
        if (a->lse_stride < 0) return fail(RAGGED_ERR_INVALID_ARG, "lse_stride is negative");
    }
    *p = ragged::bias::Problem{
        static_cast<const uint16_t*>(a->q), static_cast<const uint16_t*>(a->k), static_cast<const uint16_t*>(a->v),
        a->q_tok_stride, a->H > 1 ? a->q_head_stride : 0, a->kv_tok_stride, a->Hkv > 1 ? a->kv_head_stride : 0,
        a->cu_seqlens_q, a->cu_seqlens_k, a->pos_q, a->pos_k, static_cast<const uint16_t*>(a->table), a->buckets,
        a->lse, a->lse_stride, static_cast<int>(a->B), static_cast<int>(a->max_seqlen_q), static_cast<int>(a->max_seqlen_k),
        static_cast<int>(a->H), static_cast<int>(a->Hkv), static_cast<int>(a->H / a->Hkv),
        static_cast<int>(a->num_buckets), static_cast<int>(a->max_distance), a->scale, a->scale * ragged::bias::kLog2e};
    return RAGGED_OK;
}

int64_t tiles128(int64_t n) { return (n + ragged::bias::kQTile - 1) / ragged::bias::kQTile; }

// Average length of B sequences of at most `longest` rows: `rows`, the row
// count that a caller's stride implies, where it says less than B * longest.
int64_t average_length(int64_t B, int64_t longest, int64_t rows) {
    return B == 0 ? 1 : std::max<int64_t>(1, (std::min(B * longest, std::max<int64_t>(rows, B)) + B - 1) / B);
}

// Parts that a key row's queries are split into, where key tiles and heads
// alone leave SMs without work and each CTA has many query tiles to walk.  (2
// sequences of 3,279 to 4,099, 8 over 2 heads: 223 + 5 us for the key rows and
// the parts' sum, 341 us in one part, each kernel timed by itself.)
int64_t bwd_parts(const ragged_bias_attn* a) {
    const int64_t avg_q = average_length(a->B, a->max_seqlen_q, a->lse_stride);
    const int64_t avg_k = std::max<int64_t>(1, a->max_seqlen_k * avg_q / a->max_seqlen_q);
    const int64_t ctas = std::max<int64_t>(1, a->B * tiles128(avg_k) * a->Hkv);
    const int64_t tiles = (avg_q + ragged::bias::kTile - 1) / ragged::bias::kTile;
    return std::max<int64_t>(1, std::min<int64_t>({8, 2LL * sm_count() / ctas, tiles / 4, tiles * (a->H / a->Hkv) / 16}));
}
// Workspace of the backward pass: delta and the far rows' sums [H, lse_stride] floats, four exponents per
// (sequence, head, query tile), the tiles' sums for the table's gradient
// [H, num_buckets, B, query tiles], an exponent per (sequence, key head, key tile),
// and the parts' sums of dK and dV.
int64_t bwd_delta_floats(const ragged_bias_attn* a) { return (a->H * a->lse_stride + 3) & ~int64_t(3); }
int64_t bwd_items(const ragged_bias_attn* a) { return a->B * a->H * tiles128(a->max_seqlen_q); }
int64_t bwd_small_floats(const ragged_bias_attn* a) {
    return (2 * bwd_delta_floats(a) + bwd_items(a) * (4 + a->num_buckets) + a->B * a->Hkv * tiles128(a->max_seqlen_k) + 3) & ~int64_t(3);
}
int64_t bwd_workspace(const ragged_bias_attn* a) {
    const int64_t parts = bwd_parts(a);
    return 4 * (bwd_small_floats(a) + (parts == 1 ? 0 : parts * a->B * tiles128(a->max_seqlen_k) * ragged::bias::kQTile * a->Hkv * 128));
}
int64_t fwd_workspace(const ragged_bias_attn*) { return 0; }

// Positions that a kernel's expanded table covers: what two CTAs per SM leave
// room for next to `fixed` bytes, unless that is too little to be of use (many
// buckets, or a far-reaching map): then one CTA.  (64 sequences of 173 to 403
// tokens, D = 512, where two CTAs leave 150 positions: 118 us either way.)
constexpr int kTwoPerSm = 114 * 1024 - 1024 - 3 * 1024;   // less the reserved and the static part
constexpr int bias_span(int D, int fixed, int bytes_per_entry) {
    const int entries = (kTwoPerSm - fixed - 64 - (2 * D + 16)) / bytes_per_entry;
    const int span = (entries - 1 - ragged::bias::kVecPad) / 2 - D;
    return span < 256 ? ragged::bias::kSpan : span < ragged::bias::kSpan ? span : ragged::bias::kSpan;
}
constexpr int kBwdQSmemMax = ragged::bias::bwd_q_smem_bytes(ragged::bias::kMaxDistance, ragged::bias::kMaxBuckets, ragged::bias::kSpan);

ragged_status check_workspace(const void* ws, int64_t have, int64_t need) {
    if (need > 0 && (ws == nullptr || have < need))
        return fail(RAGGED_ERR_INVALID_ARG, "the workspace holds %lld bytes, %lld are needed", (long long)(ws ? have : 0),
                    (long long)need);
    if (need > 0 && !aligned16(ws)) return fail(RAGGED_ERR_INVALID_ARG, "the workspace must be 16-byte aligned");
    return RAGGED_OK;
}

DeviceFlags g_bias_fwd_smem[2], g_bias_bwd_q_smem[2][2], g_bias_bwd_kv_smem[2], g_bias_weight_smem[2];
template <typename T>
constexpr int kTypeSlot = std::is_same<T, __half>::value ? 0 : 1;

dim3 bias_grid(int64_t tiles, int heads, int B) {
    return dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(heads), static_cast<unsigned>(B));
}

// Heads that one CTA walks over: the number with the least time, in units of a
// tile's, of a grid of `row_tiles` per head over `slots` CTAs at a time.  A CTA's
// set-up costs about kSetup tiles, a head's start and end kHead; half a wave
// stands for the uneven end.  The costs are the forward kernel's; the gradient
// kernels' heads cost four times that, and weigh more the more a CTA has of
// them, which this rule does not see.  (Forward, 64 sequences of 173 to 403 tokens, 12
// heads: 118, 112, 109, 119, 127, 141 us with 1, 2, 3, 4, 6, 12 heads; 512 of 79
// to 118, 6 heads: 86, 74, 70, 88, 65 us with 1, 2, 3, 4, 6.)
int heads_per_cta(int64_t row_tiles, int64_t heads, int64_t col_tiles, int64_t slots) {
    constexpr double kSetup = 4, kHead = 1;
    constexpr int64_t kMost = 64;   // the set-up is then a 16th of a tile's time per head
    int best = 1;
    double best_cost = 1e300;
    for (int n = 1; n <= std::min<int64_t>(heads, kMost); ++n) {
        const double waves = static_cast<double>(row_tiles * ((heads + n - 1) / n)) / static_cast<double>(slots);
        const double cost = (std::max(1.0, waves) + 0.5) * (kSetup + n * (kHead + static_cast<double>(col_tiles)));
        if (cost < best_cost) {
            best_cost = cost;
            best = n;
        }
    }
    return best;
}

// Few query rows per key / value head go to the kernels that share one 16- or
// 32-row MMA tile among them: the 128-row tiles would be mostly empty, and
// read the keys once per query head.  (32 sequences of 4,096 to 8,192 keys, 16
// over 4 heads, 4 and 8 queries, so 16 and 32 rows: 42 and 68 us, against 205
// us either way; weights of 32 rows 78 against 184.  More rows do not fit these
// kernels' registers.)
bool few_rows(const ragged::bias::Problem& p) {
    return static_cast<int64_t>(p.group) * p.max_q <= ragged::bias::kFewMaxRows;
}
// CTAs per (sequence, key / value head): what one wave of `per_sm` per SM holds,
// each with at least one block of keys per warp.
int few_splits(const ragged::bias::Problem& p, int per_sm, int warps, int limit) {
    const int64_t base = static_cast<int64_t>(p.B) * p.Hkv, want = static_cast<int64_t>(per_sm) * sm_count() / base;
    const int64_t keys = static_cast<int64_t>(ragged::bias::kFewKeys) * warps;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, (p.max_k + keys - 1) / keys), limit)));
}
DeviceFlags g_few_smem[2][2][2], g_few_weight_smem[2][2][2];

template <typename T, int MT, int NW>
ragged_status launch_few(const ragged::bias::Problem& p, uint16_t* out, int64_t out_tok, cudaStream_t s) {
    using namespace ragged::bias;
    auto kernel = bias_few_kernel<T, MT, NW>;
    ragged_status st = ensure_smem(kernel, few_smem_bytes<MT, NW, false>(kMaxDistance, kMaxBuckets),
                                   g_few_smem[kTypeSlot<T>][MT - 1][NW == kFewWarps]);
    if (st != RAGGED_OK) return st;
    int splits = few_splits(p, NW == kFewWarps ? 2 : 4, NW, kFewMaxSplits);
    while (splits & (splits - 1)) splits &= splits - 1;   // cluster sizes are powers of two
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = bias_grid(splits, p.Hkv, p.B);
    cfg.blockDim = dim3(32 * NW);
    cfg.dynamicSmemBytes = few_smem_bytes<MT, NW, false>(p.D, p.num_buckets);
    cfg.stream = s;
    cudaLaunchAttribute cluster{};
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = static_cast<unsigned>(splits);
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    cfg.attrs = &cluster;
    cfg.numAttrs = splits > 1 ? 1 : 0;
    return cuda_check(cudaLaunchKernelEx(&cfg, kernel, p, out, out_tok), "attention (few rows) launch");
}
template <typename T, int MT, int NW>
ragged_status launch_few_weight(const ragged::bias::Problem& p, const float* prev, float* weight, int64_t stride, cudaStream_t s) {
    using namespace ragged::bias;
    auto kernel = bias_few_weight_kernel<T, MT, NW>;
    ragged_status st = ensure_smem(kernel, few_smem_bytes<MT, NW, true>(kMaxDistance, kMaxBuckets),
                                   g_few_weight_smem[kTypeSlot<T>][MT - 1][NW == kFewWarps]);
    if (st != RAGGED_OK) return st;
    const int splits = few_splits(p, NW == kFewWarps ? 2 : 8, NW, 1 << 16);
    kernel<<<bias_grid(splits, p.Hkv, p.B), 32 * NW, few_smem_bytes<MT, NW, true>(p.D, p.num_buckets), s>>>(p, prev, weight, stride);
    return cuda_check(cudaGetLastError(), "attention weight (few rows) launch");
}
// Two warps per CTA instead of eight where there are more groups than one wave
// of eight warps (two CTAs per SM) holds, the more the longer they are.
// (Attention of one query, 16 over 4 heads, with two and with eight warps: 296
// groups of up to 128 keys 11.6 and 7.2 us; 400 of up to 60 9.9 and 11.1, of up
// to 128 12.8 and 11.9, of up to 512 20 and 17; 1,024 of up to 128 15 and 22, of
// up to 512 29 and 35, of up to 1,024 47 and 47, of up to 2,048 77 and 72.)
bool few_short(const ragged::bias::Problem& p) {
    const int64_t groups = static_cast<int64_t>(p.B) * p.Hkv, wave = 2LL * sm_count();
    return groups > wave && p.max_k <= ragged::bias::kFewShortKeys && p.max_k * wave <= 160 * groups;
}
// By rows (one or two MMA tiles), and by the number and length of the sequences.
template <typename T>
ragged_status launch_few_rows(const ragged::bias::Problem& p, uint16_t* out, int64_t out_tok, cudaStream_t s) {
    using namespace ragged::bias;
    const bool one = p.group * p.max_q <= 16;
    if (few_short(p))
        return one ? launch_few<T, 1, kFewShortWarps>(p, out, out_tok, s) : launch_few<T, 2, kFewShortWarps>(p, out, out_tok, s);
    return one ? launch_few<T, 1, kFewWarps>(p, out, out_tok, s) : launch_few<T, 2, kFewWarps>(p, out, out_tok, s);
}
template <typename T>
ragged_status launch_few_rows_weight(const ragged::bias::Problem& p, const float* prev, float* weight, int64_t stride, cudaStream_t s) {
    using namespace ragged::bias;
    const bool one = p.group * p.max_q <= 16;
    if (few_short(p))
        return one ? launch_few_weight<T, 1, kFewShortWarps>(p, prev, weight, stride, s)
                   : launch_few_weight<T, 2, kFewShortWarps>(p, prev, weight, stride, s);
    return one ? launch_few_weight<T, 1, kFewWarps>(p, prev, weight, stride, s) : launch_few_weight<T, 2, kFewWarps>(p, prev, weight, stride, s);
}

template <typename T>
ragged_status launch_bias_fwd(const ragged::bias::Problem& p, uint16_t* out, int64_t out_tok, cudaStream_t s) {
    using namespace ragged::bias;
    if (few_rows(p)) return launch_few_rows<T>(p, out, out_tok, s);
    ragged_status st = ensure_smem(bias_fwd_kernel<T>, fwd_smem_bytes(kMaxDistance, kSpan), g_bias_fwd_smem[kTypeSlot<T>]);
    if (st != RAGGED_OK) return st;
    const int span = bias_span(p.D, fwd_fixed_bytes(), 5);
    const int64_t tiles = tiles128(p.max_q);
    const int64_t avg_q = average_length(p.B, p.max_q, p.lse_stride), avg_k = std::max<int64_t>(1, p.max_k * avg_q / p.max_q);
    const int heads = heads_per_cta(p.B * tiles128(avg_q), p.H, (avg_k + kTile - 1) / kTile, 2LL * sm_count());
    bias_fwd_kernel<T><<<bias_grid(tiles, (p.H + heads - 1) / heads, p.B), kThreads, fwd_smem_bytes(p.D, span), s>>>(
        p, out, out_tok, heads, span);
    return cuda_check(cudaGetLastError(), "attention (position bias) launch");
}

template <typename T>
ragged_status launch_bias_bwd(const ragged::bias::Problem& p, ragged::bias::BwdArgs a, cudaStream_t s) {
    using namespace ragged::bias;
    const bool one = p.max_k <= kTile;   // every row's keys are in one tile
    auto q_kernel = one ? bias_bwd_q_kernel<T, true> : bias_bwd_q_kernel<T, false>;
    ragged_status st = ensure_smem(q_kernel, kBwdQSmemMax, g_bias_bwd_q_smem[kTypeSlot<T>][one]);
    if (st == RAGGED_OK) st = ensure_smem(bias_bwd_kv_kernel<T>, bwd_kv_smem_bytes(kMaxDistance, kSpan), g_bias_bwd_kv_smem[kTypeSlot<T>]);
    if (st != RAGGED_OK) return st;
    const int64_t avg_q = average_length(p.B, p.max_q, p.lse_stride), avg_k = std::max<int64_t>(1, p.max_k * avg_q / p.max_q);
    const int64_t slots = 2LL * sm_count();
    a.span = bias_span(p.D, bwd_q_fixed_bytes(p.num_buckets), 3);
    a.heads = heads_per_cta(p.B * tiles128(avg_q), p.H, (avg_k + kTile - 1) / kTile, slots);
    cudaLaunchAttribute early{};   // the kernel may start before the one ahead of it has ended, and waits for it itself
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kBwdThreads);
    cfg.stream = s;
    cfg.attrs = &early;
    if (kScaled<T>) {
        bias_bwd_value_kernel<T><<<bias_grid(a.k_tiles, p.Hkv, p.B), 256, 0, s>>>(p, a);
        st = cuda_check(cudaGetLastError(), "value exponent launch");
        if (st != RAGGED_OK) return st;
        cfg.numAttrs = 1;
    }
    cfg.gridDim = bias_grid(a.q_tiles, (p.H + a.heads - 1) / a.heads, p.B);
    cfg.dynamicSmemBytes = bwd_q_smem_bytes(p.D, p.num_buckets, a.span);
    st = cuda_check(cudaLaunchKernelEx(&cfg, q_kernel, p, a), "query gradient launch");
    if (st != RAGGED_OK) return st;
    a.span = bias_span(p.D, bwd_kv_fixed_bytes(), 3);
    a.heads = a.parts > 1 ? 1 : heads_per_cta(p.B * tiles128(avg_k), p.Hkv, (avg_q + kTile - 1) / kTile * p.group, slots);
    // The table's sums go to CTAs of this launch where a column or a slice of its
    // grid has enough of them (32,768 values each) and not too many: 28 instead of
    // 31 us for 4 sequences of 79 to 197 tokens; 462 instead of 299 us where few
    // CTAs had to sum for 352 short ones.
    const int64_t columns = tiles128(p.max_k) * a.parts, groups = (p.Hkv + a.heads - 1) / a.heads;
    const int64_t values = static_cast<int64_t>(p.num_buckets) * p.H * p.B * a.q_tiles, most = std::max<int64_t>(32, columns * groups * p.B / 16);
    auto fits = [&](int64_t ctas) { return ctas * 32768 >= values && ctas <= most; };
    a.table_in = p.B < 65535 && fits(columns * groups) ? kSlice : fits(groups * p.B) ? kColumn : kOwnLaunch;
    cfg.gridDim = bias_grid(columns + (a.table_in == kColumn), static_cast<int>(groups), p.B + (a.table_in == kSlice));
    cfg.dynamicSmemBytes = bwd_kv_smem_bytes(p.D, a.span);
    cfg.numAttrs = 1;
    st = cuda_check(cudaLaunchKernelEx(&cfg, bias_bwd_kv_kernel<T>, p, a), "key and value gradient launch");
    if (st == RAGGED_OK && a.table_in == kOwnLaunch) {
        bias_bwd_table_kernel<T><<<static_cast<unsigned>((p.num_buckets * static_cast<int64_t>(p.H) + 7) / 8), 256, 0, s>>>(p, a);
        st = cuda_check(cudaGetLastError(), "table gradient launch");
    }
    if (st != RAGGED_OK || a.parts == 1) return st;
    const int64_t blocks = std::min<int64_t>((static_cast<int64_t>(p.max_k) * p.Hkv * 16 + 255) / 256, 8LL * sm_count());
    bias_bwd_parts_kernel<T><<<dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(p.B)), 256, 0, s>>>(p, a);
    return cuda_check(cudaGetLastError(), "key and value gradient sum launch");
}

template <typename T>
ragged_status launch_bias_weight(const ragged::bias::Problem& p, const float* prev, float* weight, int64_t stride,
                                 cudaStream_t s) {
    using namespace ragged::bias;
    if (few_rows(p)) return launch_few_rows_weight<T>(p, prev, weight, stride, s);
    ragged_status st = ensure_smem(bias_weight_kernel<T>, weight_smem_bytes(kMaxDistance, kSpan), g_bias_weight_smem[kTypeSlot<T>]);
    if (st != RAGGED_OK) return st;
    const int64_t avg_q = average_length(p.B, p.max_q, p.lse_stride), avg_k = std::max<int64_t>(1, p.max_k * avg_q / p.max_q);
    const int heads = heads_per_cta(p.B * tiles128(avg_k), p.H, (avg_q + kTile - 1) / kTile, 3LL * sm_count());
    bias_weight_kernel<T><<<bias_grid(tiles128(p.max_k), (p.H + heads - 1) / heads, p.B), kThreads, weight_smem_bytes(p.D, kSpan), s>>>(
        p, prev, weight, stride, heads, kSpan);
    return cuda_check(cudaGetLastError(), "attention weight launch");
}

// Products of up to 64 factors below 2^16, compared in whole numbers.
struct BigUint {
    uint32_t w[72] = {1};
    int n = 1;
    void times(uint32_t f) {
        uint64_t carry = 0;
        for (int i = 0; i < n; ++i) {
            carry += static_cast<uint64_t>(w[i]) * f;
            w[i] = static_cast<uint32_t>(carry);
            carry >>= 32;
        }
        if (carry) w[n++] = static_cast<uint32_t>(carry);
    }
    bool at_least(const BigUint& o) const {
        if (n != o.n) return n > o.n;
        for (int i = n - 1; i >= 0; --i)
            if (w[i] != o.w[i]) return w[i] > o.w[i];
        return true;
    }
};

}  // namespace

extern "C" {

ragged_status ragged_rel_buckets(int64_t num_buckets, int64_t max_distance, int32_t bidirectional, int32_t* host_out) {
    if (num_buckets < 1 || num_buckets > ragged::bias::kMaxBuckets)
        return fail(RAGGED_ERR_UNSUPPORTED, "num_buckets = %lld outside [1, %d]", (long long)num_buckets,
                    ragged::bias::kMaxBuckets);
    if (max_distance < 0 || max_distance > ragged::bias::kMaxDistance)
        return fail(RAGGED_ERR_UNSUPPORTED, "max_distance = %lld outside [0, %d]", (long long)max_distance,
                    ragged::bias::kMaxDistance);
    if (bidirectional && num_buckets % 2)
        return fail(RAGGED_ERR_INVALID_ARG, "num_buckets = %lld must be even for both directions", (long long)num_buckets);
    if (host_out == nullptr) return fail(RAGGED_ERR_INVALID_ARG, "host_out is NULL");
    const int n = static_cast<int>(bidirectional ? num_buckets / 2 : num_buckets), D = static_cast<int>(max_distance);
    const int exact = n / 2, m = n - exact;
    for (int delta = -D; delta <= D; ++delta) {
        const int d = bidirectional ? (delta < 0 ? -delta : delta) : (delta < 0 ? -delta : 0);
        int b;
        if (n == 1) {
            b = 0;
        } else if (d < exact) {
            b = d;
        } else if (exact >= D) {   // no room for a logarithmic part
            b = d < n - 1 ? d : n - 1;
        } else {
            // exact + the largest k <= m with (D / exact)^k <= (d / exact)^m
            int k = 0;
            while (k < m) {
                BigUint lhs, rhs;
                for (int i = 0; i <= k; ++i) lhs.times(static_cast<uint32_t>(D));
                for (int i = 0; i < m; ++i) lhs.times(static_cast<uint32_t>(exact));
                for (int i = 0; i < m; ++i) rhs.times(static_cast<uint32_t>(d));
                for (int i = 0; i <= k; ++i) rhs.times(static_cast<uint32_t>(exact));
                if (!rhs.at_least(lhs)) break;
                ++k;
            }
            b = exact + k < n - 1 ? exact + k : n - 1;
        }
        host_out[delta + D] = b + (bidirectional && delta > 0 ? n : 0);
    }
    return RAGGED_OK;
}

ragged_status ragged_attn_bias_fwd_workspace(const ragged_bias_attn* a, int64_t* bytes) {
    ragged::bias::Problem p;
    if (bytes == nullptr) return fail(RAGGED_ERR_INVALID_ARG, "bytes is NULL");
    ragged_status st = check_bias_problem(a, true, &p);
    if (st != RAGGED_OK) return st;
    *bytes = fwd_workspace(a);
    return RAGGED_OK;
}

ragged_status ragged_attn_bias_fwd(const ragged_bias_attn* a, void* out, int64_t out_tok_stride, void* workspace,
                                   int64_t workspace_bytes, void* stream) {
    ragged::bias::Problem p;
    ragged_status st = check_bias_problem(a, true, &p);
    if (st != RAGGED_OK || a->B == 0) return st;
    if (out == nullptr) return fail(RAGGED_ERR_INVALID_ARG, "out must not be NULL");
    if (!aligned16(out)) return fail(RAGGED_ERR_INVALID_ARG, "out must be 16-byte aligned");
    if (out_tok_stride < a->H * 64 || out_tok_stride % 8)
        return fail(RAGGED_ERR_INVALID_ARG, "out_tok_stride must be >= H * head_dim and a multiple of 16 bytes");
    st = check_workspace(workspace, workspace_bytes, fwd_workspace(a));
    if (st != RAGGED_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return a->dtype == RAGGED_F16 ? launch_bias_fwd<__half>(p, static_cast<uint16_t*>(out), out_tok_stride, s)
                                  : launch_bias_fwd<__nv_bfloat16>(p, static_cast<uint16_t*>(out), out_tok_stride, s);
}

ragged_status ragged_attn_bias_bwd_workspace(const ragged_bias_attn* a, int64_t* bytes) {
    ragged::bias::Problem p;
    if (bytes == nullptr) return fail(RAGGED_ERR_INVALID_ARG, "bytes is NULL");
    ragged_status st = check_bias_problem(a, true, &p);
    if (st != RAGGED_OK) return st;
    *bytes = bwd_workspace(a);
    return RAGGED_OK;
}

ragged_status ragged_attn_bias_bwd(const ragged_bias_attn* a, const void* out, int64_t out_tok_stride, const void* dout,
                                   int64_t dout_tok_stride, void* dq, int64_t dq_tok_stride, int64_t dq_head_stride,
                                   void* dk, void* dv, int64_t dkv_tok_stride, int64_t dkv_head_stride, void* dtable,
                                   void* workspace, int64_t workspace_bytes, void* stream) {
    ragged::bias::Problem p;
    ragged_status st = check_bias_problem(a, true, &p);
    if (st != RAGGED_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtable == nullptr || (reinterpret_cast<uintptr_t>(dtable) & 1u))
        return fail(RAGGED_ERR_INVALID_ARG, "dtable must be a 2-byte aligned device pointer");
    if (a->B == 0)
        return cuda_check(cudaMemsetAsync(dtable, 0, static_cast<size_t>(a->num_buckets * a->H * 2), s), "cudaMemsetAsync");
    if (!out || !dout || !dq || !dk || !dv)
        return fail(RAGGED_ERR_INVALID_ARG, "out, dout, dq, dk and dv must not be NULL");
    if (!aligned16(out) || !aligned16(dout) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
        return fail(RAGGED_ERR_INVALID_ARG, "out, dout, dq, dk and dv must be 16-byte aligned");
    if (out_tok_stride < a->H * 64 || out_tok_stride % 8 || dout_tok_stride < a->H * 64 || dout_tok_stride % 8)
        return fail(RAGGED_ERR_INVALID_ARG, "out_tok_stride and dout_tok_stride must be >= H * head_dim and multiples of 16 bytes");
    st = check_stride16(dq_tok_stride, "dq_tok_stride");
    if (st == RAGGED_OK) st = check_stride16(dkv_tok_stride, "dkv_tok_stride");
    if (st == RAGGED_OK && a->H > 1) st = check_stride16(dq_head_stride, "dq_head_stride");
    if (st == RAGGED_OK && a->Hkv > 1) st = check_stride16(dkv_head_stride, "dkv_head_stride");
    if (st == RAGGED_OK) st = check_workspace(workspace, workspace_bytes, bwd_workspace(a));
    if (st != RAGGED_OK) return st;
    float* ws = static_cast<float*>(workspace);
    ragged::bias::BwdArgs g{};
    g.out = static_cast<const uint16_t*>(out);
    g.dout = static_cast<const uint16_t*>(dout);
    g.out_tok = out_tok_stride;
    g.dout_tok = dout_tok_stride;
    g.dq = static_cast<uint16_t*>(dq);
    g.dk = static_cast<uint16_t*>(dk);
    g.dv = static_cast<uint16_t*>(dv);
    g.dq_tok = dq_tok_stride;
    g.dq_head = a->H > 1 ? dq_head_stride : 0;
    g.dkv_tok = dkv_tok_stride;
    g.dkv_head = a->Hkv > 1 ? dkv_head_stride : 0;
    g.delta = ws;
    g.log_sum = ws + bwd_delta_floats(a);
    g.tile_exp = reinterpret_cast<int*>(ws + 2 * bwd_delta_floats(a));
    g.partial = ws + 2 * bwd_delta_floats(a) + 4 * bwd_items(a);
    g.v_exp = reinterpret_cast<int*>(g.partial + bwd_items(a) * a->num_buckets);
    g.k_tiles = static_cast<int>(tiles128(a->max_seqlen_k));
    g.dtable = static_cast<uint16_t*>(dtable);
    g.q_tiles = static_cast<int>(tiles128(a->max_seqlen_q));
    g.parts = static_cast<int>(bwd_parts(a));
    g.part_sums = ws + bwd_small_floats(a);
    g.part_rows = tiles128(a->max_seqlen_k) * ragged::bias::kQTile;
    return a->dtype == RAGGED_F16 ? launch_bias_bwd<__half>(p, g, s) : launch_bias_bwd<__nv_bfloat16>(p, g, s);
}

ragged_status ragged_attn_weight(const ragged_bias_attn* a, const float* prev, float* weight, int64_t weight_stride,
                                 void* stream) {
    ragged::bias::Problem p;
    ragged_status st = check_bias_problem(a, false, &p);
    if (st != RAGGED_OK || a->B == 0) return st;
    if (weight == nullptr || !aligned4(weight) || !aligned4(prev))
        return fail(RAGGED_ERR_INVALID_ARG, "weight must not be NULL; weight and prev must be 4-byte aligned");
    if (weight_stride < 0) return fail(RAGGED_ERR_INVALID_ARG, "weight_stride is negative");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return a->dtype == RAGGED_F16 ? launch_bias_weight<__half>(p, prev, weight, weight_stride, s)
                                  : launch_bias_weight<__nv_bfloat16>(p, prev, weight, weight_stride, s);
}

ragged_status ragged_evict(const void* rows, int64_t row_bytes, const float* weight, int64_t weight_stride, int64_t H,
                           int64_t tokens, const int32_t* cu_seqlens, int64_t B, int64_t max_seqlen,
                           const int32_t* budget, int64_t sinks, int64_t recents, const int32_t* pos, int64_t capacity,
                           void* rows_out, int32_t* cu_out, int32_t* src_idx, float* weight_out,
                           int64_t weight_out_stride, int32_t* pos_out, void* workspace, int64_t workspace_bytes,
                           void* stream) {
    if (B < 0) return fail(RAGGED_ERR_INVALID_ARG, "B = %lld is negative", (long long)B);
    if (B > 65535) return fail(RAGGED_ERR_UNSUPPORTED, "B = %lld exceeds 65535", (long long)B);
    if (H < 1 || H > 65534) return fail(RAGGED_ERR_INVALID_ARG, "H = %lld outside [1, 65534]", (long long)H);
    if (max_seqlen < 1 || max_seqlen > RAGGED_MAX_TOKENS)
        return fail(RAGGED_ERR_INVALID_ARG, "max_seqlen = %lld outside [1, %d]", (long long)max_seqlen, RAGGED_MAX_TOKENS);
    if (sinks < 0 || recents < 0 || sinks > RAGGED_MAX_TOKENS || recents > RAGGED_MAX_TOKENS)
        return fail(RAGGED_ERR_INVALID_ARG, "sinks and recents must lie in [0, %d]", RAGGED_MAX_TOKENS);
    if (tokens < 0 || tokens >= (int64_t(1) << 31))
        return fail(RAGGED_ERR_INVALID_ARG, "tokens = %lld outside [0, 2^31)", (long long)tokens);
    if (capacity < 0 || capacity >= (int64_t(1) << 31))
        return fail(RAGGED_ERR_INVALID_ARG, "capacity = %lld outside [0, 2^31)", (long long)capacity);
    if (cu_out == nullptr || !aligned4(cu_out)) return fail(RAGGED_ERR_INVALID_ARG, "cu_out must be a 4-byte aligned device pointer");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (B == 0) return cuda_check(cudaMemsetAsync(cu_out, 0, sizeof(int32_t), s), "cudaMemsetAsync");
    if (!weight || !cu_seqlens || !budget || (capacity > 0 && !src_idx))
        return fail(RAGGED_ERR_INVALID_ARG, "weight, cu_seqlens, budget and src_idx must not be NULL");
    if ((rows == nullptr) != (rows_out == nullptr))
        return fail(RAGGED_ERR_INVALID_ARG, "rows and rows_out must both be given or both be NULL");
    if (rows != nullptr) {
        if (row_bytes <= 0 || row_bytes % 16 || row_bytes / 16 >= (int64_t(1) << 31))
            return fail(RAGGED_ERR_INVALID_ARG, "row_bytes = %lld must be a positive multiple of 16", (long long)row_bytes);
        if (!aligned16(rows) || !aligned16(rows_out))
            return fail(RAGGED_ERR_INVALID_ARG, "rows and rows_out must be 16-byte aligned");
        if (rows == rows_out) return fail(RAGGED_ERR_INVALID_ARG, "rows_out must not be rows");
    }
    if (!aligned4(weight) || !aligned4(cu_seqlens) || !aligned4(budget) || !aligned4(pos) || !aligned4(src_idx) ||
        !aligned4(weight_out) || !aligned4(pos_out))
        return fail(RAGGED_ERR_INVALID_ARG, "weights, cu_seqlens, budget, positions and src_idx must be 4-byte aligned");
    if (weight_out == weight || cu_out == cu_seqlens || (pos != nullptr && pos_out == pos))
        return fail(RAGGED_ERR_INVALID_ARG, "the outputs must not be the inputs");
    if (weight_stride < 0 || weight_out_stride < 0 || (weight_out != nullptr && H > 1 && weight_out_stride < capacity))
        return fail(RAGGED_ERR_INVALID_ARG, "weight strides are too small");
    using namespace ragged::evict;
    const bool one_launch = max_seqlen <= kShortLen;
    ragged_status st = check_workspace(workspace, workspace_bytes, one_launch ? 0 : 4 * tokens);
    if (st != RAGGED_OK) return st;
    Args a{weight, weight_stride, cu_seqlens, budget, pos, static_cast<int>(B), static_cast<int>(H),
           static_cast<int>(max_seqlen), static_cast<int>(sinks), static_cast<int>(recents), capacity, cu_out, src_idx,
           pos_out, capacity > 0 ? weight_out : nullptr, weight_out_stride, static_cast<const uint4*>(rows),
           static_cast<uint4*>(rows_out), static_cast<uint32_t>(rows ? row_bytes / 16 : 0),
           static_cast<uint32_t*>(workspace), tokens};
    if (capacity == 0) a.rows = nullptr;
    if (one_launch) {
        // A few CTAs per sequence where there are few sequences: the selection is
        // short enough to be repeated, the rows are shared out.
        const int64_t splits = std::max<int64_t>(1, std::min<int64_t>(4LL * sm_count() / B, (max_seqlen + 15) / 16));
        short_kernel<<<dim3(static_cast<unsigned>(splits), static_cast<unsigned>(B)), kShortThreads, 0, s>>>(a);
        return cuda_check(cudaGetLastError(), "evict launch");
    }
    keys_kernel<<<dim3(static_cast<unsigned>((max_seqlen + 255) / 256), static_cast<unsigned>(B)), 256, 0, s>>>(a);
    st = cuda_check(cudaGetLastError(), "evict key launch");
    if (st != RAGGED_OK) return st;
    long_kernel<<<static_cast<unsigned>(B), kLongThreads, 0, s>>>(a);
    st = cuda_check(cudaGetLastError(), "evict selection launch");
    if (st != RAGGED_OK || (a.rows == nullptr && a.weight_out == nullptr)) return st;
    const dim3 grid(static_cast<unsigned>((capacity + kCopyThreads - 1) / kCopyThreads),
                    static_cast<unsigned>(a.weight_out ? 1 + H : 1));
    copy_kernel<<<grid, kCopyThreads, 0, s>>>(a);
    return cuda_check(cudaGetLastError(), "evict copy launch");
}

}  // extern "C"
