// C ABI of the paged cache (sigattn_cache_append, sigattn_fwd_paged in
// include/sigattn.h).
#include <algorithm>
#include <cmath>

#include "host.cuh"
#include "paged_fp32.cuh"

namespace {

using namespace sigattn;

// log2 of a page size the kernels take (a power of two from 16 to 256), or -1.
int page_shift_of(int page_size) {
    for (int s = 4; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

struct CacheShape {
    int Z, L, H, Hk, D, pages, page_size, max_pages, prefix_pages;
    sigattn_dtype dtype;
};

// H may be 0 (no queries) only when `queries` is false.
sigattn_status check_cache(const CacheShape &c, bool queries, bool *empty) {
    if (c.Z < 0 || c.L < 0 || c.H < 0 || c.Hk < 0 || c.pages < 0 || c.max_pages < 0 || c.prefix_pages < 0)
        return SIGATTN_ERR_INVALID_ARG;
    if (c.D != 64 && c.D != 128) return SIGATTN_ERR_UNSUPPORTED_HEADDIM;
    if (c.dtype != SIGATTN_BF16 && c.dtype != SIGATTN_FP32) return SIGATTN_ERR_UNSUPPORTED_DTYPE;
    const int shift = page_shift_of(c.page_size);
    if (shift < 0) return SIGATTN_ERR_INVALID_ARG;
    *empty = c.Z == 0 || c.L == 0 || (queries && c.H == 0);
    if (*empty) return SIGATTN_OK;
    if (c.Hk == 0 || c.H % c.Hk != 0) return SIGATTN_ERR_INVALID_ARG;
    // places are int32, and the work of a call is counted in 32 bits
    const int64_t most = int64_t(INT_MAX) - 4096;
    const int64_t own = static_cast<int64_t>(c.max_pages) << shift, ahead = static_cast<int64_t>(c.prefix_pages) << shift;
    if (own + ahead > most || static_cast<int64_t>(c.Z) * c.L > most || c.H > 65535 || c.Hk > 65535)
        return SIGATTN_ERR_TOO_LARGE;
    return SIGATTN_OK;
}

// Row warps (1, 2 or 4, 16 rows each) of a tile over `rows` query rows.
int row_warps(int64_t rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }

constexpr int kPagedMostSms = 256;                   // more than any device has
constexpr int kPagedMostBlocks = 3 * kPagedMostSms;  // of the tile kernel

// Rows (over the batch, per key head) above which the prefix kernel takes the
// prefix. The tile kernel's row tile is 64 rows, the prefix kernel's 256: up to 64
// rows the tile kernel reads the prefix once as well and needs no further launch
// (whole call, a prefix of 16K tokens: 32 rows 18.1 us against 21.7 with the prefix
// kernel, 64 rows 24.7 against 25.6); above, it would read the prefix again for every
// 64 rows (128 rows 33.6 us against 27.4, 256 rows 57.0 against 39.3).
constexpr int64_t kPrefixKernelRows = 64;

// Rows of the output up to which a row's partials are added by 8, 4 or 2 warps.
// Few rows leave most of the SMs empty with a warp a row (1024 rows, whole call:
// 8 warps 35.6 us, 4 warps 37.2, 2 warps 40.9, 1 warp 44.5); many rows fill them
// without the exchange through shared memory. Each limit is about 1, 2 and 2
// waves of such blocks on 148 SMs.
constexpr int64_t kJoin8Rows = 2048, kJoin4Rows = 8192, kJoin2Rows = 16384;

struct PagedSizes {
    int prefix_warps, own_warps;
    int64_t prefix_rt, own_rt;     // row tiles per key head: of the prefix, of a sample
    int64_t items;                 // of a key head
    int tile_tokens;      // tokens of a row tile of the prefix kernel; 0: it does not run
    int64_t pairs;        // its pairs of row tiles
};
PagedSizes paged_sizes(int Z, int L, int H, int Hk) {
    PagedSizes s;
    const int64_t own = static_cast<int64_t>(L) * (H / Hk), all = own * Z;
    s.prefix_warps = row_warps(all);
    s.own_warps = row_warps(own);
    s.prefix_rt = (all + 16 * s.prefix_warps - 1) / (16 * s.prefix_warps);
    s.own_rt = (own + 16 * s.own_warps - 1) / (16 * s.own_warps);
    s.items = s.prefix_rt + Z * s.own_rt;
    s.tile_tokens = 0;
    s.pairs = 0;
    if (H / Hk <= 128 && all > kPrefixKernelRows) {
        s.tile_tokens = 128 / (H / Hk);
        s.pairs = (static_cast<int64_t>(Z) * L + 2 * s.tile_tokens - 1) / (2 * s.tile_tokens);
    }
    return s;
}

// a head has as many partials as groups and items; the groups' blocks are at most
// the grid's, or one a head
size_t part_bytes(const PagedSizes &s, int Hk, int D) {
    return (static_cast<size_t>(std::max(kPagedMostBlocks, Hk)) + s.items * Hk) * kPagedPartRows * D * sizeof(float);
}
// the splits are chosen so that all blocks of the prefix kernel fit the SMs once
size_t prefix_part_bytes(const PagedSizes &s, int Hk, int D) {
    return s.pairs == 0 ? 0 : (kPagedMostSms + static_cast<size_t>(s.pairs) * Hk) * 256 * D * sizeof(float);
}
size_t groups_bytes(const PagedSizes &s, int Hk) {
    return (static_cast<size_t>(s.items) * Hk * sizeof(int2) + 255) & ~size_t(255);
}

// A bf16 tensor of four dimensions (innermost first, 128-byte swizzle).
sigattn_status encode_box(CUtensorMap *m, const void *base, const cuuint64_t (&dims)[4], const cuuint64_t (&strides)[3],
                          const cuuint32_t (&box)[4]) {
    const cuuint32_t one[4] = {1, 1, 1, 1};
    const CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, one,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        g_last_cuda_error.store(10000 + static_cast<int>(r));
        return SIGATTN_ERR_CUDA;
    }
    return SIGATTN_OK;
}
// Pages [pages][page_size][Hk][D] in boxes of 64 entries of one head of `rows` places.
sigattn_status encode_pages(CUtensorMap *m, const void *base, const CacheShape &c, int rows) {
    const cuuint64_t D = c.D, Hk = c.Hk, page = c.page_size;
    return encode_box(m, base, {D, Hk, page, static_cast<cuuint64_t>(c.pages)}, {D * 2, Hk * D * 2, page * Hk * D * 2},
                      {64, 1, static_cast<cuuint32_t>(rows), 1});
}

struct PagedMaps {
    CUtensorMap k, v;                        // boxes of the tile kernel
    CUtensorMap prefix_q, prefix_k, prefix_v;
};

template <int D, int MODE, int SCORE>
sigattn_status prefix_launch(const PagedMaps &m, const PagedParams &p, cudaStream_t st) {
    constexpr int KS = FwdStages<D>::K, VS = FwdStages<D>::V;
    return launch(paged_prefix_kernel<D, MODE, SCORE>, dim3(p.splits, p.pairs, p.Hk), dim3(kFwdThreads),
                  FwdLayout<D, KS, VS>::SMEM_ALLOC, st, m.prefix_q, m.prefix_k, m.prefix_v, p);
}

template <int D, int SCORE>
sigattn_status paged_launch(const PagedMaps &m, const PagedParams &p, cudaStream_t st) {
    using Lay = PagedLayout<D>;
    sigattn_status s = SIGATTN_OK;
    if (p.splits > 0) {
        s = g_sigmoid_mode.load() == kSigmoidTanh ? prefix_launch<D, kSigmoidTanh, SCORE & ~kScoreFar>(m, p, st)
                                                  : prefix_launch<D, kSigmoidExp, SCORE>(m, p, st);
        if (s != SIGATTN_OK) return s;
    }
    // The tile kernel needs nothing of the prefix kernel's, and the join reads
    // its lengths before it waits: both may start early.
    s = launch_with(paged_tiles_kernel<D, SCORE>, dim3(p.groups * p.heads_wide), dim3(kPagedThreads), Lay::bytes(SIGATTN_PAGED_MAX_Z),
                    Lay::bytes(p.Z), p.splits > 0, 1u, st, m.k, m.v, p);
    if (s != SIGATTN_OK) return s;
    const int64_t rows = static_cast<int64_t>(p.Z) * p.L * p.H;
    auto join = [&](auto kernel, int per_block) {
        return launch_with(kernel, dim3(static_cast<unsigned>((rows + per_block - 1) / per_block)), dim3(kJoinThreads),
                           0, 0, true, 1u, st, p);
    };
    if (rows <= kJoin8Rows) return join(paged_join_kernel<D, 8>, 1);
    if (rows <= kJoin4Rows) return join(paged_join_kernel<D, 4>, 2);
    if (rows <= kJoin2Rows) return join(paged_join_kernel<D, 2>, 4);
    return join(paged_join_kernel<D, 1>, 8);
}
template <int D>
sigattn_status paged_score(int score, const PagedMaps &m, const PagedParams &p, cudaStream_t st) {
    switch (score) {
        case 0: return paged_launch<D, 0>(m, p, st);
        case kScoreCap: return paged_launch<D, kScoreCap>(m, p, st);
        case kScoreSlope: return paged_launch<D, kScoreSlope>(m, p, st);
        case kScoreCap | kScoreSlope: return paged_launch<D, kScoreCap | kScoreSlope>(m, p, st);
        case kScoreCap | kScoreFar: return paged_launch<D, kScoreCap | kScoreFar>(m, p, st);
        default: return paged_launch<D, kScoreCap | kScoreSlope | kScoreFar>(m, p, st);
    }
}

template <typename T, int D>
sigattn_status append_launch(const AppendParams &p, int sms, cudaStream_t st) {
    // Few tokens (a decoding step): eight warps share one, a block, and read ahead.
    // Many: a warp each.
    const int64_t tokens = static_cast<int64_t>(p.Z) * p.L;
    const bool few = tokens <= int64_t(4) * sms;
    const int share = few ? kAppendThreads / 32 : 1;
    const int64_t blocks = (tokens * share + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
    return launch(cache_append_kernel<T, D>, dim3(static_cast<unsigned>(blocks)), dim3(kAppendThreads), 0, st, p, share,
                  few);
}

}  // namespace

extern "C" {

sigattn_status sigattn_cache_append(const void *k, const void *v, const void *q, void *q_out, void *k_pages,
                                    void *v_pages, const int32_t *page_table, const int32_t *cache_lens,
                                    const int32_t *seqlens_new, const int32_t *prefix_len, int32_t *lens_out, int Z,
                                    int L, int H, int Hk, int D, int pages, int page_size, int max_pages,
                                    const float *inv_freq, int rot, int interleaved, sigattn_dtype dtype,
                                    void *stream) {
    const CacheShape c{Z, L, q != nullptr ? H : 0, Hk, D, pages, page_size, max_pages, 0, dtype};
    bool empty = false;
    sigattn_status s = check_cache(c, false, &empty);
    if (s != SIGATTN_OK) return s;
    if (rot < 0 || rot > D || rot % 16 != 0 || (rot > 0 && inv_freq == nullptr)) return SIGATTN_ERR_INVALID_ARG;
    if (Z == 0) return SIGATTN_OK;
    if (L == 0) return SIGATTN_ERR_INVALID_ARG;     // lens_out could not be written
    for (const void *t : {k, v, static_cast<const void *>(k_pages), static_cast<const void *>(v_pages)}) {
        if (t == nullptr && !(pages == 0 && (t == k_pages || t == v_pages))) return SIGATTN_ERR_INVALID_ARG;
        if (!aligned16(t)) return SIGATTN_ERR_MISALIGNED;
    }
    if ((page_table == nullptr && max_pages > 0) || cache_lens == nullptr || seqlens_new == nullptr ||
        lens_out == nullptr || (q != nullptr && q_out == nullptr))
        return SIGATTN_ERR_INVALID_ARG;
    if (!aligned16(q) || (q != nullptr && !aligned16(q_out))) return SIGATTN_ERR_MISALIGNED;
    int dev = 0, cc = 0, *status = nullptr;
    if ((s = device_state(&dev, &cc, &status)) != SIGATTN_OK) return s;
    AppendParams p = {};
    p.k = k;
    p.v = v;
    p.q = q;
    p.q_out = q_out;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.page_table = page_table;
    p.cache_lens = cache_lens;
    p.seqlens_new = seqlens_new;
    p.prefix_len = prefix_len;
    p.lens_out = lens_out;
    p.inv_freq = inv_freq;
    p.Z = Z;
    p.L = L;
    p.H = c.H;
    p.Hk = Hk;
    p.pages = pages;
    p.page_shift = page_shift_of(page_size);
    p.max_pages = max_pages;
    p.rot = rot;
    p.interleaved = interleaved != 0;
    p.status = status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int sms = g_sm_count[dev];
    if (dtype == SIGATTN_BF16)
        return D == 64 ? append_launch<__nv_bfloat16, 64>(p, sms, st) : append_launch<__nv_bfloat16, 128>(p, sms, st);
    return D == 64 ? append_launch<float, 64>(p, sms, st) : append_launch<float, 128>(p, sms, st);
}

size_t sigattn_fwd_paged_workspace_bytes(int Z, int L, int H, int Hk, int D, sigattn_dtype dtype) {
    if (Z <= 0 || L <= 0 || H <= 0 || Hk <= 0 || H % Hk != 0 || (D != 64 && D != 128) || dtype != SIGATTN_BF16)
        return 0;
    const PagedSizes s = paged_sizes(Z, L, H, Hk);
    return groups_bytes(s, Hk) + part_bytes(s, Hk, D) + prefix_part_bytes(s, Hk, D);
}

sigattn_status sigattn_fwd_paged(const void *q, const void *k_pages, const void *v_pages, void *o,
                                 const int32_t *page_table, const int32_t *seqlens_k, const int32_t *seqlens_q,
                                 const int32_t *prefix_table, const int32_t *prefix_len, int Z, int L, int H, int Hk,
                                 int D, int pages, int page_size, int max_pages, int prefix_pages, float alpha,
                                 float bias, const float *bias_z, float cap, const float *slopes, void *workspace,
                                 size_t workspace_bytes, sigattn_dtype dtype, void *stream) {
    const CacheShape c{Z, L, H, Hk, D, pages, page_size, max_pages, prefix_pages, dtype};
    bool empty = false;
    sigattn_status s = check_cache(c, true, &empty);
    if (s != SIGATTN_OK) return s;
    if (!(cap >= 0.0f) || !std::isfinite(cap) || (cap > 0.0f && !std::isfinite(alpha / cap)))
        return SIGATTN_ERR_INVALID_ARG;
    if (empty) return SIGATTN_OK;
    if (Z > SIGATTN_PAGED_MAX_Z) return SIGATTN_ERR_TOO_LARGE;
    if (pages == 0) return SIGATTN_ERR_INVALID_ARG;
    for (const void *t : {q, k_pages, v_pages, static_cast<const void *>(o)}) {
        if (t == nullptr) return SIGATTN_ERR_INVALID_ARG;
        if (!aligned16(t)) return SIGATTN_ERR_MISALIGNED;
    }
    if ((page_table == nullptr && max_pages > 0) || seqlens_k == nullptr || seqlens_q == nullptr)
        return SIGATTN_ERR_INVALID_ARG;
    if (prefix_len != nullptr && prefix_table == nullptr && prefix_pages > 0) return SIGATTN_ERR_INVALID_ARG;
    const int64_t rows = static_cast<int64_t>(Z) * L * H;
    const int64_t tiles = ((static_cast<int64_t>(max_pages) << page_shift_of(page_size)) + kPagedTile - 1) / kPagedTile;
    if (rows > INT_MAX || tiles * Z > INT_MAX) return SIGATTN_ERR_TOO_LARGE;
    const size_t need = sigattn_fwd_paged_workspace_bytes(Z, L, H, Hk, D, dtype);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return SIGATTN_ERR_INVALID_ARG;
    if (need > 0 && !aligned16(workspace)) return SIGATTN_ERR_MISALIGNED;
    int dev = 0, cc = 0, *status = nullptr;
    if ((s = device_state(&dev, &cc, &status)) != SIGATTN_OK) return s;
    if (dtype == SIGATTN_BF16 && cc != 100) return SIGATTN_ERR_UNSUPPORTED_DEVICE;
    const PagedSizes z = paged_sizes(Z, L, H, Hk);
    if (z.items * Hk > INT_MAX - 2 * kPagedMostBlocks || z.pairs > 65535 || Hk > 65535) return SIGATTN_ERR_TOO_LARGE;
    PagedParams p = {};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.page_table = page_table;
    p.seqlens_k = seqlens_k;
    p.seqlens_q = seqlens_q;
    p.prefix_table = prefix_table;
    p.prefix_len = prefix_len;
    p.Z = Z;
    p.L = L;
    p.H = H;
    p.Hk = Hk;
    p.group = H / Hk;
    p.pages = pages;
    p.page_shift = page_shift_of(page_size);
    p.max_pages = max_pages;
    p.prefix_pages = prefix_pages;
    p.alpha = alpha;
    p.bias = bias;
    p.cap = cap;
    p.bias_z = bias_z;
    p.slopes = slopes;
    p.status = status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == SIGATTN_FP32) {
        const dim3 grid(static_cast<unsigned>(rows)), block(32 * kPagedF32Warps);
        const float *fq = static_cast<const float *>(q), *fk = static_cast<const float *>(k_pages),
                    *fv = static_cast<const float *>(v_pages);
        float *fo = static_cast<float *>(o);
        return D == 64 ? launch(paged_f32_kernel<64>, grid, block, 0, st, p, fq, fk, fv, fo)
                       : launch(paged_f32_kernel<128>, grid, block, 0, st, p, fq, fk, fv, fo);
    }
    if ((s = get_encoder()) != SIGATTN_OK) return s;
    char *ws = static_cast<char *>(workspace);
    p.groups_of = reinterpret_cast<int2 *>(ws);
    p.part = reinterpret_cast<float *>(ws + groups_bytes(z, Hk));
    p.prefix_rt = static_cast<int>(z.prefix_rt);
    p.own_rt = static_cast<int>(z.own_rt);
    p.prefix_warps = z.prefix_warps;
    p.own_warps = z.own_warps;
    const int sms = std::min(g_sm_count[dev], kPagedMostSms);
    const int blocks = sms * (D == 64 ? PagedLayout<64>::kBlocksPerSm : PagedLayout<128>::kBlocksPerSm);
    p.heads_wide = std::min(Hk, blocks);
    p.groups = blocks / p.heads_wide;
    p.items = static_cast<int>(z.items);
    p.timeout_ns = g_timeout_ns.load();
    PagedMaps m;
    const int own_box = std::min(page_size, kPagedTile);
    if ((s = encode_pages(&m.k, k_pages, c, own_box)) != SIGATTN_OK) return s;
    if ((s = encode_pages(&m.v, v_pages, c, own_box)) != SIGATTN_OK) return s;
    if (z.tile_tokens > 0 && prefix_len != nullptr && prefix_pages > 0) {
        p.prefix_part = reinterpret_cast<float *>(ws + groups_bytes(z, Hk) + part_bytes(z, Hk, D));
        p.tile_tokens = z.tile_tokens;
        p.pairs = static_cast<int>(z.pairs);
        // as many splits as SMs allow, but no more than a full prefix needs to give each
        // the same number of tiles: the others would only add partials
        const int64_t most = std::max<int64_t>(1, sms / (z.pairs * Hk));
        const int64_t tiles = ((static_cast<int64_t>(prefix_pages) << p.page_shift) + 127) / 128;
        const int64_t each = (tiles + most - 1) / most;
        p.splits = static_cast<int>((tiles + each - 1) / each);
        const int box = std::min(page_size, 128);
        if ((s = encode_pages(&m.prefix_k, k_pages, c, box)) != SIGATTN_OK) return s;
        if ((s = encode_pages(&m.prefix_v, v_pages, c, box)) != SIGATTN_OK) return s;
        const cuuint64_t d = D, group = H / Hk, heads = Hk, tokens = static_cast<cuuint64_t>(Z) * L;
        if ((s = encode_box(&m.prefix_q, q, {d, group, heads, tokens}, {d * 2, group * d * 2, group * heads * d * 2},
                            {64, static_cast<cuuint32_t>(group), 1, static_cast<cuuint32_t>(z.tile_tokens)})) != SIGATTN_OK)
            return s;
    }
    const int score = score_terms(cap, slopes);
    return D == 64 ? paged_score<64>(score, m, p, st) : paged_score<128>(score, m, p, st);
}

}  // extern "C"
