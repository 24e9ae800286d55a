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
    if (own + ahead > most || static_cast<int64_t>(c.Z) * c.L > most || c.H > 65535) return SIGATTN_ERR_TOO_LARGE;
    return SIGATTN_OK;
}

// Row warps (1, 2 or 4, 16 rows each) of a tile over `rows` query rows.
int row_warps(int64_t rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }

constexpr int kPagedMostBlocks = 1024;    // more than any device's grid

struct PagedSizes {
    int prefix_warps, own_warps, part_rows;
    int64_t items;
};
PagedSizes paged_sizes(int Z, int L, int H, int Hk) {
    PagedSizes s;
    const int64_t own = static_cast<int64_t>(L) * (H / Hk), all = own * Z;
    s.prefix_warps = row_warps(all);
    s.own_warps = row_warps(own);
    s.part_rows = 16 * std::max(s.prefix_warps, s.own_warps);
    s.items = Hk * ((all + 16 * s.prefix_warps - 1) / (16 * s.prefix_warps) +
                    Z * ((own + 16 * s.own_warps - 1) / (16 * s.own_warps)));
    return s;
}

size_t before_bytes(int Z) { return (static_cast<size_t>(Z + 1) * 4 + 255) & ~size_t(255); }

template <int D, int SCORE>
sigattn_status paged_launch(const PagedParams &p, cudaStream_t st) {
    using Lay = PagedLayout<D>;
    sigattn_status s = launch(paged_tiles_kernel<D, SCORE>, dim3(p.blocks), dim3(kPagedThreads),
                              Lay::bytes(SIGATTN_PAGED_MAX_Z), Lay::bytes(p.Z), st, p);
    if (s != SIGATTN_OK) return s;
    const int64_t rows = static_cast<int64_t>(p.Z) * p.L * p.H;
    return launch(paged_join_kernel<D>, dim3(static_cast<unsigned>((rows + 7) / 8)), dim3(256), 0, st, p);
}
template <int D>
sigattn_status paged_score(int score, const PagedParams &p, cudaStream_t st) {
    switch (score) {
        case 0: return paged_launch<D, 0>(p, st);
        case kScoreCap: return paged_launch<D, kScoreCap>(p, st);
        case kScoreSlope: return paged_launch<D, kScoreSlope>(p, st);
        default: return paged_launch<D, kScoreCap | kScoreSlope>(p, st);
    }
}

template <typename T, int D>
sigattn_status append_launch(const AppendParams &p, int sms, cudaStream_t st) {
    const int64_t tokens = static_cast<int64_t>(p.Z) * p.L;
    // Four tokens a block keep three units in flight per thread; below two
    // blocks an SM one token a block spreads a decoding step over more SMs.
    if (tokens >= int64_t(8) * sms)
        return launch(cache_append_kernel<T, D, 4>, dim3(static_cast<unsigned>((tokens + 3) / 4)),
                      dim3(kAppendThreads), 0, st, p);
    return launch(cache_append_kernel<T, D, 1>, dim3(static_cast<unsigned>(tokens)), dim3(kAppendThreads), 0, st, p);
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
    return before_bytes(Z) + static_cast<size_t>(kPagedMostBlocks + s.items) * s.part_rows * D * sizeof(float);
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
    for (const void *t : {q, k_pages, v_pages, static_cast<const void *>(o)}) {
        if (t == nullptr && !(pages == 0 && t != q && t != o)) return SIGATTN_ERR_INVALID_ARG;
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
    if (z.items > INT_MAX - 2 * kPagedMostBlocks) return SIGATTN_ERR_TOO_LARGE;
    PagedParams p = {};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k_pages = static_cast<const __nv_bfloat16 *>(k_pages);
    p.v_pages = static_cast<const __nv_bfloat16 *>(v_pages);
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
    p.before = static_cast<int *>(workspace);
    p.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + before_bytes(Z));
    p.prefix_warps = z.prefix_warps;
    p.own_warps = z.own_warps;
    p.part_rows = z.part_rows;
    p.blocks = std::min(kPagedMostBlocks,
                        g_sm_count[dev] * (D == 64 ? PagedLayout<64>::kBlocksPerSm : PagedLayout<128>::kBlocksPerSm));
    const int score = (cap > 0.0f ? kScoreCap : 0) | (slopes != nullptr ? kScoreSlope : 0);
    return D == 64 ? paged_score<64>(score, p, st) : paged_score<128>(score, p, st);
}

}  // extern "C"
