// Backward of the masked attention (span_score.cuh), bf16: a dQ kernel by query
// tiles and a dK/dV kernel by key tiles, no atomics, with the structure of the
// padding-only backward (bwd_sm100.cuh) and these differences:
//
//  - dQ visits the key tiles of its rows' hull.  dK/dV visits the query tiles
//    whose hull meets its keys: first to last of them, from a table that
//    span_prep_kernel writes (one entry per 128 rows), so neither kernel
//    touches a tile that no pair needs under causal, prefix, document or
//    window masks;
//  - P and dS are rounded to bf16 (span_score.cuh says why); all sums are fp32;
//  - a key head serves `group` query heads: the dK/dV CTA of a key head runs
//    through the query tiles of all of them and accumulates in tensor memory,
//    so shared heads need no second pass and the sum's order is fixed;
//  - the MMA warp zeroes the rows at or beyond n of the tiles that serve as
//    the contraction side (K in dQ; Q and dO in dK/dV), so that NaN in padding
//    never meets a weight of zero.
//
//  - the three kernels overlap (programmatic dependent launch): dK/dV starts
//    beside the table kernel and waits for it, dQ beside dK/dV's last blocks,
//    which its shorter blocks fill in behind.  Against dQ first and one kernel
//    after the other: packed capped D = 64 documents 157.6 -> 134.2 us, capped prefix
//    D = 128 638 -> 547 us, documents of 4096 rows at D = 128 252.5 -> 197 us, causal 8K at
//    D = 128 1860 -> 1840 us.
//
// Bound: dQ issues 6 D and dK/dV 8 D tensor FLOP per pair against one MUFU op
// (two with a cap): tensor-bound at D = 128, near the MUFU's rate at D = 64.
#pragma once

#include "bwd_sm100.cuh"
#include "span_score.cuh"
#include "span_split.cuh"

namespace sigattn {

struct SpanBwdParams {
    __nv_bfloat16 *dq, *dk, *dv;
    SpanSource src;
    int H, Hk, group;
    int heads_first;       // grid (heads, tiles, samples) instead of (tiles, heads, samples)
    unsigned split;        // blocks of a cluster that share a tile (1: none); x is that much wider
    float alpha, bias, cap;
    const float *bias_z, *slopes;
    const int2 *clean;     // [Z][tiles * 128] clipped spans (span_prep_kernel)
    const int4 *hull;      // [Z][tiles] {least lo, greatest hi, greatest lo, least hi}
    uint64_t timeout_ns;
};

// Clipped spans of every row, rows of padding (0, 0), and per 128-row tile the
// hull of its rows' spans: {least lo and greatest hi of the rows that see a
// key, greatest lo and least hi of all 128 rows}.  A key tile [k0, k1) is met
// when least lo < k1 and greatest hi > k0, and is seen whole by every row when
// greatest lo <= k0 and least hi >= k1.
static __global__ void __launch_bounds__(128) span_prep_kernel(const SpanSource src, int2 *clean, int4 *hull) {
    __shared__ int4 part[4];
    grid_release();
    const int z = blockIdx.y, i = blockIdx.x * 128 + threadIdx.x;
    const int n = span_tokens(src, z);
    const int2 r = row_span(src, z, i, n);
    clean[static_cast<size_t>(z) * gridDim.x * 128 + i] = r;
    const bool some = r.x < r.y;
    const int4 w = make_int4(__reduce_min_sync(0xffffffffu, some ? r.x : INT_MAX),
                             __reduce_max_sync(0xffffffffu, r.y), __reduce_max_sync(0xffffffffu, r.x),
                             __reduce_min_sync(0xffffffffu, r.y));
    if (lane_id() == 0) part[warp_id()] = w;
    __syncthreads();
    if (threadIdx.x == 0) {
        int4 a = part[0];
        for (int u = 1; u < 4; ++u) {
            a.x = min(a.x, part[u].x);
            a.y = max(a.y, part[u].y);
            a.z = max(a.z, part[u].z);
            a.w = min(a.w, part[u].w);
        }
        hull[static_cast<size_t>(z) * gridDim.x + blockIdx.x] = a;
    }
}

// Shape of the backward blocks.  A step is kStep columns of a streamed 128-row
// tile (keys in dQ, queries in dK/dV): the whole tile, but half of it at D = 64, so
// that scores and accumulators take 256 columns of tensor memory and two blocks
// share an SM; one's start and end, most of a short document's time, pass while the
// other computes.  Whole backward, against one block an SM in both kernels: packed
// capped documents 133.6 -> 119.4 us, documents 130.7 -> 122.5 us, window 8K 202 -> 198 us,
// causal 8K 431 -> 425 us, full capped 4K 620 -> 652 us (half steps hand over twice
// as often).  dK/dV, whose threads hold more, then loads both rings from one warp: two
// blocks of 320 threads leave 96 registers a thread, of 384 threads 80, which lost 6 to
// 25%.
// Spills, bytes a thread stored and loaded (tanh form): dK/dV at D = 64 none to 84 / 152,
// at D = 128, 168 registers, 104 to 148 / 176 to 252 (the padding-only kernel, whose score
// has one form, 12 / 12); dQ at D = 64 up to 48 / 64, at D = 128 none.  Two copies of the
// score's forms, 32 packed weights and 32 gains are live together there.
template <int D, bool DQ>
struct SpanBwdShape {
    static constexpr bool kHalf = D == 64;
    static constexpr int kPerSm = kHalf ? 2 : 1;
    static constexpr int kStep = kHalf ? 64 : 128, kParts = 128 / kStep;
    static constexpr int NG = D == 64 && !kHalf ? 4 : 2;     // sigma warpgroups, kCols columns of a step each
    static constexpr int kAux = kHalf && !DQ ? 2 : 4;        // warps that load and issue
    static constexpr int kThreads = 32 * kAux + 128 * NG, kArrivals = 128 * NG;
    static constexpr int kCols = kStep / NG, kPacked = kCols / 2;
    static constexpr int SX = kHalf ? 2 : BwdStages<D>::X, SY = kHalf ? 2 : BwdStages<D>::Y;
    // TMEM column (relative to the buffer) of the packed bf16 values of K step kk
    // (columns 16 kk ... of the step), over the first kPacked of their warpgroup's
    static __device__ __forceinline__ uint32_t packed_col(int kk) {
        return kCols * ((16 * kk) / kCols) + ((16 * kk) % kCols) / 2;
    }
};

template <int D, bool DQ>
struct SpanBwdLayout {
    using SG = SpanBwdShape<D, DQ>;
    static constexpr int NSUB = D / 64;
    static constexpr int SUB_BYTES = 128 * 64 * 2;
    static constexpr int TILE_BYTES = NSUB * SUB_BYTES;
    static constexpr int PART_BYTES = SG::kStep * 128;             // a part's rows in one 64-column atom
    static constexpr int OFF_A = 0;                                // resident tiles (dQ: Q, dO; dK/dV: K, V)
    static constexpr int OFF_B = TILE_BYTES;
    static constexpr int OFF_X = 2 * TILE_BYTES;                   // ring (dQ: K; dK/dV: Q)
    static constexpr int OFF_Y = OFF_X + SG::SX * TILE_BYTES;      // ring (dQ: V; dK/dV: dO)
    static constexpr int OFF_BAR = OFF_Y + SG::SY * TILE_BYTES;
    static constexpr int MAX_HANDOFF = 8;
    static constexpr int NBAR = 1 + 2 * SG::SX + 2 * SG::SY + MAX_HANDOFF;
    static constexpr int OFF_TMEM = OFF_BAR + NBAR * 8;
    static constexpr int OFF_ABORT = OFF_TMEM + 8;
    static constexpr int OFF_HULL = OFF_ABORT + 8;                 // {first, last} of each warp
    static constexpr int SMEM_ALLOC = OFF_HULL + 8 * (SG::kThreads / 32) + 1024;
    static constexpr uint32_t TMEM_COLS = SG::kHalf ? 256 : 512;
    static_assert((DQ ? 3 * SG::kStep + D : 2 * SG::kStep + 2 * D) <= TMEM_COLS, "TMEM budget");
    static_assert((DQ ? D : 2 * D) * 128 * 4 <= OFF_BAR, "a split's sums fit the tiles' place");
    static_assert(SG::kPerSm * TMEM_COLS <= 512 && SG::kPerSm * (SMEM_ALLOC + 1024) <= 228 * 1024, "SM budget");
};

// dq_sigma_tile (bwd_sm100.cuh) with the masked score function: one key tile
// of a dQ sigma warpgroup.  `row` is this thread's query, `key0` the tile's
// first key, `span` the keys its row sees.
template <int D, int MODE, int SCORE>
__device__ __forceinline__ bool span_dq_tile(uint32_t trow, int w, uint32_t col_s, uint32_t dcol,
                                             uint64_t *s_full, uint32_t s_par, uint64_t *s_free,
                                             uint64_t *dp_full, uint32_t dp_par, uint64_t *ds_ready,
                                             const ScoreCoef &cf, int row, int key0, int2 span, ScorePause &pause,
                                             const WaitCtx &wctx) {
    using SG = SpanBwdShape<D, true>;
    if (!__all_sync(0xffffffffu, mbar_wait(s_full, s_par, wctx))) return false;
    tc_fence_after();
    const int first = key0 + SG::kCols * w;    // this warpgroup's first key
    const bool whole = __all_sync(0xffffffffu, span.x <= first && span.y >= first + SG::kCols);
    const bool some = whole || __any_sync(0xffffffffu, span.x < first + SG::kCols && span.y > first);
    constexpr int kChunks = SG::kCols / 32;
    if (!some) {
        // none of the warp's rows sees any of these keys: dS = 0 without a score
        tc_fence_before();
        mbar_arrive(s_free);
        if (!__all_sync(0xffffffffu, mbar_wait(dp_full, dp_par, wctx))) return false;
        tc_fence_after();
        uint32_t zero[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) zero[i] = 0u;
#pragma unroll
        for (int ch = 0; ch < kChunks; ++ch) tmem_st16(trow + dcol + SG::kCols * w + 16 * ch, zero);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(ds_ready);
        return true;
    }
    uint32_t r[SG::kCols];
    tmem_ld_cols(trow + col_s + SG::kCols * w, r);
    tc_fence_before();
    mbar_arrive(s_free);
    float2 g[16];
    auto gains = [&](int ch) {
        uint32_t unused[16];
        score_chunk<MODE, SCORE, true>(r + 32 * ch, cf, static_cast<float>(row - first - 32 * ch), unused, g, pause,
                                         whole);
    };
    gains(0);   // before dP is waited for
    const uint32_t dc = dcol + SG::kCols * w;
    if (!__all_sync(0xffffffffu, mbar_wait(dp_full, dp_par, wctx))) return false;
    tc_fence_after();
#pragma unroll
    for (int ch = 0; ch < kChunks; ++ch) {
        if (ch > 0) gains(ch);
        uint32_t d[32];
        tmem_ld32(trow + dc + 32 * ch, d);
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 ds = mul2(g[i], f2(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1])));
            pk[i] = pack_bf16x2(ds.x, ds.y);
        }
        if (!whole) keep_bits(pk, bit_range(span.x - first - 32 * ch, span.y - first - 32 * ch));
        tmem_st16(trow + dc + 16 * ch, pk);
    }
    tmem_wait_st();
    tc_fence_before();
    mbar_arrive(ds_ready);
    return true;
}

// dkdv_sigma_tile (bwd_sm100.cuh) with the masked score function: one query
// tile of a dK/dV sigma warpgroup, whose columns are the queries from q_first
// on.  `key` is this thread's key; `whole`: every row of the tile sees every
// key of this CTA's tile, otherwise `clean` points at the spans of the columns (lane
// i reads column i); keys_there: none of this warp's keys is padding.
template <int D, int MODE, int SCORE>
__device__ __forceinline__ bool span_dkdv_tile(uint32_t tS, uint32_t tD, uint64_t *s_full, uint64_t *s_free,
                                               uint64_t *dp_full, uint64_t *p_ready, uint64_t *ds_ready,
                                               uint32_t par, const ScoreCoef &cf, int key, int q_first,
                                               bool whole, bool keys_there, const int2 *clean, ScorePause &pause,
                                               const WaitCtx &wctx) {
    using SG = SpanBwdShape<D, false>;
    constexpr int W = SG::kPacked / 16;   // words of 32 columns
    float2 g[SG::kPacked];
    uint32_t pk[SG::kPacked];
    uint32_t bits[W];
    bool some = true;
    if (!whole) {
        // lane i takes column i: the keys of this warp that it sees, as bits, turned
        // round so that each key has its columns
        const int key0 = key - static_cast<int>(threadIdx.x & 31);
        some = false;
#pragma unroll
        for (int u = 0; u < W; ++u) {
            const int2 s = clean[32 * u + (threadIdx.x & 31)];
            bits[u] = warp_transpose(bit_range(s.x - key0, s.y - key0));
            some |= __any_sync(0xffffffffu, bits[u] != 0u);
        }
    }
    if (!some) {
        // no query of these columns sees a key of this warp: P^T = dS^T = 0
        if (!__all_sync(0xffffffffu, mbar_wait(s_full, par, wctx))) return false;
        mbar_arrive(s_free);
        if (!__all_sync(0xffffffffu, mbar_wait(dp_full, par, wctx))) return false;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < SG::kPacked; ++i) pk[i] = 0u;
        tmem_st_cols(tD, pk);
        tmem_st_cols(tD + SG::kPacked, pk);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_ready);
        mbar_arrive(ds_ready);
        return true;
    }
    if (!__all_sync(0xffffffffu, mbar_wait(s_full, par, wctx))) return false;
    tc_fence_after();
    {
        uint32_t r[SG::kCols];
        tmem_ld_cols(tS, r);
        // S^T is in registers: the MMA warp may compute the next S^T now
        tc_fence_before();
        mbar_arrive(s_free);
        const float rel = static_cast<float>(key - q_first);
#pragma unroll
        for (int u = 0; u < W; ++u)
            score_chunk<MODE, SCORE, true>(r + 32 * u, cf, rel - static_cast<float>(32 * u), pk + 16 * u, g + 16 * u,
                                           pause, whole && keys_there);
    }
    auto keep = [&](uint32_t (&x)[SG::kPacked]) {
#pragma unroll
        for (int u = 0; u < W; ++u) keep_bits(*reinterpret_cast<uint32_t(*)[16]>(&x[16 * u]), bits[u]);
    };
    if (!whole) keep(pk);
    if (!__all_sync(0xffffffffu, mbar_wait(dp_full, par, wctx))) return false;
    tc_fence_after();
    uint32_t ds[SG::kPacked];
    {
        // the first kPacked of this warpgroup's dP^T columns, then P^T over them
        uint32_t d[SG::kPacked];
        tmem_ld_cols(tD, d);
        tmem_st_cols(tD, pk);
#pragma unroll
        for (int ii = 0; ii < SG::kPacked / 2; ++ii) {
            const float2 v = mul2(g[ii], f2(__uint_as_float(d[2 * ii]), __uint_as_float(d[2 * ii + 1])));
            ds[ii] = pack_bf16x2(v.x, v.y);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_ready);
    }
    {
        // the other kPacked dP^T columns, then dS^T over them
        uint32_t d[SG::kPacked];
        tmem_ld_cols(tD + SG::kPacked, d);
#pragma unroll
        for (int ii = 0; ii < SG::kPacked / 2; ++ii) {
            const float2 v = mul2(g[SG::kPacked / 2 + ii],
                                  f2(__uint_as_float(d[2 * ii]), __uint_as_float(d[2 * ii + 1])));
            ds[SG::kPacked / 2 + ii] = pack_bf16x2(v.x, v.y);
        }
    }
    if (!whole) keep(ds);
    tmem_st_cols(tD + SG::kPacked, ds);
    tmem_wait_st();
    tc_fence_before();
    mbar_arrive(ds_ready);
    return true;
}

// Streams step r = 0, 1, ... (tile row0, head h) of one tensor map into a ring
// of S slots; false when a wait gave up.
template <int S, int NSUB>
__device__ __forceinline__ bool span_ring_load(const CUtensorMap *map, uint64_t *full, uint64_t *empty,
                                               uint8_t *base, int tile_bytes, int r, int row0, int h, int z,
                                               const WaitCtx &w) {
    const int st = r % S;
    if (r >= S && !mbar_wait(&empty[st], ((r / S) - 1) & 1, w)) return false;
    mbar_arrive_expect_tx(&full[st], tile_bytes);
    for (int s = 0; s < NSUB; ++s)
        tma_load_4d(map, &full[st], base + st * tile_bytes + s * (128 * 64 * 2), 64 * s, h, row0, z);
    return true;
}

// dQ: one CTA per 128-row query tile (the last rows' tiles first).  Tensor
// memory as bwd_dq_kernel, in steps of kStep keys: S, dP of even and of odd steps,
// dQ.
template <int D, int MODE, int SCORE, bool SPLIT>
__global__ void __launch_bounds__(SpanBwdShape<D, true>::kThreads, SpanBwdShape<D, true>::kPerSm)
    span_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                   const SpanBwdParams p) {
    using Lay = SpanBwdLayout<D, true>;
    using SG = SpanBwdShape<D, true>;
    constexpr int SX = SG::SX, SY = SG::SY, NP = SG::kParts;
    constexpr uint32_t kColS = 0, kColDP0 = SG::kStep, kColDP1 = 2 * SG::kStep, kColDQ = 3 * SG::kStep;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_1k(smem_raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Lay::OFF_BAR);
    uint64_t *res_full = bars;
    uint64_t *x_full = bars + 1;              // K ring
    uint64_t *x_empty = x_full + SX;
    uint64_t *y_full = x_empty + SX;          // V ring
    uint64_t *y_empty = y_full + SY;
    uint64_t *s_full = y_empty + SY;
    uint64_t *dp_full = s_full + 1;           // [2]
    uint64_t *s_free = dp_full + 2;
    uint64_t *ds_ready = s_free + 1;          // [2]
    uint64_t *drain = ds_ready + 2;
    static_assert(7 <= Lay::MAX_HANDOFF, "barrier count");
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Lay::OFF_TMEM);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + Lay::OFF_ABORT);

    const int warp = warp_id(), lane = lane_id();
    const int split = SPLIT ? static_cast<int>(p.split) : 1;
    const SplitPlace at = split_place(split);
    const int z = span_sample(p.src.seqlens, gridDim.z, blockIdx.z), h = p.heads_first ? at.x : blockIdx.y;
    const int kvh = h / p.group;
    const int tiles = p.heads_first ? gridDim.y : at.wide;
    const int qtile = tiles - 1 - (p.heads_first ? static_cast<int>(blockIdx.y) : at.x);
    const int L = p.src.L;
    const int n = span_tokens(p.src, z);
    const bool last = blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1 && blockIdx.z == gridDim.z - 1;
    // span_prep_kernel's tables.  This kernel does not wait for it: it starts once every
    // block of the dK/dV kernel has passed its own wait for that kernel's end, so the
    // tables are in L2.  They are read there (.cg), past an L1 that may hold the tables
    // of an earlier call in the same workspace, since only a wait promises more.
    const int4 hull = __ldcg(&p.hull[static_cast<size_t>(z) * tiles + qtile]);
    if (hull.y == 0) {
        // no row of this tile sees a key: zeros, written by every thread
        if (at.rank == 0) zero_rows<D>(p.dq, z, h, qtile * 128, min(128, L - qtile * 128), L, p.H);
        if constexpr (SPLIT) cluster_skip();
        if (last) grid_wait();
        return;
    }
    const int K0 = hull.x / 128, all_steps = (hull.y + 127) / 128 - K0;     // key tiles
    const int begin = split_step(all_steps, at.rank, split);
    const int J0 = K0 + begin, steps = split_step(all_steps, at.rank + 1, split) - begin;   // this block's
    const bool ragged = (n & 127) != 0 && J0 + steps == (n + 127) / 128;
    if (threadIdx.x == 0) {
        mbar_init(res_full, 1);
        for (int s = 0; s < SX; ++s) {
            mbar_init(&x_full[s], 1);
            mbar_init(&x_empty[s], 1);
        }
        for (int s = 0; s < SY; ++s) {
            mbar_init(&y_full[s], 1);
            mbar_init(&y_empty[s], 1);
        }
        mbar_init(s_full, 1);
        mbar_init(&dp_full[0], 1);
        mbar_init(&dp_full[1], 1);
        mbar_init(s_free, SG::kArrivals);
        mbar_init(&ds_ready[0], SG::kArrivals);
        mbar_init(&ds_ready[1], SG::kArrivals);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
        // the resident tiles fly while the rest of the block sets up
        uint8_t *sQ = smem + Lay::OFF_A, *sDO = smem + Lay::OFF_B;
        mbar_arrive_expect_tx(res_full, 2 * Lay::TILE_BYTES);
        for (int s = 0; s < Lay::NSUB; ++s) {
            tma_load_4d(&tmQ, res_full, sQ + s * Lay::SUB_BYTES, 64 * s, h, qtile * 128, z);
            tma_load_4d(&tmDO, res_full, sDO + s * Lay::SUB_BYTES, 64 * s, h, qtile * 128, z);
        }
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, Lay::TMEM_COLS);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtx wctx{abort_flag, p.src.status, p.timeout_ns};

    if (warp == 0) {
        if (lane == 0) {
            int ix = 0;
            for (int r = 0; r < steps; ++r) {
                if (!span_ring_load<SX, Lay::NSUB>(&tmK, x_full, x_empty, smem + Lay::OFF_X, Lay::TILE_BYTES, r,
                                                   (J0 + r) * 128, kvh, z, wctx))
                    break;
                ix = r + 1;
            }
            mbar_wait_drain(res_full, 0, p.timeout_ns);
            ring_drain<SX>(x_full, ix, p.timeout_ns);
        }
    } else if (warp == 2) {
        if (lane == 0) {
            int iy = 0;
            for (int r = 0; r < steps; ++r) {
                if (!span_ring_load<SY, Lay::NSUB>(&tmV, y_full, y_empty, smem + Lay::OFF_Y, Lay::TILE_BYTES, r,
                                                   (J0 + r) * 128, kvh, z, wctx))
                    break;
                iy = r + 1;
            }
            ring_drain<SY>(y_full, iy, p.timeout_ns);
        }
    } else if (warp == 1) {
        // the whole warp runs converged; elect.sync picks the issuing lane
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, wctx));
        };
        const uint32_t idesc_s = idesc_bf16_f32(128, SG::kStep, false, false);
        const uint32_t idesc_q = idesc_bf16_f32(128, D, false, true);
        const uint32_t sQ = smem_u32(smem + Lay::OFF_A), sDO = smem_u32(smem + Lay::OFF_B);
        const uint32_t xring = smem_u32(smem + Lay::OFF_X), yring = smem_u32(smem + Lay::OFF_Y);
        constexpr uint32_t kDescHi = desc_hi(1024);
        // rows of step r (part r % NP of tile r / NP) in its slot
        auto krows = [&](int r) { return xring + (r / NP % SX) * Lay::TILE_BYTES + (r % NP) * Lay::PART_BYTES; };
        auto vrows = [&](int r) { return yring + (r / NP % SY) * Lay::TILE_BYTES + (r % NP) * Lay::PART_BYTES; };
        // X (128 rows of Q or dO) times Y^T (a step's rows of K or V) into TMEM column `col`
        auto issue_xyT = [&](uint32_t col, uint32_t xbase, uint32_t ybase) {
            const uint32_t x_lo = desc_lo(xbase, 16), y_lo = desc_lo(ybase, 16);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t koff = ((kk >> 2) * Lay::SUB_BYTES + (kk & 3) * 32) >> 4;
                mma_ss_lhw(tmem + col, x_lo + koff, y_lo + koff, kDescHi, idesc_s, kk > 0 ? 1u : 0u);
            }
        };
        const int all = steps * NP;
        // (a block without a step still waits for its resident tiles, whose place its sums take)
        bool ok = wait(res_full, 0) && (!SPLIT || steps > 0) && wait(&x_full[0], 0) && wait(&y_full[0], 0);
        if (ok) {
            tc_fence_after();
            issue_xyT(kColS, sQ, krows(0));
            mma_commit_w(s_full);
            issue_xyT(kColDP0, sDO, vrows(0));
            mma_commit_w(&dp_full[0]);
            if (NP == 1) mma_commit_w(&y_empty[0]);
        }
        for (int r = 0; ok && r < all; ++r) {
            const bool more = r + 1 < all;
            if (more) {
                const int t = (r + 1) / NP;      // tile of the next step
                const bool opens = NP == 1 || (r + 1) % NP == 0, closes = (r + 1) % NP == NP - 1;
                if (opens && !(ok = wait(&x_full[t % SX], (t / SX) & 1))) break;
                if (!(ok = wait(s_free, r & 1))) break;
                tc_fence_after();
                issue_xyT(kColS, sQ, krows(r + 1));
                mma_commit_w(s_full);
                if (opens && !(ok = wait(&y_full[t % SY], (t / SY) & 1))) break;
                // buffer (r+1) % 2 still holds dS_{r-1}: dQ += dS_{r-1} K_{r-1} was issued
                // earlier by this thread and MMAs run in issue order
                tc_fence_after();
                issue_xyT((r + 1) & 1 ? kColDP1 : kColDP0, sDO, vrows(r + 1));
                mma_commit_w(&dp_full[(r + 1) & 1]);
                if (closes) mma_commit_w(&y_empty[t % SY]);
            }
            if (ragged && r == all - NP)
                zero_tile_rows<Lay::NSUB>(smem + Lay::OFF_X + (r / NP % SX) * Lay::TILE_BYTES, n & 127);
            if (!(ok = wait(&ds_ready[r & 1], (r >> 1) & 1))) break;
            tc_fence_after();
            const uint32_t dcol = r & 1 ? kColDP1 : kColDP0;
            const uint32_t k_lo = desc_lo(krows(r), Lay::SUB_BYTES);
#pragma unroll
            for (int kk = 0; kk < SG::kStep / 16; ++kk)
                mma_ts_lhw(tmem + kColDQ, tmem + dcol + SG::packed_col(kk), k_lo + kk * ((16 * 128) >> 4), kDescHi,
                           idesc_q, (r > 0 || kk > 0) ? 1u : 0u);
            if (r % NP == NP - 1) mma_commit_w(&x_empty[r / NP % SX]);
        }
        mma_commit_w(drain);
        mbar_wait_drain(drain, 0, p.timeout_ns);
        __syncwarp();
    } else if (warp >= 4) {
        const int w = (warp - 4) >> 2;      // warpgroup: tile columns [kCols w, kCols (w + 1))
        const int quarter = warp & 3;
        const int row = qtile * 128 + quarter * 32 + lane;
        const uint32_t lane_bits = static_cast<uint32_t>(quarter * 32) << 16;
        const int2 span = row_span(p.src, z, row, n);
        __nv_bfloat16 *drow = p.dq + (static_cast<size_t>(z) * L + row) * (static_cast<size_t>(p.H) * D) +
                              static_cast<size_t>(h) * D;
        const ScoreCoef cf = make_score<SCORE>(p.alpha, bias_of(p.bias_z, p.bias, z), p.cap,
                                                     SCORE & kScoreSlope ? p.slopes[h] : 0.0f);
        bool ok = true;
        ScorePause pause = score_pause(cf);
        for (int r = 0; r < steps * NP; ++r) {
            ok = span_dq_tile<D, MODE, SCORE>(tmem + lane_bits, w, kColS, r & 1 ? kColDP1 : kColDP0, s_full, r & 1,
                                              s_free, &dp_full[r & 1], (r >> 1) & 1, &ds_ready[r & 1], cf, row,
                                              J0 * 128 + r * SG::kStep, span, pause, wctx);
            if (!ok) break;
        }
        // every MMA of this CTA has finished once the MMA warp's final commit lands
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(drain, 0, wctx));
        constexpr int kEpi = D / SG::NG;
        if (ok) {
            tc_fence_after();
            if constexpr (SPLIT)
                split_leave(reinterpret_cast<float4 *>(smem), tmem + lane_bits + kColDQ + w * kEpi, w * kEpi, kEpi,
                            quarter * 32 + lane, steps == 0);
            else
                store_row_from_tmem<D>(tmem + lane_bits + kColDQ, drow, row < L, span.x < span.y, p.alpha, w * kEpi,
                                       kEpi);
        }
    }

    __syncwarp();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, Lay::TMEM_COLS);
    }
    if constexpr (SPLIT) {
        cluster_meet();
        split_add(reinterpret_cast<const float4 *>(smem), D / 8, at.rank, split, threadIdx.x, SG::kThreads,
                  [&](int octet, int r, const float (&x)[8]) {
                      const int i = qtile * 128 + r;
                      if (i >= L) return;
                      const int2 s = __ldcg(&p.clean[static_cast<size_t>(z) * tiles * 128 + i]);
                      reinterpret_cast<uint4 *>(p.dq + ((static_cast<size_t>(z) * L + i) * p.H + h) * D)[octet] =
                          split_pack(x, p.alpha, s.x < s.y);
                  });
        cluster_meet();     // the others may still read this block's sums
    }
    // whatever follows on the stream waits for this kernel alone: it has to end after
    // the dK/dV kernel, beside whose last blocks it may have started
    if (last) grid_wait();
}

// dK/dV: one CTA per 128-key tile of a key head; streams the query tiles that
// meet it, head after head of its group.  Tensor memory as bwd_dkdv_kernel, in
// steps of kStep queries: S^T, dP^T then P^T and dS^T over it, dV, dK.
template <int D, int MODE, int SCORE, bool SPLIT>
__global__ void __launch_bounds__(SpanBwdShape<D, false>::kThreads, SpanBwdShape<D, false>::kPerSm)
    span_dkdv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                     const SpanBwdParams p) {
    using Lay = SpanBwdLayout<D, false>;
    using SG = SpanBwdShape<D, false>;
    constexpr int SX = SG::SX, SY = SG::SY, NP = SG::kParts;
    constexpr uint32_t kColS = 0, kColDP = SG::kStep, kColDV = 2 * SG::kStep, kColDK = 2 * SG::kStep + D;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_1k(smem_raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Lay::OFF_BAR);
    uint64_t *res_full = bars;
    uint64_t *x_full = bars + 1;              // Q ring
    uint64_t *x_empty = x_full + SX;
    uint64_t *y_full = x_empty + SX;          // dO ring
    uint64_t *y_empty = y_full + SY;
    uint64_t *s_full = y_empty + SY;
    uint64_t *dp_full = s_full + 1;
    uint64_t *s_free = dp_full + 1;
    uint64_t *p_ready = s_free + 1;
    uint64_t *ds_ready = p_ready + 1;
    uint64_t *drain = ds_ready + 1;
    static_assert(6 <= Lay::MAX_HANDOFF, "barrier count");
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Lay::OFF_TMEM);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + Lay::OFF_ABORT);
    int2 *met = reinterpret_cast<int2 *>(smem + Lay::OFF_HULL);

    const int warp = warp_id(), lane = lane_id();
    const int split = SPLIT ? static_cast<int>(p.split) : 1;
    const SplitPlace at = split_place(split);
    const int z = span_sample(p.src.seqlens, gridDim.z, blockIdx.z), kvh = p.heads_first ? at.x : blockIdx.y;
    const int tiles = p.heads_first ? gridDim.y : at.wide;
    const int ktile = p.heads_first ? blockIdx.y : at.x;
    const int L = p.src.L;
    const int n = span_tokens(p.src, z);
    const int k0 = ktile * 128, k1 = min(k0 + 128, n);
    grid_wait();        // span_prep_kernel's tables (read with plain loads: they are written
                        // while this kernel may already have started)
    grid_release();     // dQ needs nothing else of this kernel
    // first and last query tile whose hull meets this key tile
    const int4 *hull = p.hull + static_cast<size_t>(z) * tiles;
    {
        int first = INT_MAX, last = -1;
        for (int i = threadIdx.x; i < tiles; i += SG::kThreads) {
            const int4 t = hull[i];
            if (t.x < k1 && t.y > k0) {
                first = min(first, i);
                last = max(last, i);
            }
        }
        first = __reduce_min_sync(0xffffffffu, first);
        last = __reduce_max_sync(0xffffffffu, last);
        if (lane == 0) met[warp] = make_int2(first, last);
    }
    __syncthreads();
    int I0 = INT_MAX, I1 = -1;
#pragma unroll
    for (int u = 0; u < SG::kThreads / 32; ++u) {
        I0 = min(I0, met[u].x);
        I1 = max(I1, met[u].y);
    }
    if (I1 < 0) {
        // no row sees a key of this tile: zeros, written by every thread
        const int rows = min(128, L - k0);
        if (at.rank == 0) {
            zero_rows<D>(p.dk, z, kvh, k0, rows, L, p.Hk);
            zero_rows<D>(p.dv, z, kvh, k0, rows, L, p.Hk);
        }
        if constexpr (SPLIT) cluster_skip();
        return;
    }
    // query tiles of a head; this block's steps and its first head and query tile
    const int per_head = I1 - I0 + 1, all_steps = per_head * p.group;
    const int begin = split_step(all_steps, at.rank, split), steps = split_step(all_steps, at.rank + 1, split) - begin;
    const int head0 = kvh * p.group + begin / per_head, first_tile = I0 + begin % per_head;
    const bool ragged = (n & 127) != 0 && I1 == n / 128;
    if (threadIdx.x == 0) {
        mbar_init(res_full, 1);
        for (int s = 0; s < SX; ++s) {
            mbar_init(&x_full[s], 1);
            mbar_init(&x_empty[s], 1);
        }
        for (int s = 0; s < SY; ++s) {
            mbar_init(&y_full[s], 1);
            mbar_init(&y_empty[s], 1);
        }
        mbar_init(s_full, 1);
        mbar_init(dp_full, 1);
        mbar_init(s_free, SG::kArrivals);
        mbar_init(p_ready, SG::kArrivals);
        mbar_init(ds_ready, SG::kArrivals);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
        // the resident tiles fly while the rest of the block sets up
        uint8_t *sK = smem + Lay::OFF_A, *sV = smem + Lay::OFF_B;
        mbar_arrive_expect_tx(res_full, 2 * Lay::TILE_BYTES);
        for (int s = 0; s < Lay::NSUB; ++s) {
            tma_load_4d(&tmK, res_full, sK + s * Lay::SUB_BYTES, 64 * s, kvh, k0, z);
            tma_load_4d(&tmV, res_full, sV + s * Lay::SUB_BYTES, 64 * s, kvh, k0, z);
        }
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, Lay::TMEM_COLS);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtx wctx{abort_flag, p.src.status, p.timeout_ns};

    if (warp == 0) {
        if (lane == 0) {
            int ix = 0, iy = 0, i = first_tile, h = head0;
            for (int r = 0; r < steps; ++r) {
                if (!span_ring_load<SX, Lay::NSUB>(&tmQ, x_full, x_empty, smem + Lay::OFF_X, Lay::TILE_BYTES, r,
                                                   i * 128, h, z, wctx))
                    break;
                ix = r + 1;
                if constexpr (SG::kAux == 2) {
                    if (!span_ring_load<SY, Lay::NSUB>(&tmDO, y_full, y_empty, smem + Lay::OFF_Y, Lay::TILE_BYTES, r,
                                                       i * 128, h, z, wctx))
                        break;
                    iy = r + 1;
                }
                if (++i > I1) {
                    i = I0;
                    ++h;
                }
            }
            mbar_wait_drain(res_full, 0, p.timeout_ns);
            ring_drain<SX>(x_full, ix, p.timeout_ns);
            ring_drain<SY>(y_full, iy, p.timeout_ns);
        }
    } else if (SG::kAux > 2 && warp == 2) {
        if (lane == 0) {
            int iy = 0, i = first_tile, h = head0;
            for (int r = 0; r < steps; ++r) {
                if (!span_ring_load<SY, Lay::NSUB>(&tmDO, y_full, y_empty, smem + Lay::OFF_Y, Lay::TILE_BYTES, r,
                                                   i * 128, h, z, wctx))
                    break;
                iy = r + 1;
                if (++i > I1) {
                    i = I0;
                    ++h;
                }
            }
            ring_drain<SY>(y_full, iy, p.timeout_ns);
        }
    } else if (warp == 1) {
        // the whole warp runs converged; elect.sync picks the issuing lane
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, wctx));
        };
        const uint32_t idesc_s = idesc_bf16_f32(128, SG::kStep, false, false);
        const uint32_t idesc_kv = idesc_bf16_f32(128, D, false, true);
        const uint32_t sK = smem_u32(smem + Lay::OFF_A), sV = smem_u32(smem + Lay::OFF_B);
        const uint32_t xring = smem_u32(smem + Lay::OFF_X), yring = smem_u32(smem + Lay::OFF_Y);
        // rows of step r (part r % NP of tile r / NP) in its slot
        auto qrows = [&](int r) { return xring + (r / NP % SX) * Lay::TILE_BYTES + (r % NP) * Lay::PART_BYTES; };
        auto dorows = [&](int r) { return yring + (r / NP % SY) * Lay::TILE_BYTES + (r % NP) * Lay::PART_BYTES; };
        constexpr uint32_t kDescHi = desc_hi(1024);
        auto issue_xyT = [&](uint32_t col, uint32_t xbase, uint32_t ybase) {
            const uint32_t x_lo = desc_lo(xbase, 16), y_lo = desc_lo(ybase, 16);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t koff = ((kk >> 2) * Lay::SUB_BYTES + (kk & 3) * 32) >> 4;
                mma_ss_lhw(tmem + col, x_lo + koff, y_lo + koff, kDescHi, idesc_s, kk > 0 ? 1u : 0u);
            }
        };
        // acc += A(TMEM, packed over `acol`) * B (a step's query rows, MN-major)
        auto issue_acc = [&](uint32_t acc, uint32_t acol, uint32_t bbase, bool first) {
            const uint32_t b_lo = desc_lo(bbase, Lay::SUB_BYTES);
#pragma unroll
            for (int kk = 0; kk < SG::kStep / 16; ++kk)
                mma_ts_lhw(tmem + acc, tmem + acol + SG::packed_col(kk), b_lo + kk * ((16 * 128) >> 4), kDescHi,
                           idesc_kv, (!first || kk > 0) ? 1u : 0u);
        };
        const int all = steps * NP;
        // (a block without a step still waits for its resident tiles, whose place its sums take)
        bool ok = wait(res_full, 0) && (!SPLIT || steps > 0) && wait(&x_full[0], 0) && wait(&y_full[0], 0);
        if (ok) {
            tc_fence_after();
            issue_xyT(kColS, sK, qrows(0));
            mma_commit_w(s_full);
            issue_xyT(kColDP, sV, dorows(0));
            mma_commit_w(dp_full);
        }
        int left = I1 + 1 - first_tile;          // query tiles left of this head
        for (int r = 0; ok && r < all; ++r) {
            const bool more = r + 1 < all;
            const int t = r / NP, t1 = (r + 1) / NP;      // tiles of this step and the next
            const bool opens = NP == 1 || (r + 1) % NP == 0, closes = r % NP == NP - 1;
            if (more) {
                if (opens && !(ok = wait(&x_full[t1 % SX], (t1 / SX) & 1))) break;
                if (!(ok = wait(s_free, r & 1))) break;
                tc_fence_after();
                issue_xyT(kColS, sK, qrows(r + 1));
                mma_commit_w(s_full);
            }
            if (ragged && left == 1 && r % NP == 0) {
                // S^T and dP^T may still be reading these rows: as columns that are masked
                zero_tile_rows<Lay::NSUB>(smem + Lay::OFF_Y + (t % SY) * Lay::TILE_BYTES, n & 127);
                zero_tile_rows<Lay::NSUB>(smem + Lay::OFF_X + (t % SX) * Lay::TILE_BYTES, n & 127);
            }
            if (!(ok = wait(p_ready, r & 1))) break;
            tc_fence_after();
            issue_acc(kColDV, kColDP, dorows(r), r == 0);       // dV += P^T dO
            if (NP == 1) mma_commit_w(&y_empty[t % SY]);
            if (!(ok = wait(ds_ready, r & 1))) break;
            tc_fence_after();
            issue_acc(kColDK, kColDP + SG::kPacked, qrows(r), r == 0);  // dK += dS^T Q
            if (closes) {
                if (NP > 1) mma_commit_w(&y_empty[t % SY]);
                mma_commit_w(&x_empty[t % SX]);
                if (--left == 0) left = per_head;
            }
            if (more) {
                // dP^T of r + 1 overwrites P^T and dS^T of r, read by the two MMAs just
                // issued (MMAs run in issue order)
                if (opens && !(ok = wait(&y_full[t1 % SY], (t1 / SY) & 1))) break;
                tc_fence_after();
                issue_xyT(kColDP, sV, dorows(r + 1));
                mma_commit_w(dp_full);
            }
        }
        mma_commit_w(drain);
        mbar_wait_drain(drain, 0, p.timeout_ns);
        __syncwarp();
    } else if (warp >= SG::kAux) {
        const int w = (warp - SG::kAux) >> 2;      // warpgroup: query columns [kCols w, kCols (w + 1))
        const int quarter = warp & 3;
        const int key = k0 + quarter * 32 + lane;
        const uint32_t lane_bits = static_cast<uint32_t>(quarter * 32) << 16;
        const size_t roff = (static_cast<size_t>(z) * L + key) * (static_cast<size_t>(p.Hk) * D) +
                            static_cast<size_t>(kvh) * D;
        constexpr int kOut = SG::NG / 2;      // warpgroups to an output
        const bool is_dv = w < kOut;
        __nv_bfloat16 *dst = (is_dv ? p.dv : p.dk) + roff;
        const int2 *clean = p.clean + static_cast<size_t>(z) * tiles * 128 + SG::kCols * w;
        const uint32_t tS = tmem + lane_bits + kColS + SG::kCols * w;
        const uint32_t tD = tmem + lane_bits + kColDP + SG::kCols * w;
        const float bias = bias_of(p.bias_z, p.bias, z);
        const bool keys_there = k0 + quarter * 32 + 32 <= n;
        int i = first_tile, h = head0, part = 0;
        ScoreCoef cf = make_score<SCORE>(p.alpha, bias, p.cap, SCORE & kScoreSlope ? p.slopes[h] : 0.0f);
        bool ok = true;
        ScorePause pause = score_pause(cf);
        for (int r = 0; r < steps * NP; ++r) {
            const int4 t = hull[i];
            const bool whole = t.z <= k0 && t.w >= k1;
            const int row0 = i * 128 + part * SG::kStep;
            ok = span_dkdv_tile<D, MODE, SCORE>(tS, tD, s_full, s_free, dp_full, p_ready, ds_ready, r & 1, cf, key,
                                                row0 + SG::kCols * w, whole, keys_there, clean + row0, pause, wctx);
            if (!ok) break;
            if (++part < NP) continue;
            part = 0;
            if (++i > I1) {
                i = I0;
                ++h;
                if (SCORE & kScoreSlope && r + 1 < steps * NP)
                    cf = make_score<SCORE>(p.alpha, bias, p.cap, p.slopes[h]);
            }
        }
        // every MMA of this CTA has finished once the MMA warp's final commit lands
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(drain, 0, wctx));
        if (ok) {
            tc_fence_after();
            const uint32_t sums = tmem + lane_bits + (is_dv ? kColDV : kColDK);
            const int col = (w % kOut) * (D / kOut);
            if constexpr (SPLIT)
                split_leave(reinterpret_cast<float4 *>(smem), sums + col, (is_dv ? 0 : D) + col, D / kOut,
                            quarter * 32 + lane, steps == 0);
            else
                store_row_from_tmem<D>(sums, dst, key < L, key < n, is_dv ? 1.0f : p.alpha, col, D / kOut);
        }
    }

    __syncwarp();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, Lay::TMEM_COLS);
    }
    if constexpr (SPLIT) {
        cluster_meet();
        split_add(reinterpret_cast<const float4 *>(smem), 2 * D / 8, at.rank, split, threadIdx.x, SG::kThreads,
                  [&](int octet, int r, const float (&x)[8]) {
                      const int j = k0 + r;
                      if (j >= L) return;
                      const bool dv = octet < D / 8;
                      const size_t row = ((static_cast<size_t>(z) * L + j) * p.Hk + kvh) * D;
                      reinterpret_cast<uint4 *>((dv ? p.dv : p.dk) + row)[octet % (D / 8)] =
                          split_pack(x, dv ? 1.0f : p.alpha, j < n);
                  });
        cluster_meet();     // the others may still read this block's sums
    }
}

}  // namespace sigattn
