// Forward of the masked attention (span_score.cuh), bf16: one CTA per one or two
// (SpanTiles) 128-row query tiles of one (sample, head), the structure of the
// padding-only forward at D = 128 (fwd_sm100.cuh), with these differences:
//
//  - the CTA reads its rows' spans first; tile t visits the key tiles of its
//    rows' hull only, [j0_t, j1_t), and the rings stream the union.  Causal tiles
//    so cost their visible tiles plus half a diagonal tile each, and packed
//    documents cost what their own keys cost;
//  - long samples start first, and of a sample the last rows, which see the
//    most keys under causal spans: the short blocks fill in behind.  Where all
//    keys and values fit L2 this goes over all heads of a sample at once;
//    otherwise head by head, so that the blocks running at one time share theirs;
//  - query head h reads key head h / (H / Hk);
//  - a warp masks a 64-key half only where one of its rows does not see all of
//    it, and writes zeros without a score where none sees any (the rows' bounds
//    are in registers; whole tiles pay two votes);
//  - the MMA warp zeroes the value rows at or beyond n of the last key tile
//    while the sigma warps work on its scores, so that NaN in padding never
//    meets the product.
//
// P is rounded to bf16 before its product with V (span_score.cuh says why); O is summed
// in fp32 and rounded once.
//
// Bound: as the padding-only forward, one MUFU op per score (two with a cap)
// against 4 D tensor FLOP; at D = 128 without a cap the two pipes balance.
#pragma once

#include "fwd_sm100.cuh"
#include "span_score.cuh"
#include "span_split.cuh"

namespace sigattn {

struct SpanFwdParams {
    __nv_bfloat16 *o;
    SpanSource src;
    int H, group;          // query heads, query heads per key head
    float alpha, bias, cap;
    const float *bias_z;   // device float[Z] or null
    const float *slopes;   // device float[H] or null
    int heads_first;       // grid (heads, pairs, samples) instead of (pairs, heads, samples)
    unsigned split;        // blocks of a cluster that share the tiles (1: none); x is that much wider
    uint64_t timeout_ns;
};

// Query tiles of one CTA, and CTAs that share an SM.  At D = 64 tensor memory and
// shared memory hold two CTAs of one tile, whose starts and ends overlap the
// other's work; against one CTA of two tiles: packed documents 53.1 -> 46.5 us, capped
// and ragged 64.9 -> 56.6 us, causal 8K 174.7 -> 154.5 us, window 8K 86.3 -> 69.4 us, full
// capped 4K 272.5 -> 281 us (keys and values are read twice as often).  At D = 128 they do
// not fit.
template <int D>
struct SpanTiles {
    static constexpr int N = D == 64 ? 1 : 2, kPerSm = 2 / N;
    static constexpr int kThreads = 128 + 256 * N;
    static constexpr int KS = D == 64 ? 2 : FwdStages<D>::K, VS = D == 64 ? 3 : FwdStages<D>::V;
};

template <int D>
struct SpanFwdLayout {
    static constexpr int NT = SpanTiles<D>::N, KS = SpanTiles<D>::KS, VS = SpanTiles<D>::VS;
    static constexpr int NSUB = D / 64;
    static constexpr int SUB_BYTES = 128 * 64 * 2;
    static constexpr int TILE_BYTES = NSUB * SUB_BYTES;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + NT * TILE_BYTES;
    static constexpr int OFF_V = OFF_K + KS * TILE_BYTES;
    static constexpr int OFF_BAR = OFF_V + VS * TILE_BYTES;
    // q_full, k_full[KS], k_empty[KS], v_full[VS], v_empty[VS], drain, then per
    // (part, tile): S ready, P ready
    static constexpr int NBAR = 2 + 2 * KS + 2 * VS + 4 * NT;
    static constexpr int OFF_TMEM = OFF_BAR + NBAR * 8;
    static constexpr int OFF_ABORT = OFF_TMEM + 8;
    static constexpr int OFF_HULL = OFF_ABORT + 8;                 // {lo, hi} of each 32 rows
    static constexpr int SMEM_ALLOC = OFF_HULL + 32 * NT + 1024;
    static constexpr uint32_t COL_S = 0, COL_O = 128 * NT;         // S_t, then O_t
    static constexpr uint32_t TMEM_COLS = NT * (128 + D) > 256 ? 512 : 256;
    static_assert(NT * (128 + D) <= TMEM_COLS && SpanTiles<D>::kPerSm * TMEM_COLS <= 512, "TMEM budget");
    static_assert(NT * D * 128 * 4 <= OFF_BAR, "a split's sums fit the tiles' place");
    static_assert(SpanTiles<D>::kPerSm * (SMEM_ALLOC + 1024) <= 228 * 1024, "shared memory budget");
};

// Parts that a 128-key tile's scores are handed over in.  Two halves let a sigma
// warpgroup start as soon as its own 64 keys are there, and its scores of the
// next tile be computed while the other warpgroup still works; but an N = 64
// score MMA runs at 2/3 of the N = 128 rate (shared-memory reads).  That pays
// where the MUFU is the bound: D = 64 packed documents 63.2 -> 59.8 us, D = 128
// with a cap 224.7 -> 213.7 us, but causal L = 16384 at D = 128 without one 1066 ->
// 1211 us.
template <int D, int SCORE>
struct SpanParts {
    static constexpr int N = D == 64 || (SCORE & kScoreCap) ? 2 : 1;
};

template <int D, int MODE, int SCORE, bool SPLIT>
__global__ void __launch_bounds__(SpanTiles<D>::kThreads, SpanTiles<D>::kPerSm)
    span_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const SpanFwdParams p) {
    using Lay = SpanFwdLayout<D>;
    constexpr int NT = Lay::NT, KS = Lay::KS, VS = Lay::VS;
    constexpr int NP = SpanParts<D, SCORE>::N, PK = 128 / NP;   // parts of a key tile, keys of a part
    constexpr int kThreads = SpanTiles<D>::kThreads;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_1k(smem_raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Lay::OFF_BAR);
    uint64_t *q_full = bars;
    uint64_t *k_full = bars + 1;
    uint64_t *k_empty = k_full + KS;
    uint64_t *v_full = k_empty + KS;
    uint64_t *v_empty = v_full + VS;
    uint64_t *drain = v_empty + VS;
    uint64_t *s_full = drain + 1;              // [part][tile]
    uint64_t *p_full = s_full + 2 * NT;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Lay::OFF_TMEM);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + Lay::OFF_ABORT);
    int2 *hull = reinterpret_cast<int2 *>(smem + Lay::OFF_HULL);

    const int warp = warp_id(), lane = lane_id();
    const int split = SPLIT ? static_cast<int>(p.split) : 1;
    const SplitPlace at = split_place(split);
    const int z = span_sample(p.src.seqlens, gridDim.z, blockIdx.z), h = p.heads_first ? at.x : blockIdx.y;
    const int kvh = h / p.group;
    const int qtile0 = NT * (p.heads_first ? static_cast<int>(gridDim.y - 1 - blockIdx.y) : at.wide - 1 - at.x);
    const int L = p.src.L;
    const int n = span_tokens(p.src, z);
    const int loads = min(max((n + 127) / 128 - qtile0, 0), NT);     // query tiles below n
    if (warp < 4 * NT) {
        const int2 r = row_span(p.src, z, qtile0 * 128 + static_cast<int>(threadIdx.x), n);
        const int lo = __reduce_min_sync(0xffffffffu, r.x < r.y ? r.x : INT_MAX);
        const int hi = __reduce_max_sync(0xffffffffu, r.y);
        if (lane == 0) hull[warp] = make_int2(lo, hi);
    }
    if (threadIdx.x == 64) {
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        for (int s = 0; s < KS; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], 1);
        }
        for (int s = 0; s < VS; ++s) {
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], 1);
        }
        for (int u = 0; u < NT * NP; ++u) {
            mbar_init(&s_full[u], 1);
            mbar_init(&p_full[u], 256 / NP);  // the sigma warpgroups of this tile and part
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
        // the query tiles fly while the rest of the block sets up
        if (loads > 0) mbar_arrive_expect_tx(q_full, loads * Lay::TILE_BYTES);
        for (int t = 0; t < loads; ++t)
            for (int s = 0; s < Lay::NSUB; ++s)
                tma_load_4d(&tmQ, q_full, smem + Lay::OFF_Q + t * Lay::TILE_BYTES + s * Lay::SUB_BYTES, 64 * s, h,
                            (qtile0 + t) * 128, z);
    }
    __syncthreads();
    // key tiles [j0[t], j1[t]) of query tile t, and [J0, J1) of all; an empty tile
    // has j0 = j1 = 0
    int j0[NT], j1[NT], J0 = INT_MAX, J1 = 0, live = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        int lo = INT_MAX, hi = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int2 r = hull[4 * t + w];
            lo = min(lo, r.x);
            hi = max(hi, r.y);
        }
        j0[t] = hi > 0 ? lo / 128 : 0;
        j1[t] = (hi + 127) / 128;
        if (hi > 0) {
            J0 = min(J0, j0[t]);
            J1 = max(J1, j1[t]);
            ++live;
        }
    }
    const size_t row_stride = static_cast<size_t>(p.H) * D;
    if (live == 0) {
        // no row sees a key: zeros, written by every thread
        const int r0 = qtile0 * 128, rows = min(128 * NT, L - r0);
        constexpr int V4 = D / 8;
        for (int e = threadIdx.x; e < rows * V4; e += kThreads) {
            uint4 *dst = reinterpret_cast<uint4 *>(p.o + (static_cast<size_t>(z) * L + r0 + e / V4) * row_stride +
                                                   static_cast<size_t>(h) * D);
            if (at.rank == 0) dst[e % V4] = make_uint4(0u, 0u, 0u, 0u);
        }
        if (threadIdx.x == 0 && loads > 0) mbar_wait_drain(q_full, 0, p.timeout_ns);
        if constexpr (SPLIT) cluster_skip();
        return;
    }
    if constexpr (SPLIT) {
        // this block's part of the key tiles
        const int a = J0 + split_step(J1 - J0, at.rank, split), b = J0 + split_step(J1 - J0, at.rank + 1, split);
        J0 = a;
        J1 = b;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            j0[t] = max(j0[t], a);
            j1[t] = min(j1[t], b);
            if (j0[t] >= j1[t]) j0[t] = j1[t] = 0;
        }
    }
    const int steps = J1 - J0;
    // the last key tile, when n ends inside it: its value rows are cleaned
    const bool ragged = (n & 127) != 0 && J1 == (n + 127) / 128;
    // the first key tile flies while tensor memory is allocated (0 to 3% at D = 128; the
    // same in the backward, whose blocks have their resident tiles in flight by then, was
    // 0 to 4% slower)
    auto load_k = [&](int r) {
        uint8_t *to = smem + Lay::OFF_K + r % KS * Lay::TILE_BYTES;
        mbar_arrive_expect_tx(&k_full[r % KS], Lay::TILE_BYTES);
        for (int s = 0; s < Lay::NSUB; ++s)
            tma_load_4d(&tmK, &k_full[r % KS], to + s * Lay::SUB_BYTES, 64 * s, kvh, (J0 + r) * 128, z);
    };
    auto load_v = [&](int r) {
        uint8_t *to = smem + Lay::OFF_V + r % VS * Lay::TILE_BYTES;
        mbar_arrive_expect_tx(&v_full[r % VS], Lay::TILE_BYTES);
        for (int s = 0; s < Lay::NSUB; ++s)
            tma_load_4d(&tmV, &v_full[r % VS], to + s * Lay::SUB_BYTES, 64 * s, kvh, (J0 + r) * 128, z);
    };
    const int early = min(steps, 1);
    if (warp == 0 && lane == 0 && early > 0) load_k(0);
    if (warp == 2 && lane == 0 && early > 0) load_v(0);
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
            int issued = early;
            for (int r = early; r < steps; ++r) {
                if (r >= KS && !mbar_wait(&k_empty[r % KS], ((r / KS) - 1) & 1, wctx)) break;
                load_k(r);
                issued = r + 1;
            }
            // every issued load must land before the CTA's shared memory is released
            mbar_wait_drain(q_full, 0, p.timeout_ns);
            for (int r = (issued > KS ? issued - KS : 0); r < issued; ++r)
                mbar_wait_drain(&k_full[r % KS], (r / KS) & 1, p.timeout_ns);
        }
    } else if (warp == 2) {
        if (lane == 0) {
            int issued = early;
            for (int r = early; r < steps; ++r) {
                if (r >= VS && !mbar_wait(&v_empty[r % VS], ((r / VS) - 1) & 1, wctx)) break;
                load_v(r);
                issued = r + 1;
            }
            for (int r = (issued > VS ? issued - VS : 0); r < issued; ++r)
                mbar_wait_drain(&v_full[r % VS], (r / VS) & 1, p.timeout_ns);
        }
    } else if (warp == 1) {
        // the whole warp runs converged; elect.sync picks the issuing lane
        auto wt = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, wctx));
        };
        const uint32_t idesc_s = idesc_bf16_f32(128, PK, false, false);
        const uint32_t idesc_o = idesc_bf16_f32(128, D, false, true);
        const uint32_t sQ = smem_u32(smem + Lay::OFF_Q);
        const uint32_t sK = smem_u32(smem + Lay::OFF_K);
        const uint32_t sV = smem_u32(smem + Lay::OFF_V);
        constexpr uint32_t kDescHi = desc_hi(1024);
        // scores of query tile t against part c of the key tile at kbase
        auto issue_s = [&](int t, int c, uint32_t kbase) {
            const uint32_t q_lo = desc_lo(sQ + t * Lay::TILE_BYTES, 16), k_lo = desc_lo(kbase + c * PK * 128, 16);
            const uint32_t d_tmem = tmem + Lay::COL_S + 128 * t + PK * c;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t koff = ((kk >> 2) * Lay::SUB_BYTES + (kk & 3) * 32) >> 4;
                mma_ss_lhw(d_tmem, q_lo + koff, k_lo + koff, kDescHi, idesc_s, kk > 0 ? 1u : 0u);
            }
            mma_commit_w(&s_full[NT * c + t]);
        };
        auto issue_pv = [&](int t, int c, uint32_t vbase, bool first) {
            const uint32_t d_tmem = tmem + Lay::COL_O + D * t;
            const uint32_t a_tmem = tmem + Lay::COL_S + 128 * t;
            const uint32_t v_lo = desc_lo(vbase, Lay::SUB_BYTES);
            // 16 keys = 8 packed columns per step; keys 64-127 sit 32 columns further on
#pragma unroll
            for (int kk = c * PK / 16; kk < (c + 1) * PK / 16; ++kk)
                mma_ts_lhw(d_tmem, a_tmem + kk * 8 + (kk >= 4 ? 32 : 0), v_lo + kk * ((16 * 128) >> 4), kDescHi,
                           idesc_o, (!first || kk > 0) ? 1u : 0u);
        };
        // Per key tile j and part c: for each query tile that visits j, O_t += P V
        // over the part's keys once its P is there, then the same part's scores of
        // j + 1 over it.  MMAs from one thread run in issue order, so P has been
        // read before the next scores are written.  A key tile that neither visits
        // (a gap between the two hulls) passes through the rings unread.
        // (a block without a step still waits for its query tiles, whose place its sums take)
        bool ok = wt(q_full, 0) && (!SPLIT || steps > 0) && wt(&k_full[0], 0);
        if (ok) {
            tc_fence_after();
#pragma unroll
            for (int u = 0; u < NT * NP; ++u)
                if (j0[u % NT] == J0 && J0 < j1[u % NT]) issue_s(u % NT, u / NT, sK);
            mma_commit_w(&k_empty[0]);
        }
        for (int r = 0; ok && r < steps; ++r) {
            const int j = J0 + r, sv = r % VS, sk = (r + 1) % KS;
            const bool more = r + 1 < steps;
            const uint32_t vbase = sV + sv * Lay::TILE_BYTES;
            const uint32_t knext = sK + sk * Lay::TILE_BYTES;
            if (!(ok = wt(&v_full[sv], (r / VS) & 1))) break;
            if (!more && ragged)
                zero_tile_rows<Lay::NSUB>(smem + Lay::OFF_V + sv * Lay::TILE_BYTES, n & 127);
            bool have_k = false;
#pragma unroll
            for (int u = 0; u < NT * NP; ++u) {
                const int t = u % NT, c = u / NT;
                if (j >= j0[t] && j < j1[t]) {
                    if (!(ok = wt(&p_full[u], (j - j0[t]) & 1))) break;
                    tc_fence_after();
                    issue_pv(t, c, vbase, j == j0[t] && c == 0);
                }
                if (u == NT * NP - 1) mma_commit_w(&v_empty[sv]);
                if (more && j + 1 >= j0[t] && j + 1 < j1[t]) {
                    if (!have_k && !(ok = wt(&k_full[sk], ((r + 1) / KS) & 1))) break;
                    have_k = true;
                    tc_fence_after();
                    issue_s(t, c, knext);
                }
            }
            if (!ok) break;
            if (more) {
                if (!have_k && !(ok = wt(&k_full[sk], ((r + 1) / KS) & 1))) break;
                mma_commit_w(&k_empty[sk]);
            }
        }
        // no MMA may still be running when TMEM is released
        mma_commit_w(drain);
        mbar_wait_drain(drain, 0, p.timeout_ns);
        __syncwarp();
    } else if (warp >= 4) {
        // sigma warpgroups: warpgroup g works on query tile t = g / 2, key columns
        // [64 c, 64 c + 64) of each key tile, c = g % 2
        const int g = (warp - 4) >> 2;
        const int t = g >> 1, c = g & 1;
        const int part = NT * (c * NP / 2) + t;   // barriers of this tile and part
        const int quarter = warp & 3;  // TMEM lane quarter this warp may access
        const uint32_t lane_bits = static_cast<uint32_t>(quarter * 32) << 16;
        const int row = (qtile0 + t) * 128 + quarter * 32 + lane;
        const int2 span = row_span(p.src, z, row, n);
        const int ja = t ? j0[NT - 1] : j0[0], jb = t ? j1[NT - 1] : j1[0];
        bool ok = true;
        if (jb > 0) {
            const ScoreCoef cf = make_score<SCORE>(p.alpha, bias_of(p.bias_z, p.bias, z), p.cap,
                                                         SCORE & kScoreSlope ? p.slopes[h] : 0.0f);
            const uint32_t tS = tmem + lane_bits + Lay::COL_S + 128 * t + 64 * c;
            ScorePause pause = score_pause(cf);
            for (int j = ja; j < jb; ++j) {
                ok = __all_sync(0xffffffffu, mbar_wait(&s_full[part], (j - ja) & 1, wctx));
                if (!ok) break;
                tc_fence_after();
                const int key0 = j * 128 + 64 * c;   // first key of this half
                const bool whole = __all_sync(0xffffffffu, span.x <= key0 && span.y >= key0 + 64);
                const bool some = whole || __any_sync(0xffffffffu, span.x < key0 + 64 && span.y > key0);
                // two chunks of 32 scores per thread; P of chunk u lies over S
                // columns [16 u, 16 u + 16) of this half, already read
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t pk[16];
                    if (some) {
                        uint32_t r[32];
                        tmem_ld32(tS + 32 * u, r);
                        score_chunk<MODE, SCORE, false, true>(r, cf, static_cast<float>(row - key0 - 32 * u), pk, nullptr,
                                                              pause, whole);
                        if (!whole) keep_bits(pk, bit_range(span.x - key0 - 32 * u, span.y - key0 - 32 * u));
                    } else {
                        // none of the warp's rows sees any of the half
#pragma unroll
                        for (int i = 0; i < 16; ++i) pk[i] = 0u;
                    }
                    tmem_st16(tS + 16 * u, pk);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&p_full[part]);
            }
            // every MMA of this CTA has finished once the MMA warp's final commit lands
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(drain, 0, wctx));
        }
        // epilogue: warpgroup g writes columns [c D/2, c D/2 + D/2) of query tile t
        constexpr int HALF = D / 2;
        __nv_bfloat16 *orow = p.o + (static_cast<size_t>(z) * L + row) * row_stride +
                              static_cast<size_t>(h) * D + c * HALF;
        if constexpr (SPLIT) {
            // the sums take the place of tiles that the other query tile may still use
            if (jb == 0) ok = __all_sync(0xffffffffu, mbar_wait(drain, 0, wctx));
            if (ok) {
                tc_fence_after();
                split_leave(reinterpret_cast<float4 *>(smem), tmem + lane_bits + Lay::COL_O + D * t + c * HALF,
                            D * t + c * HALF, HALF, quarter * 32 + lane, jb == 0);
            }
        } else if (jb > 0) {
            if (ok) {
                tc_fence_after();
                const uint32_t tO = tmem + lane_bits + Lay::COL_O + D * t + c * HALF;
                const bool valid = span.x < span.y;
#pragma unroll
                for (int cc = 0; cc < HALF / 32; ++cc) {
                    uint32_t r[32];
                    tmem_ld32(tO + 32 * cc, r);
                    if (row < L) {
                        uint4 *dst = reinterpret_cast<uint4 *>(orow + 32 * cc);
#pragma unroll
                        for (int v4 = 0; v4 < 4; ++v4) {
                            uint4 w;
                            w.x = valid ? pack_bf16x2(__uint_as_float(r[8 * v4 + 0]), __uint_as_float(r[8 * v4 + 1])) : 0u;
                            w.y = valid ? pack_bf16x2(__uint_as_float(r[8 * v4 + 2]), __uint_as_float(r[8 * v4 + 3])) : 0u;
                            w.z = valid ? pack_bf16x2(__uint_as_float(r[8 * v4 + 4]), __uint_as_float(r[8 * v4 + 5])) : 0u;
                            w.w = valid ? pack_bf16x2(__uint_as_float(r[8 * v4 + 6]), __uint_as_float(r[8 * v4 + 7])) : 0u;
                            dst[v4] = w;
                        }
                    }
                }
            }
        } else if (row < L) {
            // no row of this tile sees a key: exact zeros
            uint4 *dst = reinterpret_cast<uint4 *>(orow);
#pragma unroll
            for (int v4 = 0; v4 < HALF / 8; ++v4) dst[v4] = make_uint4(0u, 0u, 0u, 0u);
        }
    }

    // every warp converges before the block-wide barrier (the producer roles
    // ran on one lane)
    __syncwarp();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, Lay::TMEM_COLS);
    }
    if constexpr (SPLIT) {
        cluster_meet();
        split_add(reinterpret_cast<const float4 *>(smem), NT * D / 8, at.rank, split, threadIdx.x, kThreads,
                  [&](int octet, int r, const float (&x)[8]) {
                      const int i = (qtile0 + octet / (D / 8)) * 128 + r;
                      if (i >= L) return;
                      const int2 s = row_span(p.src, z, i, n);
                      reinterpret_cast<uint4 *>(p.o + (static_cast<size_t>(z) * L + i) * row_stride +
                                                static_cast<size_t>(h) * D)[octet % (D / 8)] =
                          split_pack(x, 1.0f, s.x < s.y);
                  });
        cluster_meet();     // the others may still read this block's sums
    }
}

}  // namespace sigattn
