// Attention of new tokens against a paged cache whose samples may share one
// prefix.
//
// The batch's keys are a prefix of `prefix_len` tokens (pages prefix_table) that
// every sample sees, followed by each sample's own tokens (pages page_table[z],
// seqlens_k[z] of them).  A sample's n_q queries are its last n_q tokens: query l
// stands at own place n - n_q + l and sees the prefix and its own places up to that.
//
// sigma needs no row normalisation, so O is the plain sum of a prefix part and
// an own part, and each of them of the parts of any split of the keys: no running
// maximum, no rescaling, nothing but fp32 partial sums to add at the end.
//
// Two kernels compute, one adds up:
//
//  paged_prefix_kernel (tcgen05): the prefix against the rows of all samples'
//    tokens and of all query heads of a key head, 256 rows a block, so that the
//    prefix is read once per 256 rows and not once per sample.  The key range is
//    split over blocks until they fill the device.
//  paged_tiles_kernel (mma.sync): the samples' own keys, and the prefix where the
//    batch has few rows.  Work is a list of items, each a run of 64-key tiles,
//    alike for every key head:
//      prefix items: a tile of the rows above;
//      own items:    (sample, tile of its query rows).
//    The tiles of a head's items form one sequence that is cut evenly over groups
//    of blocks (group g of B <= T takes [g T / B, (g + 1) T / B)), whatever the
//    lengths; the blocks of a group each take a head, so that the heads' rows of
//    one place, which lie side by side in memory, are read at about the same time
//    (block by block over one head's keys after the other's, 128-byte rows came in at
//    4.4 TB/s).  A producer warp walks a block's range with TMA, across item
//    borders, and the consumer warps write one fp32 partial per item that they
//    touch.  Walking on either starts a new group or a new item, so (group + item)
//    numbers a head's partials without a table.
//  paged_join_kernel adds the partials of each row in a fixed order (the result
//    does not depend on scheduling) and rounds once.
//
// The prefix kernel and the tile kernel with 64 rows round P to one bf16 number, as the
// masked forward does; with fewer rows the tile kernel keeps it in two (PagedItem).
//
// Bound: memory.  Every key and value is read once per row tile; a 64-key tile
// at D = 128 is 32 KB, 1.4 kclk of an SM's share of HBM.  The few rows of one
// sample leave a tcgen05 tile of 128 rows mostly empty and its sigma warps with
// 128 rows of work; mma.sync works on 16 rows at a time.  Many rows turn that
// round (64 rows of mma.sync take 3 kclk a tile), hence the two kernels.
#pragma once

#include "cache_append.cuh"
#include "span_fwd_sm100.cuh"

namespace sigattn {

struct PagedParams {
    const __nv_bfloat16 *q;
    __nv_bfloat16 *o;
    const int *page_table, *seqlens_k, *seqlens_q, *prefix_table, *prefix_len;
    int Z, L, H, Hk, group;
    int pages, page_shift, max_pages, prefix_pages;
    float alpha, bias, cap;
    const float *bias_z, *slopes;
    float *part;          // [key head][group + item][kPagedPartRows][D]
    int2 *groups_of;      // [key head][item] first and last group of each item that has tiles
    int heads_wide;       // blocks of a group: the key heads, or the grid where it has fewer
    int groups, items;    // groups of the grid; items of a head
    int prefix_warps, own_warps;   // warps along the rows (1, 2, 4): row tiles of 16 times that
    int prefix_rt, own_rt;         // row tiles of the prefix and of a sample, per key head
    // the prefix kernel, when it runs (splits > 0; the tile kernel then leaves the prefix out)
    float *prefix_part;   // [split][key head][pair][256][D]
    int splits, pairs;    // blocks along the keys; pairs of row tiles
    int tile_tokens;      // tokens of a row tile: 128 / group
    int *status;
    uint64_t timeout_ns;
};

constexpr int kPagedConsumers = 128;
constexpr int kPagedThreads = kPagedConsumers + 32;
constexpr int kPagedTile = 64;    // keys per tile
// Rows of one partial: each of the four warps writes its own 16 (WM warps along
// the rows, 4 / WM along the keys of a tile), so that nothing waits at an item's
// end; the join adds the warps along the keys as well.
constexpr int kPagedPartRows = 64;

template <int D>
struct PagedLayout {
    static constexpr int kStages = D == 128 ? 3 : 4;
    static constexpr int kBlocksPerSm = D == 128 ? 2 : 3;
    static constexpr int NSUB = D / 64;
    static constexpr int kAtom = kPagedTile * 128;             // [64 keys][64 entries], 128-byte swizzle
    static constexpr int kOperand = NSUB * kAtom;              // one K or V tile
    static constexpr int OFF_BAR = kStages * 2 * kOperand;     // full[kStages], empty[kStages]
    static constexpr int OFF_ABORT = OFF_BAR + 2 * kStages * 8;
    static constexpr int OFF_SUMS = OFF_ABORT + 8;             // one int per consumer warp
    static constexpr int OFF_BEFORE = OFF_SUMS + 24;
    static constexpr int bytes(int Z) { return OFF_BEFORE + (Z + 1) * 4 + 1024; }
};

__device__ __forceinline__ int paged_prefix(const PagedParams &p) {
    if (p.prefix_len == nullptr) return 0;
    const int cap = p.prefix_pages << p.page_shift;
    const int n = *p.prefix_len;
    if (n < 0 || n > cap) {
        if (threadIdx.x == 0) record_status(p.status, kStatusSeqlenRange);
        return min(max(n, 0), cap);
    }
    return n;
}

// {own keys, queries} of sample z, clamped.
__device__ __forceinline__ int2 paged_lengths(const PagedParams &p, int z) {
    const int cap = p.max_pages << p.page_shift;
    int nk = p.seqlens_k[z], nq = p.seqlens_q[z];
    if (nk < 0 || nk > cap || nq < 0 || nq > p.L || nq > nk) {
        record_status(p.status, kStatusSeqlenRange);
        nk = min(max(nk, 0), cap);
        nq = min(min(max(nq, 0), p.L), nk);
    }
    return make_int2(nk, nq);
}

// The shape of the item list.
struct PagedPlan {
    int prefix_tiles, prefix_rows, prefix_rt;   // tiles of the prefix; rows of a row tile; row tiles, an item each
    int own_rows, own_rt;
    int64_t own_first;        // tiles of a head's prefix items: where own items begin
};
__device__ __forceinline__ PagedPlan paged_plan(const PagedParams &p, int prefix) {
    PagedPlan a;
    if (p.splits > 0) prefix = 0;    // the prefix kernel's
    a.prefix_tiles = (prefix + kPagedTile - 1) / kPagedTile;
    a.prefix_rows = 16 * p.prefix_warps;
    a.prefix_rt = p.prefix_rt;
    a.own_rows = 16 * p.own_warps;
    a.own_rt = p.own_rt;
    a.own_first = static_cast<int64_t>(a.prefix_tiles) * a.prefix_rt;
    return a;
}

// A place in the tile sequence of key head kvh.
struct PagedCursor {
    int item;             // number of the item among the head's
    int z;                // sample of an own item, -1 for a prefix item
    int kvh, rt, tile, tiles;
};

__device__ __forceinline__ PagedCursor paged_locate(const PagedPlan &a, int Z, const int *before, int kvh, int64_t t) {
    PagedCursor c;
    c.kvh = kvh;
    if (t < a.own_first) {
        c.item = c.rt = static_cast<int>(t / a.prefix_tiles);
        c.z = -1;
        c.tile = static_cast<int>(t % a.prefix_tiles);
        c.tiles = a.prefix_tiles;
        return c;
    }
    const int64_t u = t - a.own_first;
    const int at = static_cast<int>(u / a.own_rt);
    int lo = 0, hi = Z - 1;             // the last sample with before[z] <= at
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (before[mid] <= at) lo = mid;
        else hi = mid - 1;
    }
    c.z = lo;
    c.tiles = before[lo + 1] - before[lo];
    const int64_t in = u - static_cast<int64_t>(before[lo]) * a.own_rt;
    c.rt = static_cast<int>(in / c.tiles);
    c.tile = static_cast<int>(in % c.tiles);
    c.item = a.prefix_rt + lo * a.own_rt + c.rt;
    return c;
}

// The next tile; the caller knows that there is one.
__device__ __forceinline__ void paged_next(const PagedPlan &a, const int *before, PagedCursor &c) {
    if (++c.tile < c.tiles) return;
    c.tile = 0;
    ++c.item;
    if (++c.rt < (c.z < 0 ? a.prefix_rt : a.own_rt)) return;
    c.rt = 0;
    do {
        ++c.z;            // from -1: the first sample
        c.tiles = before[c.z + 1] - before[c.z];
        c.item = a.prefix_rt + c.z * a.own_rt;
    } while (c.tiles == 0);
}

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// c += a b: 16 x 8 += 16 x 16 by 16 x 8, bf16 operands, fp32 sums
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The two query rows of a thread (accumulator rows lane / 4 and + 8 of its
// warp's 16): where they come from and what they see.
struct PagedRows {
    const __nv_bfloat16 *q[2];   // null: no such row
    int pos[2];                  // place of the query among the item's keys (distances are taken in
                                 // whole numbers: fp32 does not hold places beyond 2^24)
    int limit[2];                // keys below it are seen
};

// Everything a block does with the tiles of one item kind: WM warps along the
// rows (16 each), 4 / WM along the keys of a tile.
template <int D, int SCORE, int WM>
struct PagedItem {
    using Lay = PagedLayout<D>;
    static constexpr int WK = 4 / WM, KW = kPagedTile / WK, NK = D / 16;
    uint32_t qf[NK][4];
    float acc[D / 8][4];
    ScoreCoef cf[2];
    PagedRows rows;

    __device__ __forceinline__ void begin(const PagedParams &p, const PagedCursor &c, int prefix) {
        const int lane = lane_id(), wm = warp_id() % WM;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t r = static_cast<int64_t>(c.rt) * (16 * WM) + wm * 16 + lane / 4 + 8 * i;
            const int64_t tok = r / p.group + (c.z < 0 ? 0 : static_cast<int64_t>(c.z) * p.L);
            const int h = c.kvh * p.group + static_cast<int>(r % p.group);
            const bool in = c.z < 0 ? tok < static_cast<int64_t>(p.Z) * p.L : r < static_cast<int64_t>(p.L) * p.group;
            rows.q[i] = nullptr;
            rows.pos[i] = 0;
            rows.limit[i] = 0;
            cf[i] = ScoreCoef{};
            if (!in) continue;
            const int z = static_cast<int>(tok / p.L), l = static_cast<int>(tok % p.L);
            const int2 n = paged_lengths(p, z);
            if (l >= n.y) continue;
            const int at = n.x - n.y + l;     // own place
            rows.q[i] = p.q + (static_cast<size_t>(tok) * p.H + h) * D;
            rows.pos[i] = c.z < 0 ? prefix + at : at;
            rows.limit[i] = c.z < 0 ? prefix : at + 1;
            cf[i] = make_score<SCORE>(p.alpha, bias_of(p.bias_z, p.bias, z), p.cap,
                                            SCORE & kScoreSlope ? p.slopes[h] : 0.0f);
        }
#pragma unroll
        for (int kk = 0; kk < NK; ++kk)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const __nv_bfloat16 *src = rows.q[u & 1];
                qf[kk][u] = src != nullptr
                                ? *reinterpret_cast<const uint32_t *>(src + 16 * kk + 8 * (u >> 1) + 2 * (lane & 3))
                                : 0u;
            }
#pragma unroll
        for (int d = 0; d < D / 8; ++d) acc[d][0] = acc[d][1] = acc[d][2] = acc[d][3] = 0.0f;
    }

    __device__ __forceinline__ void tile(uint32_t sK, uint32_t sV, int key0) {
        const int lane = lane_id(), wk = warp_id() / WM;
        if (!__any_sync(0xffffffffu, max(rows.limit[0], rows.limit[1]) > key0 + wk * KW)) return;
        // distance of this thread's first key; the others' follow in fp32, where a step that
        // rounds is one of 2^24 places or more (a conversion for each pair would go through
        // the MUFU's pipe)
        const int first = key0 + wk * KW + 2 * (lane & 3);
        const float rel[2] = {static_cast<float>(rows.pos[0] - first), static_cast<float>(rows.pos[1] - first)};
#pragma unroll
        for (int g = 0; g < KW / 16; ++g) {
            const int k16 = wk * KW + 16 * g;     // first of 16 keys
            float s[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
            {
                // lanes 0-7: keys 0-7 low half, 8-15: keys 0-7 high half, then keys 8-15
                const int row = k16 + (lane & 7) + ((lane >> 4) << 3);
                const uint32_t base = sK + row * 128;
#pragma unroll
                for (int kk = 0; kk < NK; ++kk) {
                    uint32_t b[4];
                    ldmatrix4(base + (kk >> 2) * Lay::kAtom + (((2 * (kk & 3) + ((lane >> 3) & 1)) ^ (row & 7)) << 4),
                              b);
                    mma16816(s[0], qf[kk], b[0], b[1]);
                    mma16816(s[1], qf[kk], b[2], b[3]);
                }
            }
            // P as a sum of two bf16 numbers, where few rows leave the product far from being
            // the bound (2% of the time for 16 rows): its rounding adds as much to O's error as
            // O's own does (2-norm 1.6e-3 -> 2.3e-3).  A full 64-row tile would lose 13%.
            constexpr bool kSplit = WM < 4;
            uint32_t a[4], low[4];
#pragma unroll
            for (int n8 = 0; n8 < 2; ++n8)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int key = first + 16 * g + 8 * n8;
                    float2 w = score_p2<SCORE>(s[n8][2 * i], s[n8][2 * i + 1], cf[i], rel[i] - static_cast<float>(16 * g + 8 * n8));
                    w.x = key < rows.limit[i] ? w.x : 0.0f;
                    w.y = key + 1 < rows.limit[i] ? w.y : 0.0f;
                    const uint32_t hi = pack_bf16x2(w.x, w.y);
                    a[2 * n8 + i] = hi;
                    if (kSplit)
                        low[2 * n8 + i] =
                            pack_bf16x2(w.x - __uint_as_float(hi << 16), w.y - __uint_as_float(hi & 0xFFFF0000u));
                }
            {
                // lanes 0-7: keys 0-7, 8-15: keys 8-15, then the next 8 columns
                const int row = k16 + (lane & 15);
                const uint32_t base = sV + row * 128;
#pragma unroll
                for (int d = 0; d < D / 16; ++d) {
                    uint32_t b[4];
                    ldmatrix4_trans(base + (d >> 2) * Lay::kAtom + (((2 * (d & 3) + (lane >> 4)) ^ (row & 7)) << 4),
                                    b);
                    mma16816(acc[2 * d], a, b[0], b[1]);
                    mma16816(acc[2 * d + 1], a, b[2], b[3]);
                    if (kSplit) {
                        mma16816(acc[2 * d], low, b[0], b[1]);
                        mma16816(acc[2 * d + 1], low, b[2], b[3]);
                    }
                }
            }
        }
    }

    // Writes the rows that exist: [warp along the keys][row of the tile][D].
    __device__ __forceinline__ void end(float *dst) {
        const int lane = lane_id(), wm = warp_id() % WM, wk = warp_id() / WM;
        dst += (wk * 16 * WM + wm * 16 + lane / 4) * D + 2 * (lane & 3);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (rows.q[i] == nullptr) continue;
#pragma unroll
            for (int d = 0; d < D / 8; ++d)
                *reinterpret_cast<float2 *>(dst + 8 * i * D + 8 * d) = make_float2(acc[d][2 * i], acc[d][2 * i + 1]);
        }
    }
};

// Page number of each of the 16-key groups of tile `tile` that start a box (pages
// hold at least 16 keys), or `pages` where there is no such page: a box there
// lies outside the tensor and arrives as zeros.  Bad numbers are flagged.
template <int KEYS>
__device__ __forceinline__ void paged_numbers(const PagedParams &p, const int *table, int tile, int keys, int box,
                                              int (&page)[KEYS / 16]) {
#pragma unroll
    for (int i = 0; i < KEYS / 16; ++i) {
        const int key = tile * KEYS + 16 * i;
        page[i] = p.pages;
        if ((16 * i) % box == 0 && key < keys) {
            const int n = __ldg(table + (key >> p.page_shift));
            if (n >= 0 && n < p.pages) page[i] = n;
            else record_status(p.status, kStatusPageRange);
        }
    }
}
// Loads a tile of KEYS keys of one operand, box by box.
template <int KEYS, int NSUB>
__device__ __forceinline__ void paged_boxes(const PagedParams &p, const CUtensorMap *map, uint64_t *bar, uint8_t *dst,
                                            int tile, int kvh, int box, const int (&page)[KEYS / 16]) {
    const int mask = (1 << p.page_shift) - 1;
#pragma unroll
    for (int i = 0; i < KEYS / 16; ++i) {
        if ((16 * i) % box != 0) continue;
#pragma unroll
        for (int s = 0; s < NSUB; ++s)
            tma_load_4d(map, bar, dst + s * (KEYS * 128) + i * 16 * 128, 64 * s, kvh, (tile * KEYS + 16 * i) & mask,
                        page[i]);
    }
}

template <int D, int SCORE>
__global__ void __launch_bounds__(kPagedThreads, PagedLayout<D>::kBlocksPerSm)
    paged_tiles_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ PagedParams p) {
    using Lay = PagedLayout<D>;
    constexpr int S = Lay::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_1k(smem_raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Lay::OFF_BAR), *empty = full + S;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + Lay::OFF_ABORT);
    int *sums = reinterpret_cast<int *>(smem + Lay::OFF_SUMS);
    int *before = reinterpret_cast<int *>(smem + Lay::OFF_BEFORE);
    const int tid = threadIdx.x, warp = warp_id(), lane = lane_id();

    grid_release();
    if (tid == kPagedConsumers) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 4);
        }
        *abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    // own tiles of the samples before each: one scan over the batch
    int carry = 0;
    for (int z0 = 0; z0 < p.Z; z0 += kPagedConsumers) {
        const int z = z0 + tid;
        int t = 0;
        if (tid < kPagedConsumers && z < p.Z) {
            const int2 n = paged_lengths(p, z);
            t = n.y > 0 ? (n.x + kPagedTile - 1) / kPagedTile : 0;       // no query: nothing to do
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += u;
        }
        if (lane == 31) sums[warp] = t;
        __syncthreads();
        for (int w = 0; w < 4; ++w)
            if (w < warp) t += sums[w];
        if (tid < kPagedConsumers && z < p.Z) before[z + 1] = carry + t;
        carry += sums[0] + sums[1] + sums[2] + sums[3];
        __syncthreads();
    }
    if (tid == 0) before[0] = 0;
    __syncthreads();
    const int prefix = paged_prefix(p);
    const PagedPlan a = paged_plan(p, prefix);
    const int64_t total = a.own_first + static_cast<int64_t>(carry) * a.own_rt;
    const int64_t groups = min(static_cast<int64_t>(p.groups), total);   // each has at least one tile
    const int group = blockIdx.x / p.heads_wide, head0 = blockIdx.x % p.heads_wide;
    if (group >= groups) {
        grid_wait();
        return;
    }
    // this block's range, the same for each of its heads
    const int64_t t0 = total * group / groups;
    const int range = static_cast<int>(total * (group + 1) / groups - t0);
    const int count = range * ((p.Hk - 1 - head0) / p.heads_wide + 1);
    const PagedCursor start = paged_locate(a, p.Z, before, head0, t0);
    PagedCursor now = start;
    // tile `done` of the block's; the caller knows that there is one
    auto advance = [&](int done) {
        if (done % range != 0) {
            paged_next(a, before, now);
        } else {
            const int kvh = now.kvh + p.heads_wide;
            now = start;
            now.kvh = kvh;
        }
    };
    auto keys_of = [&](const PagedCursor &c) { return c.z < 0 ? prefix : paged_lengths(p, c.z).x; };
    const WaitCtx wctx{abort_flag, p.status, p.timeout_ns};

    if (warp == 4) {
        // ------------------------------------------------------------ producer
        const int box = min(1 << p.page_shift, kPagedTile);
        int page[kPagedTile / 16];
        int keys = 0, issued = 0;
        const int *table = nullptr;
        for (int t = 0; t < count; ++t) {
            if (t % range == 0 || now.tile == 0) {
                keys = keys_of(now);
                table = now.z < 0 ? p.prefix_table : p.page_table + static_cast<size_t>(now.z) * p.max_pages;
                // the query rows that the consumers will want for this item, a line per lane
                const int rows = now.z < 0 ? a.prefix_rows : a.own_rows;
                for (int e = lane; e < rows * Lay::NSUB; e += 32) {
                    const int64_t r = static_cast<int64_t>(now.rt) * rows + e / Lay::NSUB;
                    const int64_t tok = r / p.group + (now.z < 0 ? 0 : static_cast<int64_t>(now.z) * p.L);
                    if (tok < static_cast<int64_t>(p.Z) * p.L)
                        asm volatile("prefetch.global.L1 [%0];" ::"l"(
                            p.q + (static_cast<size_t>(tok) * p.H + now.kvh * p.group + r % p.group) * D +
                            64 * (e % Lay::NSUB)));
                }
            }
            if (lane == 0) paged_numbers<kPagedTile>(p, table, now.tile, keys, box, page);
            const int s = t % S;
            if (t >= S && !__all_sync(0xffffffffu, mbar_wait(&empty[s], ((t / S) - 1) & 1, wctx))) break;
            if (lane == 0) {
                uint8_t *st = smem + s * 2 * Lay::kOperand;
                mbar_arrive_expect_tx(&full[s], 2 * Lay::kOperand);
                paged_boxes<kPagedTile, Lay::NSUB>(p, &tmK, &full[s], st, now.tile, now.kvh, box, page);
                paged_boxes<kPagedTile, Lay::NSUB>(p, &tmV, &full[s], st + Lay::kOperand, now.tile, now.kvh, box, page);
            }
            __syncwarp();
            issued = t + 1;
            if (issued < count) advance(issued);
        }
        // every issued load must land before the block's shared memory is released
        for (int t = (issued > S ? issued - S : 0); t < issued; ++t)
            mbar_wait_drain(&full[t % S], (t / S) & 1, p.timeout_ns);
        grid_wait();
        return;
    }

    // ---------------------------------------------------------------- consumers
    // The tiles of one item, from `now` on; leaves `now` at the next item.  A wait
    // that gave up does not change the flow: all four warps meet the same
    // barriers, and the results of an aborted call are not used.
    int t = 0;
    auto run = [&]<int WM>() {
        PagedItem<D, SCORE, WM> it;
        const PagedCursor c = now;
        const int keys = keys_of(c);
        if (tid == 0 && c.tile == 0) p.groups_of[c.kvh * p.items + c.item].x = group;
        it.begin(p, c, prefix);
        for (;;) {
            const int s = t % S;
            uint8_t *st = smem + s * 2 * Lay::kOperand;
            mbar_wait(&full[s], (t / S) & 1, wctx);
            __syncwarp();
            const int valid = keys - now.tile * kPagedTile;
            if (valid < kPagedTile) {
                // rows behind the last key may hold anything: as values they are zeroed, as
                // keys their scores are never used
                for (int e = valid * 8 + tid; e < kPagedTile * 8; e += kPagedConsumers)
#pragma unroll
                    for (int u = 0; u < Lay::NSUB; ++u)
                        reinterpret_cast<uint4 *>(st + Lay::kOperand + u * Lay::kAtom)[e] = make_uint4(0u, 0u, 0u, 0u);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before the slot's next TMA writes
                sigma_warps_sync(kPagedConsumers);
            }
            it.tile(smem_u32(st), smem_u32(st + Lay::kOperand), now.tile * kPagedTile);
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
            if (tid == 0 && now.tile == now.tiles - 1) p.groups_of[c.kvh * p.items + c.item].y = group;
            if (++t >= count) break;
            advance(t);
            if (now.item != c.item || now.kvh != c.kvh) break;
        }
        it.end(p.part + (static_cast<size_t>(c.kvh) * (p.groups + p.items) + group + c.item) * kPagedPartRows * D);
    };
    while (t < count) {
        const int w = now.z < 0 ? p.prefix_warps : p.own_warps;
        if (w == 1) run.template operator()<1>();
        else if (w == 2) run.template operator()<2>();
        else run.template operator()<4>();
    }
    // the join waits for this kernel alone: it has to end after the prefix kernel
    grid_wait();
}

// ============================================================================
// The prefix against many rows: the pair-of-tiles forward (span_fwd_sm100.cuh)
// on gathered rows and paged keys.  Row r of row tile i is query head r % group
// of token i * tile_tokens + r / group: a TMA box of (64 entries, group heads,
// one key head, tile_tokens tokens) brings a tile's rows in that order.  Grid
// (splits, pairs, key heads); block s takes the prefix's key tiles
// [s T / S, (s + 1) T / S) and writes its rows' fp32 sums.
// ============================================================================
template <int D, int MODE, int SCORE>
__global__ void __launch_bounds__(kFwdThreads, 1)
    paged_prefix_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PagedParams p) {
    constexpr int KS = FwdStages<D>::K, VS = FwdStages<D>::V;
    using Lay = FwdLayout<D, KS, VS>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_1k(smem_raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Lay::OFF_BAR);
    uint64_t *q_full = bars;
    uint64_t *k_full = bars + 1;
    uint64_t *k_empty = k_full + KS;
    uint64_t *v_full = k_empty + KS;
    uint64_t *v_empty = v_full + VS;
    uint64_t *s_full = v_empty + VS;
    uint64_t *p_full = s_full + 2;
    uint64_t *drain = p_full + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Lay::OFF_TMEM);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + Lay::OFF_ABORT);

    const int warp = warp_id(), lane = lane_id();
    const int split = blockIdx.x, pair = blockIdx.y, kvh = blockIdx.z;
    grid_release();     // the tile kernel reads nothing of this one's
    const int prefix = paged_prefix(p);
    const int T = (prefix + 127) / 128, S = min(p.splits, T);
    const int J0 = split < S ? static_cast<int>(static_cast<int64_t>(T) * split / S) : 0;
    const int steps = split < S ? static_cast<int>(static_cast<int64_t>(T) * (split + 1) / S) - J0 : 0;
    const bool ragged = (prefix & 127) != 0 && J0 + steps == T;
    const int64_t tokens = static_cast<int64_t>(p.Z) * p.L;
    const int64_t tok0 = static_cast<int64_t>(pair) * 2 * p.tile_tokens;
    const int ntiles = tok0 + p.tile_tokens < tokens ? 2 : 1;
    const int box = min(1 << p.page_shift, 128);
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
        for (int t = 0; t < 2; ++t) {
            mbar_init(&s_full[t], 1);
            mbar_init(&p_full[t], 256);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tmQ);
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, Lay::TMEM_COLS);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtx wctx{abort_flag, p.status, p.timeout_ns};
    if (steps == 0) {
        // more splits than tiles (the prefix's length was not needed before this point, so
        // that its load overlaps the set-up)
        if (warp == 1) tmem_dealloc(tmem, Lay::TMEM_COLS);
        return;
    }

    if (warp == 0) {
        if (lane == 0) {
            const int rows = p.tile_tokens * p.group;
            mbar_arrive_expect_tx(q_full, ntiles * Lay::NSUB * rows * 128);
            for (int t = 0; t < ntiles; ++t)
                for (int s = 0; s < Lay::NSUB; ++s)
                    tma_load_4d(&tmQ, q_full, smem + Lay::OFF_Q + t * Lay::TILE_BYTES + s * Lay::SUB_BYTES, 64 * s, 0,
                                kvh, static_cast<int>(tok0) + t * p.tile_tokens);
            int issued = 0, page[8];
            for (int r = 0; r < steps; ++r) {
                const int sk = r % KS;
                paged_numbers<128>(p, p.prefix_table, J0 + r, prefix, box, page);
                if (r >= KS && !mbar_wait(&k_empty[sk], ((r / KS) - 1) & 1, wctx)) break;
                mbar_arrive_expect_tx(&k_full[sk], Lay::TILE_BYTES);
                paged_boxes<128, Lay::NSUB>(p, &tmK, &k_full[sk], smem + Lay::OFF_K + sk * Lay::TILE_BYTES, J0 + r, kvh,
                                            box, page);
                issued = r + 1;
            }
            mbar_wait_drain(q_full, 0, p.timeout_ns);
            for (int r = (issued > KS ? issued - KS : 0); r < issued; ++r)
                mbar_wait_drain(&k_full[r % KS], (r / KS) & 1, p.timeout_ns);
        }
    } else if (warp == 2) {
        if (lane == 0) {
            int issued = 0, page[8];
            for (int r = 0; r < steps; ++r) {
                const int sv = r % VS;
                paged_numbers<128>(p, p.prefix_table, J0 + r, prefix, box, page);
                if (r >= VS && !mbar_wait(&v_empty[sv], ((r / VS) - 1) & 1, wctx)) break;
                mbar_arrive_expect_tx(&v_full[sv], Lay::TILE_BYTES);
                paged_boxes<128, Lay::NSUB>(p, &tmV, &v_full[sv], smem + Lay::OFF_V + sv * Lay::TILE_BYTES, J0 + r, kvh,
                                            box, page);
                issued = r + 1;
            }
            for (int r = (issued > VS ? issued - VS : 0); r < issued; ++r)
                mbar_wait_drain(&v_full[r % VS], (r / VS) & 1, p.timeout_ns);
        }
    } else if (warp == 1) {
        auto wt = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, wctx));
        };
        const uint32_t idesc_s = idesc_bf16_f32(128, 128, false, false);
        const uint32_t idesc_o = idesc_bf16_f32(128, D, false, true);
        const uint32_t sQ = smem_u32(smem + Lay::OFF_Q);
        const uint32_t sK = smem_u32(smem + Lay::OFF_K);
        const uint32_t sV = smem_u32(smem + Lay::OFF_V);
        constexpr uint32_t kDescHi = desc_hi(1024);
        auto issue_s = [&](int t, uint32_t kbase) {
            const uint32_t q_lo = desc_lo(sQ + t * Lay::TILE_BYTES, 16), k_lo = desc_lo(kbase, 16);
            const uint32_t d_tmem = tmem + (t ? Lay::COL_S1 : Lay::COL_S0);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t koff = ((kk >> 2) * Lay::SUB_BYTES + (kk & 3) * 32) >> 4;
                mma_ss_lhw(d_tmem, q_lo + koff, k_lo + koff, kDescHi, idesc_s, kk > 0 ? 1u : 0u);
            }
            mma_commit_w(&s_full[t]);
        };
        auto issue_pv = [&](int t, uint32_t vbase, bool first) {
            const uint32_t d_tmem = tmem + (t ? Lay::COL_O1 : Lay::COL_O0);
            const uint32_t a_tmem = tmem + (t ? Lay::COL_S1 : Lay::COL_S0);
            const uint32_t v_lo = desc_lo(vbase, Lay::SUB_BYTES);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                mma_ts_lhw(d_tmem, a_tmem + kk * 8 + (kk >= 4 ? 32 : 0), v_lo + kk * ((16 * 128) >> 4), kDescHi,
                           idesc_o, (!first || kk > 0) ? 1u : 0u);
        };
        // order per key tile as in span_fwd_kernel
        bool ok = wt(q_full, 0) && wt(&k_full[0], 0);
        if (ok) {
            tc_fence_after();
            for (int t = 0; t < ntiles; ++t) issue_s(t, sK);
            mma_commit_w(&k_empty[0]);
        }
        for (int r = 0; ok && r < steps; ++r) {
            const int sv = r % VS, sk = (r + 1) % KS;
            const bool more = r + 1 < steps;
            if (!(ok = wt(&v_full[sv], (r / VS) & 1))) break;
            if (!more && ragged)
                zero_tile_rows<Lay::NSUB>(smem + Lay::OFF_V + sv * Lay::TILE_BYTES, prefix & 127);
            for (int t = 0; t < ntiles; ++t) {
                if (!(ok = wt(&p_full[t], r & 1))) break;
                tc_fence_after();
                issue_pv(t, sV + sv * Lay::TILE_BYTES, r == 0);
                if (t == ntiles - 1) mma_commit_w(&v_empty[sv]);
                if (more) {
                    if (t == 0 && !(ok = wt(&k_full[sk], ((r + 1) / KS) & 1))) break;
                    tc_fence_after();
                    issue_s(t, sK + sk * Lay::TILE_BYTES);
                    if (t == ntiles - 1) mma_commit_w(&k_empty[sk]);
                }
            }
        }
        mma_commit_w(drain);
        mbar_wait_drain(drain, 0, p.timeout_ns);
        __syncwarp();
    } else if (warp >= 4) {
        const int g = (warp - 4) >> 2;
        const int t = g >> 1, c = g & 1;
        const int quarter = warp & 3;
        const uint32_t lane_bits = static_cast<uint32_t>(quarter * 32) << 16;
        const int row = quarter * 32 + lane;
        if (t < ntiles) {
            // the token and head of this row
            const int64_t tok = tok0 + static_cast<int64_t>(t) * p.tile_tokens + row / p.group;
            const int h = kvh * p.group + row % p.group;
            ScoreCoef cf = {0.0f, -64.0f};    // of rows that are not there: sigma of almost nothing
            bool live = row < p.tile_tokens * p.group && tok < tokens;
            int pos = 0;
            if (live) {
                const int z = static_cast<int>(tok / p.L), l = static_cast<int>(tok % p.L);
                const int2 n = paged_lengths(p, z);
                live = l < n.y;
                pos = prefix + n.x - n.y + l;
                cf = make_score<SCORE>(p.alpha, bias_of(p.bias_z, p.bias, z), p.cap,
                                       SCORE & kScoreSlope ? p.slopes[h] : 0.0f);
            }
            // the same choice in the whole warp
            ScorePause pause = score_pause(cf);
            pause.tail = __all_sync(0xffffffffu, !live || pause.tail == 0) ? 0 : kNever;
            pause.poly = __all_sync(0xffffffffu, !live || pause.poly == 0) ? 0 : kNever;
            bool ok = true;
            const uint32_t tS = tmem + lane_bits + (t ? Lay::COL_S1 : Lay::COL_S0) + 64 * c;
            for (int r = 0; r < steps; ++r) {
                ok = __all_sync(0xffffffffu, mbar_wait(&s_full[t], r & 1, wctx));
                if (!ok) break;
                tc_fence_after();
                const int key0 = (J0 + r) * 128 + 64 * c;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t x[32], pk[16];
                    tmem_ld32(tS + 32 * u, x);
                    score_chunk<MODE, SCORE, false, true>(x, cf, static_cast<float>(pos - key0 - 32 * u), pk, nullptr, pause,
                                                          prefix - key0 >= 64, live);
                    if (prefix - key0 < 64) keep_bits(pk, bit_range(0, prefix - key0 - 32 * u));
                    tmem_st16(tS + 16 * u, pk);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&p_full[t]);
            }
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(drain, 0, wctx));
            if (ok) {
                tc_fence_after();
                // fp32 rows through shared memory (the rings are idle: every load has landed
                // and every MMA is done), so that whole sectors are written: this warp's 32
                // rows of 64 columns, 16-byte chunks swizzled by row
                constexpr int HALF = D / 2, CH = HALF / 4;
                const uint32_t tO = tmem + lane_bits + (t ? Lay::COL_O1 : Lay::COL_O0) + c * HALF;
                float4 *buf = reinterpret_cast<float4 *>(smem + Lay::OFF_K) + (warp - 4) * 32 * CH;
                const unsigned there = __ballot_sync(0xffffffffu, live);
#pragma unroll
                for (int cc = 0; cc < HALF / 32; ++cc) {
                    uint32_t x[32];
                    tmem_ld32(tO + 32 * cc, x);
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        buf[lane * CH + ((8 * cc + v) ^ (lane & 7))] =
                            make_float4(__uint_as_float(x[4 * v]), __uint_as_float(x[4 * v + 1]),
                                        __uint_as_float(x[4 * v + 2]), __uint_as_float(x[4 * v + 3]));
                }
                __syncwarp();
                float *dst = p.prefix_part +
                             (((static_cast<size_t>(split) * p.Hk + kvh) * p.pairs + pair) * 256 + t * 128 + quarter * 32) * D +
                             c * HALF;
#pragma unroll
                for (int e = lane; e < 32 * CH; e += 32) {
                    const int r = e / CH, ch = e % CH;
                    if ((there >> r) & 1u) *reinterpret_cast<float4 *>(dst + r * D + 4 * ch) = buf[r * CH + (ch ^ (r & 7))];
                }
            }
        }
    }

    __syncwarp();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, Lay::TMEM_COLS);
    }
}

// Adds up the partials of each output row, prefix first, and rounds.  W warps
// share a row, warp w taking every W-th partial, and their sums are added in warp
// order; a block has 8 / W rows.
constexpr int kJoinThreads = 256;
template <int D, int W>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ PagedParams p) {
    constexpr int E = D / 32, R = 8 / W;
    __shared__ float sums[W > 1 ? 8 : 1][W > 1 ? D : 1];
    const unsigned rows = static_cast<unsigned>(p.Z) * p.L * p.H;      // below 2^31
    const bool there = blockIdx.x * R + warp_id() / W < rows;
    const unsigned r = there ? blockIdx.x * R + warp_id() / W : 0u;
    const int lane = lane_id(), w = warp_id() % W;
    const unsigned tok = r / p.H, h = r % p.H, z = tok / p.L, l = tok % p.L;
    const unsigned kvh = h / p.group, g = h % p.group;
    const unsigned own_row = l * p.group + g;
    const unsigned own_rows = 16 * p.own_warps, prefix_rows = 16 * p.prefix_warps;
    const unsigned own_item = p.prefix_rt + z * p.own_rt + own_row / own_rows;
    const int2 n = paged_lengths(p, z);
    const int prefix = paged_prefix(p);
    const bool live = there && static_cast<int>(l) < n.y;
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    int done = 0;     // partials before these
    // `count` partials, `step` floats apart
    auto sum = [&](const float *src, size_t step, int count) {
        int b = (w - done) & (W - 1);
        done += count;
#pragma unroll 8
        for (; b < count; b += W) {
            if constexpr (E == 4) {
                const float4 v = __ldcg(reinterpret_cast<const float4 *>(src + b * step));
                acc[0] += v.x;
                acc[1] += v.y;
                acc[2] += v.z;
                acc[3] += v.w;
            } else {
                const float2 v = __ldcg(reinterpret_cast<const float2 *>(src + b * step));
                acc[0] += v.x;
                acc[1] += v.y;
            }
        }
    };
    // partials of row `row` of an item's `rows`: the warps along the keys lie `rows`
    // rows apart, the groups kPagedPartRows
    auto add = [&](unsigned item, unsigned row, unsigned rows) {
        const int2 b = __ldcg(&p.groups_of[kvh * p.items + item]);
        const size_t slot = static_cast<size_t>(kvh) * (p.groups + p.items) + b.x + item;
        sum(p.part + (slot * kPagedPartRows + row) * D + lane * E,
            static_cast<size_t>(rows) * D, (b.y - b.x + 1) * static_cast<int>(kPagedPartRows / rows));
    };
    grid_wait();
    if (live) {
        if (p.splits > 0) {
            const int T = (prefix + 127) / 128, S = min(p.splits, T);
            const unsigned tile = tok / p.tile_tokens;      // row tile
            const unsigned row = tok % p.tile_tokens * p.group + g;
            sum(p.prefix_part + (static_cast<size_t>(kvh * p.pairs + tile / 2) * 256 + (tile & 1) * 128 + row) * D + lane * E,
                static_cast<size_t>(p.Hk) * p.pairs * 256 * D, S);
        } else if (prefix > 0) {
            const unsigned row = tok * p.group + g;
            add(row / prefix_rows, row % prefix_rows, prefix_rows);
        }
        add(own_item, own_row % own_rows, own_rows);     // a live row has at least its own key
    }
    if constexpr (W > 1) {
        float *mine = sums[warp_id()] + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) mine[e] = acc[e];
        __syncthreads();
        if (w != 0) return;
#pragma unroll
        for (int u = 1; u < W; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += mine[u * D + e];
    }
    if (!there) return;
    __nv_bfloat16 *dst = p.o + static_cast<size_t>(r) * D + lane * E;
    if constexpr (E == 4)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
    else
        *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(acc[0], acc[1]);
}

}  // namespace sigattn
