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
// Work is a list of items, each a run of 64-key tiles:
//   prefix items: (key head, tile of query rows), the rows being those of all
//                 samples' tokens and of all query heads of the key head, so that
//                 the prefix is read once per row tile and not once per sample;
//   own items:    (sample, key head, tile of its query rows).
// The tiles of all items form one sequence that is cut evenly over the grid
// (block b of B <= T takes [b T / B, (b + 1) T / B)), whatever the lengths: a block walks its
// range, keeps kStages tiles in flight with cp.async across item borders, and
// writes one fp32 partial per item it touches.  Walking on either starts a new
// block or a new item, so (block + item) numbers the partials without a table.
// paged_join_kernel adds the partials of each row in that order (the result
// does not depend on scheduling) and rounds once.
//
// Bound: memory.  Every key and value is read once per row tile; a 64-key tile
// at D = 128 is 32 KB, 1.4 kclk of an SM's share of HBM, against 1.0 kclk of
// mma.sync for a full 64-row tile and far less for the few rows of one sample.
#pragma once

#include "cache_append.cuh"
#include "span_score.cuh"

namespace sigattn {

struct PagedParams {
    const __nv_bfloat16 *q, *k_pages, *v_pages;
    __nv_bfloat16 *o;
    const int *page_table, *seqlens_k, *seqlens_q, *prefix_table, *prefix_len;
    int Z, L, H, Hk, group;
    int pages, page_shift, max_pages, prefix_pages;
    float alpha, bias, cap;
    const float *bias_z, *slopes;
    float *part;          // [block + item][rows][D]
    int *before;          // [Z + 1] own tiles of the samples before z, written by block 0
    int prefix_warps, own_warps;   // warps along the rows (1, 2, 4): row tiles of 16 times that
    int part_rows;        // rows of one partial: the larger row tile
    int blocks;           // grid of the tile kernel
    int *status;
};

constexpr int kPagedThreads = 128;
constexpr int kPagedTile = 64;    // keys per tile

template <int D>
struct PagedLayout {
    static constexpr int kStages = D == 128 ? 3 : 4;
    static constexpr int kBlocksPerSm = D == 128 ? 2 : 3;
    static constexpr int kRow = D * 2;                         // bytes of one key
    static constexpr int kOperand = kPagedTile * kRow;         // one K or V tile
    static constexpr int OFF_RED = kStages * 2 * kOperand;     // [16][D] fp32 sum over warps
    static constexpr int OFF_BEFORE = OFF_RED + 16 * D * 4;
    static constexpr int bytes(int Z) { return OFF_BEFORE + (Z + 1) * 4 + 64; }
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
    int prefix_tiles, prefix_rows, prefix_rt, prefix_items;   // tiles of the prefix; rows per tile; row tiles; items
    int own_rows, own_rt;
    int64_t own_first;        // tiles of all prefix items: where own items begin
};
__device__ __forceinline__ PagedPlan paged_plan(const PagedParams &p, int prefix) {
    PagedPlan a;
    a.prefix_tiles = (prefix + kPagedTile - 1) / kPagedTile;
    a.prefix_rows = 16 * p.prefix_warps;
    a.prefix_rt = static_cast<int>((static_cast<int64_t>(p.Z) * p.L * p.group + a.prefix_rows - 1) / a.prefix_rows);
    a.prefix_items = a.prefix_rt * p.Hk;
    a.own_rows = 16 * p.own_warps;
    a.own_rt = (p.L * p.group + a.own_rows - 1) / a.own_rows;
    a.own_first = static_cast<int64_t>(a.prefix_tiles) * a.prefix_items;
    return a;
}

// A place in the tile sequence.
struct PagedCursor {
    int item;             // number of the item
    int z;                // sample of an own item, -1 for a prefix item
    int kvh, rt, tile, tiles;
};

__device__ __forceinline__ PagedCursor paged_locate(const PagedParams &p, const PagedPlan &a, const int *before,
                                                    int64_t t) {
    PagedCursor c;
    if (t < a.own_first) {
        c.item = static_cast<int>(t / a.prefix_tiles);
        c.z = -1;
        c.kvh = c.item / a.prefix_rt;
        c.rt = c.item % a.prefix_rt;
        c.tile = static_cast<int>(t % a.prefix_tiles);
        c.tiles = a.prefix_tiles;
        return c;
    }
    const int per = p.Hk * a.own_rt;    // items of a sample
    const int64_t u = t - a.own_first;
    const int at = static_cast<int>(u / per);
    int lo = 0, hi = p.Z - 1;           // the last sample with before[z] <= at
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (before[mid] <= at) lo = mid;
        else hi = mid - 1;
    }
    c.z = lo;
    c.tiles = before[lo + 1] - before[lo];
    const int64_t in = u - static_cast<int64_t>(before[lo]) * per;
    const int i = static_cast<int>(in / c.tiles);
    c.tile = static_cast<int>(in % c.tiles);
    c.kvh = i / a.own_rt;
    c.rt = i % a.own_rt;
    c.item = a.prefix_items + lo * per + i;
    return c;
}

// The next tile; the caller knows that there is one.
__device__ __forceinline__ void paged_next(const PagedParams &p, const PagedPlan &a, const int *before,
                                           PagedCursor &c) {
    if (++c.tile < c.tiles) return;
    c.tile = 0;
    ++c.item;
    if (++c.rt < (c.z < 0 ? a.prefix_rt : a.own_rt)) return;
    c.rt = 0;
    if (++c.kvh < p.Hk) return;
    c.kvh = 0;
    do {
        ++c.z;            // from -1: the first sample
        c.tiles = c.z < p.Z ? before[c.z + 1] - before[c.z] : 1;
        c.item = a.prefix_items + c.z * p.Hk * a.own_rt;
    } while (c.tiles == 0);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
    // a row that does not exist reads nothing and arrives as zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
    float pos[2];                // place of the query among the item's keys
    int limit[2];                // keys below it are seen
};

// Everything a block does with the tiles of one item kind: WM warps along the
// rows (16 each), 4 / WM along the keys of a tile.
template <int D, int SCORE, int WM>
struct PagedItem {
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
            rows.pos[i] = 0.0f;
            rows.limit[i] = 0;
            cf[i] = ScoreCoef{0.0f, 0.0f, 0.0f, 0.0f};
            if (!in) continue;
            const int z = static_cast<int>(tok / p.L), l = static_cast<int>(tok % p.L);
            const int2 n = paged_lengths(p, z);
            if (l >= n.y) continue;
            const int at = n.x - n.y + l;     // own place
            rows.q[i] = p.q + (static_cast<size_t>(tok) * p.H + h) * D;
            rows.pos[i] = static_cast<float>(c.z < 0 ? prefix + at : at);
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
#pragma unroll
        for (int g = 0; g < KW / 16; ++g) {
            const int k16 = wk * KW + 16 * g;     // first of 16 keys
            float s[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
            {
                // lanes 0-7: keys 0-7 low half, 8-15: keys 0-7 high half, then keys 8-15
                const int row = k16 + (lane & 7) + ((lane >> 4) << 3);
                const uint32_t base = sK + row * (D * 2);
#pragma unroll
                for (int kk = 0; kk < NK; ++kk) {
                    uint32_t b[4];
                    ldmatrix4(base + (((2 * kk + ((lane >> 3) & 1)) ^ (row & 7)) << 4), b);
                    mma16816(s[0], qf[kk], b[0], b[1]);
                    mma16816(s[1], qf[kk], b[2], b[3]);
                }
            }
            uint32_t a[4];
#pragma unroll
            for (int n8 = 0; n8 < 2; ++n8)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int key = key0 + k16 + 8 * n8 + 2 * (lane & 3);
                    float2 w = score_p2<SCORE>(s[n8][2 * i], s[n8][2 * i + 1], cf[i],
                                                     rows.pos[i] - static_cast<float>(key));
                    w.x = key < rows.limit[i] ? w.x : 0.0f;
                    w.y = key + 1 < rows.limit[i] ? w.y : 0.0f;
                    a[2 * n8 + i] = pack_bf16x2(w.x, w.y);
                }
            {
                // lanes 0-7: keys 0-7, 8-15: keys 8-15, then the next 8 columns
                const int row = k16 + (lane & 15);
                const uint32_t base = sV + row * (D * 2);
#pragma unroll
                for (int d = 0; d < D / 16; ++d) {
                    uint32_t b[4];
                    ldmatrix4_trans(base + (((2 * d + (lane >> 4)) ^ (row & 7)) << 4), b);
                    mma16816(acc[2 * d], a, b[0], b[1]);
                    mma16816(acc[2 * d + 1], a, b[2], b[3]);
                }
            }
        }
    }

    // Adds the warps along the keys up, in warp order (16 rows at a time), and
    // writes the rows.
    __device__ __forceinline__ void end(float *red, float *dst) {
        const int lane = lane_id(), wm = warp_id() % WM, wk = warp_id() / WM;
        const int r0 = lane / 4, c0 = 2 * (lane & 3);
#pragma unroll
        for (int m = 0; m < WM; ++m) {
#pragma unroll
            for (int w = 1; w < WK; ++w) {
                if (wm == m && wk == w) {
#pragma unroll
                    for (int d = 0; d < D / 8; ++d)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float2 *at = reinterpret_cast<float2 *>(red + (r0 + 8 * i) * D + 8 * d + c0);
                            const float2 old = w > 1 ? *at : make_float2(0.0f, 0.0f);
                            *at = make_float2(old.x + acc[d][2 * i], old.y + acc[d][2 * i + 1]);
                        }
                }
                __syncthreads();
            }
            if (wm == m && wk == 0) {
#pragma unroll
                for (int d = 0; d < D / 8; ++d)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (rows.q[i] == nullptr) continue;
                        const int at = (r0 + 8 * i) * D + 8 * d + c0;
                        float2 v = make_float2(acc[d][2 * i], acc[d][2 * i + 1]);
                        if constexpr (WK > 1) {
                            const float2 o = *reinterpret_cast<const float2 *>(red + at);
                            v.x += o.x;
                            v.y += o.y;
                        }
                        *reinterpret_cast<float2 *>(dst + 16 * m * D + at) = v;
                    }
            }
            if (WK > 1 && m + 1 < WM) __syncthreads();
        }
    }
};

// Issues the loads of one tile (K then V) into a stage.  A key that does not
// exist, or whose page number is bad (flagged), arrives as zeros.
template <int D>
__device__ __forceinline__ void paged_load(const PagedParams &p, const PagedCursor &c, int keys, uint32_t stage) {
    constexpr int CH = D / 8;                       // 16-byte chunks of a key
    constexpr int STEP = kPagedThreads / CH;        // keys per pass
    const int *table = c.z < 0 ? p.prefix_table : p.page_table + static_cast<size_t>(c.z) * p.max_pages;
    const int ch = threadIdx.x % CH, r0 = threadIdx.x / CH;
    const int mask = (1 << p.page_shift) - 1;
    // pages hold at least 16 keys: four numbers cover a tile
    int64_t base[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int key = c.tile * kPagedTile + 16 * i;
        int page = -1;
        if (key < keys) {
            page = __ldg(table + (key >> p.page_shift));
            if (page < 0 || page >= p.pages) {
                if (threadIdx.x == 0) record_status(p.status, kStatusPageRange);
                page = -1;
            }
        }
        base[i] = page < 0 ? -1
                           : (((static_cast<int64_t>(page) << p.page_shift) + (key & mask)) * p.Hk + c.kvh) * D;
    }
#pragma unroll
    for (int i = 0; i < kPagedTile / STEP; ++i) {
        const int r = r0 + i * STEP;
        const int64_t b = base[(i * STEP) / 16];   // STEP divides 16
        const bool ok = b >= 0 && c.tile * kPagedTile + r < keys;
        const size_t off = ok ? static_cast<size_t>(b) + static_cast<size_t>(r & 15) * p.Hk * D + 8 * ch : 0;
        const uint32_t dst = stage + r * (D * 2) + ((ch ^ (r & 7)) << 4);
        cp_async16(dst, p.k_pages + off, ok);
        cp_async16(dst + kPagedTile * D * 2, p.v_pages + off, ok);
    }
}

template <int D, int SCORE>
__global__ void __launch_bounds__(kPagedThreads, PagedLayout<D>::kBlocksPerSm)
    paged_tiles_kernel(const PagedParams p) {
    using Lay = PagedLayout<D>;
    constexpr int S = Lay::kStages;
    extern __shared__ __align__(128) uint8_t smem[];
    float *red = reinterpret_cast<float *>(smem + Lay::OFF_RED);
    int *before = reinterpret_cast<int *>(smem + Lay::OFF_BEFORE);
    __shared__ int sums[4];
    const int tid = threadIdx.x;

    // own tiles of the samples before each: one scan over the batch
    int carry = 0;
    for (int z0 = 0; z0 < p.Z; z0 += kPagedThreads) {
        const int z = z0 + tid;
        int t = z < p.Z ? (paged_lengths(p, z).x + kPagedTile - 1) / kPagedTile : 0;
        if (z < p.Z && paged_lengths(p, z).y == 0) t = 0;       // no query: nothing to do
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, t, o);
            if (lane_id() >= o) t += u;
        }
        if (lane_id() == 31) sums[warp_id()] = t;
        __syncthreads();
        for (int w = 0; w < 4; ++w) {
            if (w < warp_id()) t += sums[w];
        }
        if (z < p.Z) before[z + 1] = carry + t;
        carry += sums[0] + sums[1] + sums[2] + sums[3];
        __syncthreads();
    }
    if (tid == 0) before[0] = 0;
    __syncthreads();
    if (blockIdx.x == 0)
        for (int z = tid; z <= p.Z; z += kPagedThreads) p.before[z] = before[z];

    const int prefix = paged_prefix(p);
    const PagedPlan a = paged_plan(p, prefix);
    const int64_t total = a.own_first + static_cast<int64_t>(carry) * p.Hk * a.own_rt;
    const int64_t blocks = min(static_cast<int64_t>(gridDim.x), total);   // each has at least one tile
    if (blockIdx.x >= blocks) return;
    const int64_t t0 = total * blockIdx.x / blocks, t1 = total * (blockIdx.x + 1) / blocks;
    PagedCursor now = paged_locate(p, a, before, t0), ahead = now;
    const uint32_t ring = smem_u32(smem);
    auto keys_of = [&](const PagedCursor &c) { return c.z < 0 ? prefix : paged_lengths(p, c.z).x; };
    int64_t issued = t0;
    auto issue = [&]() {
        if (issued < t1) {
            paged_load<D>(p, ahead, keys_of(ahead), ring + static_cast<uint32_t>((issued - t0) % S) * 2 * Lay::kOperand);
            if (++issued < t1) paged_next(p, a, before, ahead);
        }
        cp_async_commit();    // a group per step, empty at the end, so that the wait counts right
    };
#pragma unroll
    for (int s = 0; s < S - 1; ++s) issue();

    // The tiles of one item, from `now` on; leaves `now` at the next item.
    int64_t t = t0;
    auto run = [&]<int WM>() {
        PagedItem<D, SCORE, WM> it;
        const PagedCursor c = now;
        it.begin(p, c, prefix);
        for (;;) {
            cp_async_wait<S - 2>();
            __syncthreads();      // tile t is here, and tile t - 1's slot is free
            issue();
            const uint32_t st = ring + static_cast<uint32_t>((t - t0) % S) * 2 * Lay::kOperand;
            it.tile(st, st + Lay::kOperand, now.tile * kPagedTile);
            ++t;
            if (t >= t1) break;
            paged_next(p, a, before, now);
            if (now.item != c.item) break;
        }
        it.end(red, p.part + (static_cast<size_t>(blockIdx.x) + c.item) * p.part_rows * D);
    };
    while (t < t1) {
        const int w = now.z < 0 ? p.prefix_warps : p.own_warps;
        if (w == 1) run.template operator()<1>();
        else if (w == 2) run.template operator()<2>();
        else run.template operator()<4>();
    }
}

// Adds up the partials of each output row, prefix items first, in block order.
// One warp per row.
template <int D>
__global__ void __launch_bounds__(256) paged_join_kernel(const PagedParams p) {
    constexpr int E = D / 32;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + warp_id();
    if (r >= static_cast<int64_t>(p.Z) * p.L * p.H) return;
    const int lane = lane_id();
    const int h = static_cast<int>(r % p.H);
    const int64_t tok = r / p.H;
    const int z = static_cast<int>(tok / p.L), l = static_cast<int>(tok % p.L);
    const int kvh = h / p.group, g = h % p.group;
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    if (l < paged_lengths(p, z).y) {
        const int prefix = paged_prefix(p);
        const PagedPlan a = paged_plan(p, prefix);
        const int64_t per = static_cast<int64_t>(p.Hk) * a.own_rt;
        const int64_t total = a.own_first + p.before[p.Z] * per;
        const int64_t blocks = min(static_cast<int64_t>(p.blocks), total);
        // partials of the item with tiles [first, first + tiles), row `row` of it
        auto add = [&](int64_t first, int tiles, int64_t item, int row) {
            if (tiles == 0) return;
            const int64_t b0 = ((first + 1) * blocks - 1) / total;
            const int64_t b1 = ((first + tiles) * blocks - 1) / total;
            const float *src = p.part + ((b0 + item) * p.part_rows + row) * D + lane * E;
            const size_t step = static_cast<size_t>(p.part_rows) * D;
#pragma unroll 4
            for (int64_t b = b0; b <= b1; ++b, src += step) {
                if constexpr (E == 4) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(src));
                    acc[0] += v.x;
                    acc[1] += v.y;
                    acc[2] += v.z;
                    acc[3] += v.w;
                } else {
                    const float2 v = __ldcg(reinterpret_cast<const float2 *>(src));
                    acc[0] += v.x;
                    acc[1] += v.y;
                }
            }
        };
        {
            const int64_t row = tok * p.group + g;
            const int64_t item = static_cast<int64_t>(kvh) * a.prefix_rt + row / a.prefix_rows;
            add(item * a.prefix_tiles, a.prefix_tiles, item, static_cast<int>(row % a.prefix_rows));
        }
        {
            const int row = l * p.group + g;
            const int i = kvh * a.own_rt + row / a.own_rows;
            const int tiles = p.before[z + 1] - p.before[z];
            add(a.own_first + p.before[z] * per + static_cast<int64_t>(i) * tiles, tiles,
                a.prefix_items + z * per + i, row % a.own_rows);
        }
    }
    __nv_bfloat16 *dst = p.o + r * D + lane * E;
    if constexpr (E == 4)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
    else
        *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(acc[0], acc[1]);
}

}  // namespace sigattn
