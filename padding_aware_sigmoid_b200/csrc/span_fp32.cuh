// fp32 accuracy path of the masked attention (span_score.cuh): fp32 arithmetic
// throughout, library expf and tanhf.  The four rows of a block share chunks of 32
// rows of the other side in shared memory; lanes are those rows while scores are
// formed, so that a weight is computed once and no reduction is needed, and
// entries of the output row while it is accumulated.  Groups of four warps, one
// per row, take every G-th chunk on their own, and their sums are added in order
// at the end.  Bound by latency and shared-memory reads: meant for accuracy
// checks at small sizes.
#pragma once

#include "fp32_simt.cuh"
#include "span_score.cuh"

namespace sigattn {

struct SpanF32Params {
    const float *q, *k, *v, *dout;
    float *o, *dq, *dk, *dv;
    SpanSource src;
    int Z, H, Hk, group;
    float alpha, bias, cap;
    const float *bias_z, *slopes;
};

// P and dP/d(alpha s) of one score; cap 0: no cap.
__device__ __forceinline__ void span_exact(float y, float cap, float add, float &p, float &g) {
    float f = 1.0f;
    if (cap > 0.0f) {
        // 1 - tanh^2 as 4 e / (1 + e)^2, e = exp(-2 |y / cap|): nothing cancels
        const float u = y / cap, e = expf(-2.0f * fabsf(u)), r = 1.0f / (1.0f + e);
        y = cap * tanhf(u);
        f = 4.0f * e * r * r;
    }
    exact_sigma(y + add, p, g);
    g *= f;
}

// Rows of a block, one warp of each group, and rows of a chunk, which a group
// shares in shared memory, kStride floats apart (16-byte reads of 32 rows then
// meet no bank twice).
constexpr int kF32Rows = 4, kF32Chunk = 32;
template <int D, int G>
struct SpanF32Smem {
    static constexpr int kStride = D + 4;
    static constexpr int kThreads = 32 * kF32Rows * G;
    struct Chunk {
        float a[kF32Chunk][kStride], b[kF32Chunk][kStride];   // K and V, or Q and dO
    };
    Chunk chunk[G];
    float x[kF32Rows][D], y[kF32Rows][D];                      // the block's own rows of the other side
};

// Barrier of the four warps of a group.
__device__ __forceinline__ void span_f32_meet(int group) {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(32 * kF32Rows) : "memory");
}

// Rows r0 ... r0 + kF32Chunk - 1 below `end` of two tensors (row r at base + r *
// stride) into a chunk; the others as zeros, whatever memory holds there.
template <int D, typename Chunk>
__device__ __forceinline__ void span_f32_chunk(Chunk &sm, const float *a, const float *b, int64_t stride,
                                               int r0, int end) {
    constexpr int V = D / 4;
    for (int e = threadIdx.x % (32 * kF32Rows); e < kF32Chunk * V; e += 32 * kF32Rows) {
        const int r = e / V, c = 4 * (e % V);
        float4 u = make_float4(0.0f, 0.0f, 0.0f, 0.0f), v = u;
        if (r0 + r < end) {
            u = __ldg(reinterpret_cast<const float4 *>(a + (r0 + r) * stride + c));
            v = __ldg(reinterpret_cast<const float4 *>(b + (r0 + r) * stride + c));
        }
        *reinterpret_cast<float4 *>(&sm.a[r][c]) = u;
        *reinterpret_cast<float4 *>(&sm.b[r][c]) = v;
    }
}

template <int D>
__device__ __forceinline__ float span_f32_dot(const float *x, const float *a) {
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < D; e += 4) {
        const float4 u = *reinterpret_cast<const float4 *>(x + e), v = *reinterpret_cast<const float4 *>(a + e);
        s[0] = fmaf(u.x, v.x, s[0]);
        s[1] = fmaf(u.y, v.y, s[1]);
        s[2] = fmaf(u.z, v.z, s[2]);
        s[3] = fmaf(u.w, v.w, s[3]);
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// Forward (DQ false) or dQ (DQ true) of query rows 4 g ... 4 g + 3 of one head.
template <int D, int G, bool DQ>
__device__ __forceinline__ void span_f32_rows(const SpanF32Params &p, SpanF32Smem<D, G> &sm, int64_t block) {
    constexpr int E = D / 32;
    const int lane = lane_id(), warp = warp_id() % kF32Rows, group = G > 1 ? warp_id() / kF32Rows : 0;
    const int L = p.src.L, groups = (L + kF32Rows - 1) / kF32Rows;
    auto &ch = sm.chunk[group];
    const int g = static_cast<int>(block % groups);
    const int h = static_cast<int>((block / groups) % p.H);
    const int z = static_cast<int>(block / (static_cast<int64_t>(groups) * p.H));
    const int i = g * kF32Rows + warp;
    const int n = span_tokens(p.src, z);
    const int2 span = row_span(p.src, z, i, n);
    const float bias = bias_of(p.bias_z, p.bias, z), slope = p.slopes != nullptr ? p.slopes[h] : 0.0f;
    const int64_t krow = static_cast<int64_t>(p.Hk) * D;
    const int64_t kbase = static_cast<int64_t>(z) * L * krow + static_cast<int64_t>(h / p.group) * D;
    const int64_t row = ((static_cast<int64_t>(z) * L + i) * p.H + h) * D;
    int lo = INT_MAX, hi = 0;            // keys that any row of the block sees
#pragma unroll
    for (int w = 0; w < kF32Rows; ++w) {
        const int2 s = row_span(p.src, z, g * kF32Rows + w, n);
        if (s.x < s.y) {
            lo = min(lo, s.x);
            hi = max(hi, s.y);
        }
    }
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        acc[e] = 0.0f;
        if (group == 0 && i < L) {
            sm.x[warp][lane + 32 * e] = p.q[row + lane + 32 * e];
            if (DQ) sm.y[warp][lane + 32 * e] = p.dout[row + lane + 32 * e];
        }
    }
    if constexpr (G > 1) __syncthreads();
    for (int64_t at = static_cast<int64_t>(lo) + kF32Chunk * group; at < hi; at += kF32Chunk * G) {
        const int j0 = static_cast<int>(at);
        span_f32_meet(group);
        span_f32_chunk<D>(ch, p.k + kbase, p.v + kbase, krow, j0, hi);
        span_f32_meet(group);
        const int j = j0 + lane;
        float w = 0.0f;
        if (j >= span.x && j < span.y) {
            float pr, gr;
            span_exact(p.alpha * span_f32_dot<D>(sm.x[warp], ch.a[lane]), p.cap,
                       fmaf(-slope, fabsf(static_cast<float>(i - j)), bias), pr, gr);
            w = DQ ? gr * span_f32_dot<D>(sm.y[warp], ch.b[lane]) : pr;
        }
        if (__any_sync(0xffffffffu, w != 0.0f)) {
#pragma unroll
            for (int u = 0; u < kF32Chunk; ++u) {
                const float wu = __shfl_sync(0xffffffffu, w, u);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = fmaf(wu, (DQ ? ch.a : ch.b)[u][lane + 32 * e], acc[e]);
            }
        }
    }
    if constexpr (G > 1) {
        span_f32_meet(group);      // the chunk's place takes the sums
#pragma unroll
        for (int e = 0; e < E; ++e) ch.a[warp][lane + 32 * e] = acc[e];
        __syncthreads();
    }
    if (group == 0 && i < L) {
#pragma unroll
        for (int u = 1; u < G; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += sm.chunk[u].a[warp][lane + 32 * e];
        float *out = (DQ ? p.dq : p.o) + row + lane;
#pragma unroll
        for (int e = 0; e < E; ++e) out[32 * e] = DQ ? p.alpha * acc[e] : acc[e];
    }
}

// dK and dV of keys 4 g ... 4 g + 3 of one key head, over the queries of its heads.
template <int D, int G>
__device__ __forceinline__ void span_f32_keys(const SpanF32Params &p, SpanF32Smem<D, G> &sm, int64_t block) {
    constexpr int E = D / 32;
    const int lane = lane_id(), warp = warp_id() % kF32Rows, group = G > 1 ? warp_id() / kF32Rows : 0;
    const int L = p.src.L, groups = (L + kF32Rows - 1) / kF32Rows;
    auto &ch = sm.chunk[group];
    const int g = static_cast<int>(block % groups);
    const int kvh = static_cast<int>((block / groups) % p.Hk);
    const int z = static_cast<int>(block / (static_cast<int64_t>(groups) * p.Hk));
    const int j = g * kF32Rows + warp;
    const int n = span_tokens(p.src, z);
    const float bias = bias_of(p.bias_z, p.bias, z);
    const int64_t qrow = static_cast<int64_t>(p.H) * D;
    const int64_t row = ((static_cast<int64_t>(z) * L + j) * p.Hk + kvh) * D;
    float ak[E], av[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        ak[e] = av[e] = 0.0f;
        if (group == 0 && j < L) {
            sm.x[warp][lane + 32 * e] = p.k[row + lane + 32 * e];
            sm.y[warp][lane + 32 * e] = p.v[row + lane + 32 * e];
        }
    }
    if constexpr (G > 1) __syncthreads();
    for (int64_t at = kF32Chunk * group; at < n; at += kF32Chunk * G) {
        const int i0 = static_cast<int>(at);
        // does any row of the chunk see a key of the block?
        const int i = i0 + lane;
        const int2 sp = row_span(p.src, z, i, n);
        if (!__any_sync(0xffffffffu, sp.x < (g + 1) * kF32Rows && sp.y > g * kF32Rows)) continue;   // alike in the group
        const bool sees = j >= sp.x && j < sp.y;
        for (int h = kvh * p.group; h < (kvh + 1) * p.group; ++h) {
            const int64_t base = static_cast<int64_t>(z) * L * qrow + static_cast<int64_t>(h) * D;
            span_f32_meet(group);
            span_f32_chunk<D>(ch, p.q + base, p.dout + base, qrow, i0, n);
            span_f32_meet(group);
            float pr = 0.0f, gr = 0.0f;
            if (sees) {
                span_exact(p.alpha * span_f32_dot<D>(sm.x[warp], ch.a[lane]), p.cap,
                           fmaf(p.slopes != nullptr ? -p.slopes[h] : 0.0f, fabsf(static_cast<float>(i - j)), bias), pr, gr);
                gr *= span_f32_dot<D>(sm.y[warp], ch.b[lane]);
            }
            if (__any_sync(0xffffffffu, sees)) {
#pragma unroll
                for (int u = 0; u < kF32Chunk; ++u) {
                    const float pu = __shfl_sync(0xffffffffu, pr, u), gu = __shfl_sync(0xffffffffu, gr, u);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        ak[e] = fmaf(gu, ch.a[u][lane + 32 * e], ak[e]);
                        av[e] = fmaf(pu, ch.b[u][lane + 32 * e], av[e]);
                    }
                }
            }
        }
    }
    if constexpr (G > 1) {
        span_f32_meet(group);      // the chunk's place takes the sums
#pragma unroll
        for (int e = 0; e < E; ++e) {
            ch.a[warp][lane + 32 * e] = ak[e];
            ch.b[warp][lane + 32 * e] = av[e];
        }
        __syncthreads();
    }
    if (group == 0 && j < L) {
#pragma unroll
        for (int u = 1; u < G; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                ak[e] += sm.chunk[u].a[warp][lane + 32 * e];
                av[e] += sm.chunk[u].b[warp][lane + 32 * e];
            }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            p.dk[row + lane + 32 * e] = p.alpha * ak[e];
            p.dv[row + lane + 32 * e] = av[e];
        }
    }
}

template <int D, int G>
__global__ void __launch_bounds__(SpanF32Smem<D, G>::kThreads) span_f32_fwd_kernel(const SpanF32Params p) {
    extern __shared__ __align__(16) uint8_t span_f32_smem[];
    auto &sm = *reinterpret_cast<SpanF32Smem<D, G> *>(span_f32_smem);
    span_f32_rows<D, G, false>(p, sm, blockIdx.x);
}

// Both halves of the backward in one launch: blocks [0, row_blocks) take rows of
// dQ, the others keys.
template <int D, int G>
__global__ void __launch_bounds__(SpanF32Smem<D, G>::kThreads) span_f32_bwd_kernel(const SpanF32Params p, unsigned row_blocks) {
    extern __shared__ __align__(16) uint8_t span_f32_smem[];
    auto &sm = *reinterpret_cast<SpanF32Smem<D, G> *>(span_f32_smem);
    if (blockIdx.x < row_blocks) span_f32_rows<D, G, true>(p, sm, blockIdx.x);
    else span_f32_keys<D, G>(p, sm, blockIdx.x - row_blocks);
}

}  // namespace sigattn
