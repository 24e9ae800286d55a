// fp32 accuracy path of the masked attention (span_score.cuh): one warp per
// output row, fp32 arithmetic throughout, library expf and tanhf.  Lanes are
// keys (or queries) while scores are formed, so that a weight is computed once and
// no reduction is needed, and entries of the row while it is accumulated.
// Bound by latency: meant for accuracy checks at small sizes.
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

// Dot products of the row `x` (D floats, the same address in every lane) with
// this lane's rows a and b.
template <int D>
__device__ __forceinline__ float row_dot(const float *x, const float *a) {
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const float4 *x4 = reinterpret_cast<const float4 *>(x), *a4 = reinterpret_cast<const float4 *>(a);
#pragma unroll
    for (int e = 0; e < D / 4; ++e) {
        const float4 u = __ldg(x4 + e), v = __ldg(a4 + e);
        s[0] = fmaf(u.x, v.x, s[0]);
        s[1] = fmaf(u.y, v.y, s[1]);
        s[2] = fmaf(u.z, v.z, s[2]);
        s[3] = fmaf(u.w, v.w, s[3]);
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// Forward (DQ false) or dQ (DQ true): one warp per (z, i, h).
template <int D, bool DQ>
__device__ __forceinline__ void span_f32_row(const SpanF32Params &p, int64_t r) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, L = p.src.L;
    if (r >= static_cast<int64_t>(p.Z) * L * p.H) return;
    const int h = static_cast<int>(r % p.H);
    const int i = static_cast<int>((r / p.H) % L);
    const int z = static_cast<int>(r / (static_cast<int64_t>(p.H) * L));
    const int n = span_tokens(p.src, z);
    const int2 span = row_span(p.src, z, i, n);
    const float bias = bias_of(p.bias_z, p.bias, z), slope = p.slopes != nullptr ? p.slopes[h] : 0.0f;
    const int64_t krow = static_cast<int64_t>(p.Hk) * D;
    const int64_t kbase = static_cast<int64_t>(z) * L * krow + static_cast<int64_t>(h / p.group) * D;
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    for (int j0 = span.x; j0 < span.y; j0 += 32) {
        const int j = j0 + lane;
        float w = 0.0f;
        if (j < span.y) {
            const int64_t at = kbase + j * krow;
            float pr, g;
            span_exact(p.alpha * row_dot<D>(p.q + r * D, p.k + at), p.cap,
                       fmaf(-slope, fabsf(static_cast<float>(i - j)), bias), pr, g);
            w = DQ ? g * row_dot<D>(p.dout + r * D, p.v + at) : pr;
        }
        const float *src = (DQ ? p.k : p.v) + kbase + j0 * krow + lane;
        const int m = min(32, span.y - j0);
        if (m == 32) {
#pragma unroll 8
            for (int u = 0; u < 32; ++u) {
                const float wu = __shfl_sync(0xffffffffu, w, u);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = fmaf(wu, __ldg(src + u * krow + 32 * e), acc[e]);
            }
        } else {
            for (int u = 0; u < m; ++u) {
                const float wu = __shfl_sync(0xffffffffu, w, u);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = fmaf(wu, __ldg(src + u * krow + 32 * e), acc[e]);
            }
        }
    }
    float *out = (DQ ? p.dq : p.o) + r * D + lane;
#pragma unroll
    for (int e = 0; e < E; ++e) out[32 * e] = DQ ? p.alpha * acc[e] : acc[e];
}

// dK and dV: one warp per (z, j, key head), over the queries of its heads.
template <int D>
__device__ __forceinline__ void span_f32_key(const SpanF32Params &p, int64_t r) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, L = p.src.L;
    if (r >= static_cast<int64_t>(p.Z) * L * p.Hk) return;
    const int kvh = static_cast<int>(r % p.Hk);
    const int j = static_cast<int>((r / p.Hk) % L);
    const int z = static_cast<int>(r / (static_cast<int64_t>(p.Hk) * L));
    const int n = span_tokens(p.src, z);
    const float bias = bias_of(p.bias_z, p.bias, z);
    const int64_t qrow = static_cast<int64_t>(p.H) * D;
    float ak[E], av[E];
#pragma unroll
    for (int e = 0; e < E; ++e) ak[e] = av[e] = 0.0f;
    for (int h = kvh * p.group; j < n && h < (kvh + 1) * p.group; ++h) {
        const float slope = p.slopes != nullptr ? p.slopes[h] : 0.0f;
        const int64_t base = static_cast<int64_t>(z) * L * qrow + static_cast<int64_t>(h) * D;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int i = i0 + lane;
            const int2 sp = row_span(p.src, z, i, n);
            const bool sees = j >= sp.x && j < sp.y;
            unsigned who = __ballot_sync(0xffffffffu, sees);
            if (who == 0) continue;
            float pr = 0.0f, g = 0.0f;
            if (sees) {
                const int64_t at = base + i * qrow;
                span_exact(p.alpha * row_dot<D>(p.k + r * D, p.q + at), p.cap,
                           fmaf(-slope, fabsf(static_cast<float>(i - j)), bias), pr, g);
                g *= row_dot<D>(p.v + r * D, p.dout + at);
            }
            // only rows that see the key are read: the others may be padding
            const int64_t at = base + i0 * qrow + lane;
            auto add = [&](int u) {
                const float pu = __shfl_sync(0xffffffffu, pr, u), gu = __shfl_sync(0xffffffffu, g, u);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    ak[e] = fmaf(gu, __ldg(p.q + at + u * qrow + 32 * e), ak[e]);
                    av[e] = fmaf(pu, __ldg(p.dout + at + u * qrow + 32 * e), av[e]);
                }
            };
            if (who == 0xffffffffu) {
#pragma unroll 8
                for (int u = 0; u < 32; ++u) add(u);
            } else {
                for (; who != 0; who &= who - 1) add(__ffs(who) - 1);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
        p.dk[r * D + lane + 32 * e] = p.alpha * ak[e];
        p.dv[r * D + lane + 32 * e] = av[e];
    }
}

template <int D>
__global__ void __launch_bounds__(256) span_f32_fwd_kernel(const SpanF32Params p) {
    span_f32_row<D, false>(p, static_cast<int64_t>(blockIdx.x) * 8 + warp_id());
}

// Both halves of the backward in one launch: blocks [0, row_blocks) take rows of
// dQ, the others keys.
template <int D>
__global__ void __launch_bounds__(256) span_f32_bwd_kernel(const SpanF32Params p, unsigned row_blocks) {
    if (blockIdx.x < row_blocks)
        span_f32_row<D, true>(p, static_cast<int64_t>(blockIdx.x) * 8 + warp_id());
    else
        span_f32_key<D>(p, static_cast<int64_t>(blockIdx.x - row_blocks) * 8 + warp_id());
}

}  // namespace sigattn
