// fp32 accuracy path of the masked attention (span_score.cuh): one warp per
// output row, fp32 arithmetic throughout, library expf and tanhf.  Four keys
// (or queries) go side by side so that their reductions overlap.  Meant for
// accuracy checks at small sizes, not for speed.
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

template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

// Forward (DQ false) or dQ (DQ true): one warp per (z, i, h).
template <int D, bool DQ>
__global__ void __launch_bounds__(256) span_f32_rows_kernel(const SpanF32Params p) {
    constexpr int E = D / 32, U = 4;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, L = p.src.L;
    if (r >= static_cast<int64_t>(p.Z) * L * p.H) return;
    const int h = static_cast<int>(r % p.H);
    const int i = static_cast<int>((r / p.H) % L);
    const int z = static_cast<int>(r / (static_cast<int64_t>(p.H) * L));
    const int n = span_tokens(p.src, z);
    const int2 span = row_span(p.src, z, i, n);
    const float bias = bias_of(p.bias_z, p.bias, z), slope = p.slopes != nullptr ? p.slopes[h] : 0.0f;
    const int64_t krow = static_cast<int64_t>(p.Hk) * D;
    const int64_t kbase = static_cast<int64_t>(z) * L * krow + static_cast<int64_t>(h / p.group) * D + lane;
    float acc[E], qv[E], gv[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        acc[e] = 0.0f;
        qv[e] = p.q[r * D + lane + 32 * e];
        gv[e] = DQ ? p.dout[r * D + lane + 32 * e] : 0.0f;
    }
    for (int j = span.x; j < span.y; j += U) {
        float s[U], dp[U], kv[U][E], vv[U][E];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t at = kbase + static_cast<int64_t>(min(j + u, span.y - 1)) * krow;
            s[u] = dp[u] = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                kv[u][e] = p.k[at + 32 * e];
                vv[u][e] = p.v[at + 32 * e];
                s[u] = fmaf(qv[e], kv[u][e], s[u]);
                if (DQ) dp[u] = fmaf(gv[e], vv[u][e], dp[u]);
            }
        }
        warp_sums(s);
        if (DQ) warp_sums(dp);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j + u >= span.y) break;
            float pr, g;
            span_exact(p.alpha * s[u], p.cap, fmaf(-slope, fabsf(static_cast<float>(i - j - u)), bias), pr, g);
            const float w = DQ ? g * dp[u] : pr;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(w, DQ ? kv[u][e] : vv[u][e], acc[e]);
        }
    }
    float *out = (DQ ? p.dq : p.o) + r * D + lane;
#pragma unroll
    for (int e = 0; e < E; ++e) out[32 * e] = DQ ? p.alpha * acc[e] : acc[e];
}

// dK and dV: one warp per (z, j, key head), over the queries of its heads.
template <int D>
__global__ void __launch_bounds__(256) span_f32_dkdv_kernel(const SpanF32Params p) {
    constexpr int E = D / 32, U = 4;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, L = p.src.L;
    if (r >= static_cast<int64_t>(p.Z) * L * p.Hk) return;
    const int kvh = static_cast<int>(r % p.Hk);
    const int j = static_cast<int>((r / p.Hk) % L);
    const int z = static_cast<int>(r / (static_cast<int64_t>(p.Hk) * L));
    const int n = span_tokens(p.src, z);
    const float bias = bias_of(p.bias_z, p.bias, z);
    const int64_t qrow = static_cast<int64_t>(p.H) * D;
    float ak[E], av[E], kv[E], vv[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        ak[e] = av[e] = 0.0f;
        kv[e] = p.k[r * D + lane + 32 * e];
        vv[e] = p.v[r * D + lane + 32 * e];
    }
    for (int h = kvh * p.group; j < n && h < (kvh + 1) * p.group; ++h) {
        const float slope = p.slopes != nullptr ? p.slopes[h] : 0.0f;
        const int64_t base = static_cast<int64_t>(z) * L * qrow + static_cast<int64_t>(h) * D + lane;
        for (int i = 0; i < n; i += U) {
            bool sees[U];
            bool any = false;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int2 sp = row_span(p.src, z, i + u, n);
                sees[u] = j >= sp.x && j < sp.y;
                any |= sees[u];
            }
            if (!any) continue;
            float s[U], dp[U], qv[U][E], gv[U][E];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t at = base + static_cast<int64_t>(min(i + u, n - 1)) * qrow;
                s[u] = dp[u] = 0.0f;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    qv[u][e] = p.q[at + 32 * e];
                    gv[u][e] = p.dout[at + 32 * e];
                    s[u] = fmaf(kv[e], qv[u][e], s[u]);
                    dp[u] = fmaf(vv[e], gv[u][e], dp[u]);
                }
            }
            warp_sums(s);
            warp_sums(dp);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!sees[u]) continue;
                float pr, g;
                span_exact(p.alpha * s[u], p.cap, fmaf(-slope, fabsf(static_cast<float>(i + u - j)), bias), pr, g);
                g *= dp[u];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    ak[e] = fmaf(g, qv[u][e], ak[e]);
                    av[e] = fmaf(pr, gv[u][e], av[e]);
                }
            }
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
        p.dk[r * D + lane + 32 * e] = p.alpha * ak[e];
        p.dv[r * D + lane + 32 * e] = av[e];
    }
}

}  // namespace sigattn
