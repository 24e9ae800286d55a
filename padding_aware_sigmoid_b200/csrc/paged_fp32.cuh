// fp32 accuracy path of the paged attention: one block per output row, its
// warps taking groups of four keys in turn, library expf and tanhf.
#pragma once

#include "paged_sm100.cuh"
#include "span_fp32.cuh"

namespace sigattn {

constexpr int kPagedF32Warps = 8;

template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

// The shapes, tables and lengths of `p` are those of the bf16 path; its
// tensors are not used.
template <int D>
__global__ void __launch_bounds__(32 * kPagedF32Warps)
    paged_f32_kernel(const PagedParams p, const float *q, const float *k_pages, const float *v_pages, float *o) {
    constexpr int E = D / 32, U = 4;
    __shared__ float sums[kPagedF32Warps][D];
    const int64_t r = blockIdx.x;
    const int lane = lane_id(), warp = warp_id();
    const int h = static_cast<int>(r % p.H);
    const int64_t tok = r / p.H;
    const int z = static_cast<int>(tok / p.L), l = static_cast<int>(tok % p.L);
    const int kvh = h / p.group;
    const int2 n = paged_lengths(p, z);
    const int prefix = paged_prefix(p);
    const bool live = l < n.y;
    const int own = live ? n.x - n.y + l + 1 : 0;           // own keys that the row sees
    const int64_t keys = live ? static_cast<int64_t>(prefix) + own : 0;
    const float bias = bias_of(p.bias_z, p.bias, z), slope = p.slopes != nullptr ? p.slopes[h] : 0.0f;
    const int mask = (1 << p.page_shift) - 1;
    float acc[E], qv[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        acc[e] = 0.0f;
        qv[e] = q[r * D + lane + 32 * e];
    }
    for (int64_t j = static_cast<int64_t>(warp) * U; j < keys; j += U * kPagedF32Warps) {
        float s[U], vv[U][E];
        bool ok[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t key = j + u;
            ok[u] = key < keys;
            s[u] = 0.0f;
            int64_t row = 0;
            if (ok[u]) {
                const bool ahead = key < prefix;
                const int at = static_cast<int>(ahead ? key : key - prefix);
                const int page = ahead ? p.prefix_table[at >> p.page_shift]
                                       : p.page_table[static_cast<size_t>(z) * p.max_pages + (at >> p.page_shift)];
                if (page < 0 || page >= p.pages) {
                    if (lane == 0) record_status(p.status, kStatusPageRange);
                    ok[u] = false;
                } else {
                    row = (((static_cast<int64_t>(page) << p.page_shift) + (at & mask)) * p.Hk + kvh) * D + lane;
                }
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                s[u] = fmaf(qv[e], ok[u] ? k_pages[row + 32 * e] : 0.0f, s[u]);
                vv[u][e] = ok[u] ? v_pages[row + 32 * e] : 0.0f;
            }
        }
        warp_sums(s);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float w, g;
            span_exact(p.alpha * s[u], p.cap, fmaf(-slope, static_cast<float>(keys - 1 - j - u), bias), w, g);
            w = ok[u] ? w : 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(w, vv[u][e], acc[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sums[warp][lane + 32 * e] = acc[e];
    __syncthreads();
    for (int e = threadIdx.x; e < D; e += 32 * kPagedF32Warps) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < kPagedF32Warps; ++w) t += sums[w][e];
        o[r * D + e] = t;
    }
}

}  // namespace sigattn
