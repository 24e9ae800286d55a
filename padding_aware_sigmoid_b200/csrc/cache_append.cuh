// Appending keys and values to a paged cache, with the position rotation
// applied on the way.
//
// Token l of sample z goes to place at = cache_lens[z] + l of the sample's own
// pages, row at % page of page page_table[z][at / page], and is rotated by its
// position p = prefix_len + at: pair i of the first `rot` entries of each head
// turns by the angle p * inv_freq[i].  Values are copied, queries rotated out.
//
// Pure traffic: every row is read once and written once, 16 bytes a thread and
// access.  The angles of a token (rot / 2 of them) are shared by all its heads:
// a block holds a few tokens, issues its loads first, forms the angles of its
// tokens while they fly, and rotates and stores after one barrier.
#pragma once

#include <stdint.h>

#include "sm100.cuh"

namespace sigattn {

constexpr int kStatusPageRange = 10;

struct AppendParams {
    const void *k, *v, *q;
    void *q_out, *k_pages, *v_pages;
    const int *page_table, *cache_lens, *seqlens_new, *prefix_len;
    int *lens_out;
    const float *inv_freq;
    int Z, L, H, Hk;              // H: query heads (0: no queries)
    int pages, page_shift, max_pages;
    int rot, interleaved;
    int *status;
};

constexpr int kAppendThreads = 256;
constexpr int kAppendPairs = 64;     // most angle pairs of a head (D / 2)

// sin and cos of p * f for any position: the product and its reduction to
// [-pi, pi] in 64 bits (an angle of 10^6 keeps 2^-30 of a radian), the
// functions in 32.
__device__ __forceinline__ float2 position_angle(double p, float f) {
    const double a = p * static_cast<double>(f);
    const double turns = rint(a * 0.15915494309189535);
    double r = fma(turns, -6.283185307179586, a);
    r = fma(turns, -2.4492935982947064e-16, r);
    float s, c;
    sincosf(static_cast<float>(r), &s, &c);
    return make_float2(c, s);
}

template <typename T>
struct AppendVec;
template <>
struct AppendVec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void open(const uint4 &u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    // one rounding, to nearest even
    static __device__ __forceinline__ uint4 close(const float (&x)[8]) {
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                          pack_bf16x2(x[6], x[7]));
    }
};
template <>
struct AppendVec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void open(const uint4 &u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x);
        x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z);
        x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 close(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
    }
};

// TOK tokens a block.  A head row is D / N vectors of 16 bytes, handled in
// D / 2N units of two vectors each: with half-split pairs a unit of the rotated
// part is (vector u, vector u + rot / 2N), otherwise two neighbours.
template <typename T, int D, int TOK>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const AppendParams p) {
    using Vec = AppendVec<T>;
    constexpr int N = Vec::N, VECS = D / N, UNITS = VECS / 2;
    __shared__ float2 turn[TOK][kAppendPairs];
    __shared__ int64_t dest[TOK];      // cache row (page * page_size + slot) times Hk, or < 0
    __shared__ int live[TOK];          // 1: a token of its sample, 0: padding
    __shared__ int after[TOK];         // its sample's new length, < 0: written by another token
    const int64_t tokens = static_cast<int64_t>(p.Z) * p.L;
    const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * TOK;
    const int capacity = p.max_pages << p.page_shift;     // checked on the host to fit
    const int tid = threadIdx.x;

    // where each token goes
    if (tid < TOK) {
        const int64_t tok = tok0 + tid;
        int ok = 0, sum = -1;
        int64_t to = -1;
        if (tok < tokens) {
            const int z = static_cast<int>(tok / p.L), l = static_cast<int>(tok % p.L);
            int have = p.cache_lens[z], add = p.seqlens_new[z];
            if (have < 0 || have > capacity || add < 0 || add > p.L || add > capacity - have) {
                record_status(p.status, kStatusSeqlenRange);
                have = min(max(have, 0), capacity);
                add = min(max(add, 0), p.L);
            }
            ok = l < add;
            if (l == 0) sum = min(have + min(add, capacity - have), capacity);
            const int64_t at = static_cast<int64_t>(have) + l;
            if (ok && at < capacity) {
                const int page = p.page_table[static_cast<size_t>(z) * p.max_pages + (at >> p.page_shift)];
                if (page < 0 || page >= p.pages)
                    record_status(p.status, kStatusPageRange);
                else
                    to = ((static_cast<int64_t>(page) << p.page_shift) + (at & ((1 << p.page_shift) - 1))) * p.Hk;
            }
        }
        after[tid] = sum;
        live[tid] = ok;
        dest[tid] = to;
    }
    // the tokens' angles
    const int pairs = p.rot / 2;
    const int base = p.prefix_len != nullptr ? max(*p.prefix_len, 0) : 0;
    for (int e = tid; e < TOK * pairs; e += kAppendThreads) {
        const int t = e / pairs, i = e % pairs;
        const int64_t tok = tok0 + t;
        if (tok < tokens) {
            const int z = static_cast<int>(tok / p.L), l = static_cast<int>(tok % p.L);
            const int have = min(max(p.cache_lens[z], 0), capacity);
            if (l < p.seqlens_new[z])
                turn[t][i] = position_angle(static_cast<double>(base) + have + l, p.inv_freq[i]);
        }
    }
    __syncthreads();
    // not before the barrier: with single tokens lens_out may be cache_lens
    if (tid < TOK && after[tid] >= 0) p.lens_out[(tok0 + tid) / p.L] = after[tid];

    const int heads = p.H + 2 * p.Hk;       // queries, keys, values
    const int per_token = heads * UNITS;
    const int half_units = pairs / N;       // rotated units with half-split pairs
    const uint4 *q = static_cast<const uint4 *>(p.q), *k = static_cast<const uint4 *>(p.k),
                *v = static_cast<const uint4 *>(p.v);
    constexpr int U = 4;                    // units in flight per thread
    for (int e0 = tid; e0 < TOK * per_token; e0 += U * kAppendThreads) {
        uint4 a[U], b[U];
        const uint4 *from[U];
        uint4 *to[U];
        int va[U], vb[U], tk[U], pair0[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = e0 + u * kAppendThreads;
            from[u] = nullptr;
            to[u] = nullptr;
            if (e >= TOK * per_token) continue;
            const int t = e / per_token, w = e % per_token;
            const int head = w / UNITS, un = w % UNITS;
            const int64_t tok = tok0 + t;
            if (tok >= tokens) continue;
            tk[u] = t;
            pair0[u] = -1;
            if (p.interleaved || un >= half_units) {
                // two neighbouring vectors
                va[u] = p.interleaved ? 2 * un : 2 * half_units + 2 * (un - half_units);
                vb[u] = va[u] + 1;
                if (p.interleaved && va[u] * N < p.rot) pair0[u] = va[u] * N / 2;
            } else {
                va[u] = un;
                vb[u] = un + half_units;
                pair0[u] = un * N;
            }
            if (head < p.H) {
                const size_t row = (static_cast<size_t>(tok) * p.H + head) * VECS;
                to[u] = static_cast<uint4 *>(p.q_out) + row;
                if (live[t]) from[u] = q + row;
            } else if (live[t] && dest[t] >= 0) {
                const bool key = head < p.H + p.Hk;
                const int hk = head - p.H - (key ? 0 : p.Hk);
                from[u] = (key ? k : v) + (static_cast<size_t>(tok) * p.Hk + hk) * VECS;
                to[u] = static_cast<uint4 *>(key ? p.k_pages : p.v_pages) + (static_cast<size_t>(dest[t]) + hk) * VECS;
                if (!key) pair0[u] = -1;
            }
            if (from[u] != nullptr) {
                a[u] = from[u][va[u]];
                b[u] = from[u][vb[u]];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (to[u] == nullptr) continue;
            if (from[u] == nullptr) {          // a padded query row
                to[u][va[u]] = to[u][vb[u]] = make_uint4(0u, 0u, 0u, 0u);
                continue;
            }
            if (pair0[u] >= 0) {
                float x[N], y[N];
                Vec::open(a[u], x);
                Vec::open(b[u], y);
                const float2 *cs = &turn[tk[u]][pair0[u]];
                if (p.interleaved) {
#pragma unroll
                    for (int i = 0; i < N; i += 2) {
                        const float2 c = cs[i / 2], d = cs[N / 2 + i / 2];
                        const float x0 = x[i], y0 = y[i];
                        x[i] = x0 * c.x - x[i + 1] * c.y;
                        x[i + 1] = x[i + 1] * c.x + x0 * c.y;
                        y[i] = y0 * d.x - y[i + 1] * d.y;
                        y[i + 1] = y[i + 1] * d.x + y0 * d.y;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const float2 c = cs[i];
                        const float x0 = x[i];
                        x[i] = x0 * c.x - y[i] * c.y;
                        y[i] = y[i] * c.x + x0 * c.y;
                    }
                }
                a[u] = Vec::close(x);
                b[u] = Vec::close(y);
            }
            to[u][va[u]] = a[u];
            to[u][vb[u]] = b[u];
        }
    }
}

}  // namespace sigattn
