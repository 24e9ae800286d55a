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
// part is (vector u, vector u + rot / 2N), otherwise two neighbours.  Every
// thread reads its first UNR units before the lookups and the angles, which the
// loads cover.  With one token a block (latency counts) nothing at all is known
// about the token by then: a padded row is there to be read, too.  With several
// (traffic counts) rows of padding are left out.
template <typename T, int D, int TOK>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const AppendParams p) {
    using Vec = AppendVec<T>;
    constexpr int N = Vec::N, VECS = D / N, UNITS = VECS / 2;
    constexpr int UNR = 3;
    __shared__ float2 turn[TOK][kAppendPairs];
    __shared__ int64_t dest[TOK];      // cache row (page * page_size + slot) times Hk, or < 0
    __shared__ int live[TOK];          // 1: a token of its sample, 0: padding
    __shared__ int after[TOK];         // its sample's new length, < 0: written by another token
    const int64_t tokens = static_cast<int64_t>(p.Z) * p.L;
    const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * TOK;
    const int here = static_cast<int>(min(static_cast<int64_t>(TOK), tokens - tok0));
    const int capacity = p.max_pages << p.page_shift;     // checked on the host to fit
    const int tid = threadIdx.x;
    const int pairs = p.rot / 2;
    const int heads = p.H + 2 * p.Hk;       // queries, keys, values
    const int per_token = heads * UNITS, all = here * per_token;
    const int half_units = pairs / N;       // rotated units with half-split pairs
    const uint4 *q = static_cast<const uint4 *>(p.q), *k = static_cast<const uint4 *>(p.k),
                *v = static_cast<const uint4 *>(p.v);

    // one unit: its token and head, its vectors, its first pair (-1: not rotated)
    struct Unit {
        int t, head, va, vb, pair;
    };
    auto unit_of = [&](int e) {
        Unit u;
        u.t = TOK == 1 ? 0 : e / per_token;
        const int w = e - u.t * per_token, un = w % UNITS;
        u.head = w / UNITS;
        u.pair = -1;
        if (p.interleaved || un >= half_units) {
            u.va = p.interleaved ? 2 * un : 2 * half_units + 2 * (un - half_units);
            u.vb = u.va + 1;
            if (p.interleaved && u.va * N < p.rot) u.pair = u.va * N / 2;
        } else {
            u.va = un;
            u.vb = un + half_units;
            u.pair = un * N;
        }
        if (u.head >= p.H + p.Hk) u.pair = -1;    // a value
        return u;
    };
    auto is_live = [&](int t) {
        const unsigned tok = static_cast<unsigned>(tok0) + t, z = tok / p.L;     // below 2^31
        return static_cast<int>(tok - z * p.L) < __ldg(p.seqlens_new + z);
    };
    auto load = [&](const Unit &u, uint4 &a, uint4 &b) {
        const size_t tok = static_cast<size_t>(tok0 + u.t);
        const uint4 *row = u.head < p.H ? q + (tok * p.H + u.head) * VECS
                           : u.head < p.H + p.Hk ? k + (tok * p.Hk + (u.head - p.H)) * VECS
                                                 : v + (tok * p.Hk + (u.head - p.H - p.Hk)) * VECS;
        a = __ldg(row + u.va);
        b = __ldg(row + u.vb);
    };
    auto finish = [&](const Unit &u, uint4 a, uint4 b) {
        uint4 *to;
        if (u.head < p.H) {
            to = static_cast<uint4 *>(p.q_out) + (static_cast<size_t>(tok0 + u.t) * p.H + u.head) * VECS;
            if (!live[u.t]) {      // a padded query row
                to[u.va] = to[u.vb] = make_uint4(0u, 0u, 0u, 0u);
                return;
            }
        } else {
            if (dest[u.t] < 0) return;
            const bool key = u.head < p.H + p.Hk;
            to = static_cast<uint4 *>(key ? p.k_pages : p.v_pages) +
                 (static_cast<size_t>(dest[u.t]) + u.head - p.H - (key ? 0 : p.Hk)) * VECS;
        }
        if (u.pair >= 0) {
            float x[N], y[N];
            Vec::open(a, x);
            Vec::open(b, y);
            const float2 *cs = &turn[u.t][u.pair];
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
            a = Vec::close(x);
            b = Vec::close(y);
        }
        to[u.va] = a;
        to[u.vb] = b;
    };

    uint4 a[UNR], b[UNR];
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
        const int e = tid + u * kAppendThreads;
        if (e < all) {
            const Unit un = unit_of(e);
            if (TOK == 1 || is_live(un.t)) load(un, a[u], b[u]);
        }
    }

    // where each token goes, by the last warp
    if (tid >= kAppendThreads - 32 && tid - (kAppendThreads - 32) < here) {
        const int t = tid - (kAppendThreads - 32);
        const int64_t tok = tok0 + t;
        const int z = static_cast<int>(tok / p.L), l = static_cast<int>(tok % p.L);
        int have = p.cache_lens[z], add = p.seqlens_new[z];
        if (have < 0 || have > capacity || add < 0 || add > p.L || add > capacity - have) {
            record_status(p.status, kStatusSeqlenRange);
            have = min(max(have, 0), capacity);
            add = min(max(add, 0), p.L);
        }
        after[t] = l == 0 ? min(have + min(add, capacity - have), capacity) : -1;
        live[t] = l < add;
        const int64_t at = static_cast<int64_t>(have) + l;
        int64_t to = -1;
        if (l < add && at < capacity) {
            const int page = p.page_table[static_cast<size_t>(z) * p.max_pages + (at >> p.page_shift)];
            if (page < 0 || page >= p.pages)
                record_status(p.status, kStatusPageRange);
            else
                to = ((static_cast<int64_t>(page) << p.page_shift) + (at & ((1 << p.page_shift) - 1))) * p.Hk;
        }
        dest[t] = to;
    }
    // the tokens' angles
    const int base = p.prefix_len != nullptr ? max(*p.prefix_len, 0) : 0;
    for (int e = tid; e < here * pairs; e += kAppendThreads) {
        const int t = TOK == 1 ? 0 : e / pairs, i = e - t * pairs;
        const int64_t tok = tok0 + t;
        const int z = static_cast<int>(tok / p.L), l = static_cast<int>(tok % p.L);
        const int have = min(max(p.cache_lens[z], 0), capacity);
        if (l < p.seqlens_new[z]) turn[t][i] = position_angle(static_cast<double>(base) + have + l, p.inv_freq[i]);
    }
    __syncthreads();
    // not before the barrier: with single tokens lens_out may be cache_lens
    if (tid < here && after[tid] >= 0) p.lens_out[(tok0 + tid) / p.L] = after[tid];

#pragma unroll
    for (int u = 0; u < UNR; ++u) {
        const int e = tid + u * kAppendThreads;
        if (e < all) finish(unit_of(e), a[u], b[u]);
    }
    for (int e = tid + UNR * kAppendThreads; e < all; e += kAppendThreads) {
        const Unit un = unit_of(e);
        if (live[un.t]) load(un, a[0], b[0]);
        finish(un, a[0], b[0]);
    }
}

}  // namespace sigattn
