// Appending keys and values to a paged cache, with the position rotation
// applied on the way.
//
// Token l of sample z goes to place at = cache_lens[z] + l of the sample's own
// pages, row at % page of page page_table[z][at / page], and is rotated by its
// position p = prefix_len + at: pair i of the first `rot` entries of each head
// turns by the angle p * inv_freq[i].  Values are copied, queries rotated out.
//
// Every row is read once and written once, 16 bytes a thread and access.  One warp takes
// a token (or a share of its heads, when tokens are few).  Its lanes keep their place
// within a head, so that each holds the angles of its pairs in registers for all heads
// of the token; what is left per head is the loads, two FMAs an entry and the stores.
// (One thread per unit of any head with the angles in shared memory spent its time on
// instructions: 40 us for 4 x 4096 prompt tokens, 16 + 4 heads of 128.)
//
// Bound, for many tokens, by latency: a warp's chain is the lengths, the page, its
// angles in 64 bits and two or three rounds of loads and stores, and then it ends.  The
// same 4 x 4096 tokens now take 38.4 us, 4.3 TB/s of the 6.46 that a copy reaches, with
// DRAM 39% busy under ncu and 7.8 cycles an issue spent on loads.  The bf16 instances
// spill 16 bytes at 64 registers, four blocks an SM.
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

__device__ __forceinline__ void turn_pair(float &a, float &b, float c, float s) {
    const float a0 = a;
    a = a0 * c - b * s;
    b = b * c + a0 * s;
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

// A head row is D / N vectors of 16 bytes, handled in UNITS units of two vectors
// each: with half-split pairs a unit of the rotated part is (vector u, vector u +
// rot / 2N), otherwise two neighbours.  32 / UNITS heads make one pass of a warp;
// `share` warps split a token's passes.
//
// With `ahead` the first rows are read before anything is known about the token
// (a padded row is there to be read, too), which hides the lookups of a decoding
// step; without it rows of padding cost nothing.
template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads, 4) cache_append_kernel(const AppendParams p, int share, bool ahead) {
    using Vec = AppendVec<T>;
    constexpr int N = Vec::N, VECS = D / N, UNITS = VECS / 2, HEADS = 32 / UNITS;
    constexpr int UNR = 2;        // passes whose rows are in flight together
    __shared__ __align__(16) float2 turns[kAppendThreads / 32][kAppendPairs];
    const int lane = lane_id();
    const unsigned id = blockIdx.x * (kAppendThreads / 32) + warp_id();
    const unsigned tok = id / share, sub = id % share;     // Z L tokens, below 2^31
    if (tok >= static_cast<unsigned>(p.Z) * p.L) return;
    const unsigned z = tok / p.L;
    const int l = static_cast<int>(tok - z * p.L);
    const int capacity = p.max_pages << p.page_shift;     // checked on the host to fit
    const int un = lane % UNITS, pairs = p.rot / 2, half_units = pairs / N;
    const int heads = p.H + 2 * p.Hk;                      // queries, keys, values
    // this lane's vectors, and its first pair (-1: not rotated)
    const bool neighbours = p.interleaved || un >= half_units;
    const int va = !neighbours ? un : p.interleaved ? 2 * un : 2 * half_units + 2 * (un - half_units);
    const int vb = !neighbours ? un + half_units : va + 1;
    const int pair = !neighbours ? un * N : p.interleaved && va * N < p.rot ? va * N / 2 : -1;

    const int keys = p.H, values = p.H + p.Hk;     // first head of each
    const uint4 *qrow = static_cast<const uint4 *>(p.q) + static_cast<size_t>(tok) * p.H * VECS;
    const uint4 *krow = static_cast<const uint4 *>(p.k) + (static_cast<size_t>(tok) * p.Hk - keys) * VECS;
    const uint4 *vrow = static_cast<const uint4 *>(p.v) + (static_cast<size_t>(tok) * p.Hk - values) * VECS;
    auto load = [&](int head, uint4 &a, uint4 &b) {
        const uint4 *row = (head < keys ? qrow : head < values ? krow : vrow) + head * VECS;
        a = __ldg(row + va);
        b = __ldg(row + vb);
    };
    const int first = static_cast<int>(sub) * HEADS + lane / UNITS, step = share * HEADS;
    uint4 a[UNR], b[UNR];
    if (ahead) {
#pragma unroll
        for (int u = 0; u < UNR; ++u)
            if (first + u * step < heads) load(first + u * step, a[u], b[u]);
    }

    int have = p.cache_lens[z], add = p.seqlens_new[z];
    const int base = p.prefix_len != nullptr ? max(*p.prefix_len, 0) : 0;
    if (have < 0 || have > capacity || add < 0 || add > p.L || add > capacity - have ||
        (p.prefix_len != nullptr && *p.prefix_len < 0)) {
        record_status(p.status, kStatusSeqlenRange);
        have = min(max(have, 0), capacity);
        add = min(max(add, 0), p.L);
    }
    // lens_out may be cache_lens when L is 1: then the token's warps all have to have
    // read it, and they are one warp, or one block that meets here
    if (share > 1) __syncthreads();
    if (l == 0 && sub == 0 && lane == 0) p.lens_out[z] = min(have + min(add, capacity - have), capacity);
    const bool live = l < add;
    int64_t dest = -1;       // cache row (page * page_size + slot) times Hk
    const int64_t place = static_cast<int64_t>(have) + l;
    if (live && place < capacity) {
        const int page = p.page_table[static_cast<size_t>(z) * p.max_pages + (place >> p.page_shift)];
        if (page < 0 || page >= p.pages)
            record_status(p.status, kStatusPageRange);
        else
            dest = ((static_cast<int64_t>(page) << p.page_shift) + (place & ((1 << p.page_shift) - 1))) * p.Hk;
    }
    if (live && !ahead) {
#pragma unroll
        for (int u = 0; u < UNR; ++u)
            if (first + u * step < heads) load(first + u * step, a[u], b[u]);
    }
    float2 *turn = turns[warp_id()];     // cos, sin of the token's pairs
    if (live && pairs > 0) {
        for (int i = lane; i < pairs; i += 32)
            turn[i] = position_angle(static_cast<double>(base) + place, p.inv_freq[i]);
        __syncwarp();
    }
    uint4 *qto = static_cast<uint4 *>(p.q_out) + static_cast<size_t>(tok) * p.H * VECS;
    uint4 *kto = static_cast<uint4 *>(p.k_pages) + (dest - keys) * VECS;
    uint4 *vto = static_cast<uint4 *>(p.v_pages) + (dest - values) * VECS;
    const float4 *cs = reinterpret_cast<const float4 *>(turn + max(pair, 0));
    auto finish = [&](int head, uint4 x16, uint4 y16) {
        if (head < keys) {
            if (!live) x16 = y16 = make_uint4(0u, 0u, 0u, 0u);      // a padded query row
        } else if (dest < 0) {
            return;
        }
        uint4 *to = (head < keys ? qto : head < values ? kto : vto) + head * VECS;
        if (pair >= 0 && live && head < values) {
            float x[N], y[N];
            Vec::open(x16, x);
            Vec::open(y16, y);
            if (p.interleaved) {
#pragma unroll
                for (int i = 0; i < N; i += 4) {
                    const float4 c = cs[i / 4], d = cs[N / 4 + i / 4];      // two pairs each
                    turn_pair(x[i], x[i + 1], c.x, c.y);
                    turn_pair(x[i + 2], x[i + 3], c.z, c.w);
                    turn_pair(y[i], y[i + 1], d.x, d.y);
                    turn_pair(y[i + 2], y[i + 3], d.z, d.w);
                }
            } else {
#pragma unroll
                for (int i = 0; i < N; i += 2) {
                    const float4 c = cs[i / 2];
                    turn_pair(x[i], y[i], c.x, c.y);
                    turn_pair(x[i + 1], y[i + 1], c.z, c.w);
                }
            }
            x16 = Vec::close(x);
            y16 = Vec::close(y);
        }
        to[va] = x16;
        to[vb] = y16;
    };
#pragma unroll
    for (int u = 0; u < UNR; ++u)
        if (first + u * step < heads) finish(first + u * step, a[u], b[u]);
    for (int h0 = first + UNR * step; h0 < heads; h0 += UNR * step) {
#pragma unroll
        for (int u = 0; u < UNR; ++u)
            if (live && h0 + u * step < heads) load(h0 + u * step, a[u], b[u]);
#pragma unroll
        for (int u = 0; u < UNR; ++u)
            if (h0 + u * step < heads) finish(h0 + u * step, a[u], b[u]);
    }
}

}  // namespace sigattn
