// What the masked-attention kernels share: the score function and the spans.
//
//   x_ij = c tanh(alpha s_ij / c) - m_h |i - j| + b     (c = 0: alpha s_ij)
//   P_ij = sigma(x_ij) where row i sees key j, 0 elsewhere
//   dP -> ds: dx/d(alpha s) = 1 - tanh^2(alpha s / c)
//
// Row i of a sample of n tokens sees the keys lo_i <= j < hi_i of its span,
// clipped to [0, n); rows at or beyond n see none.  One interval a row covers
// causal, prefix, document and window masks, and the hull of a tile's rows
// gives the key tiles it has to visit, so nothing else is loaded or computed.
#pragma once

#include <stdint.h>

#include "sigmoid.cuh"
#include "sm100.cuh"

namespace sigattn {

// SCORE: which terms a kernel instance evaluates.
enum ScoreTerms : int { kScoreCap = 1, kScoreSlope = 2 };

__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Coefficients of one (sample, head).  k = 1/2 (TANH) or log2 e (EXP) is the
// factor each sigma form wants on its argument (see SigmoidCoef).
struct ScoreCoef {
    float a;    // on the raw product: k alpha, or alpha / cap with a cap
    float c;    // k b
    float cap;  // k cap
    float m;    // -k m_h
};

template <int MODE, int SCORE>
__device__ __forceinline__ ScoreCoef make_score(float alpha, float bias, float cap, float slope) {
    const float k = MODE == kSigmoidTanh ? 0.5f : kLog2e;
    ScoreCoef r;
    r.a = SCORE & kScoreCap ? alpha / cap : k * alpha;
    r.c = k * bias;
    r.cap = k * cap;
    r.m = -k * slope;
    return r;
}

// Additive part of the arguments of two neighbouring columns; `rel` is this
// row's position less the first column's.
template <int SCORE>
__device__ __forceinline__ float2 score_addend(const ScoreCoef &cf, float rel) {
    if constexpr (SCORE & kScoreSlope)
        return fma2(f2(fabsf(rel), fabsf(rel - 1.0f)), f2(cf.m, cf.m), f2(cf.c, cf.c));
    else
        return f2(cf.c, cf.c);
}

// tanh of two capped scores, and 1 - tanh^2.  TANH mode takes the hardware
// tanh (relative error 2^-11, so the capped score moves by at most 2^-11 of
// itself); EXP mode forms (1 - e) / (1 + e) with e = exp(-2 |y|), accurate to
// 2^-21 absolutely, and 4 e / (1 + e)^2, in which nothing cancels.
template <int MODE, bool GRAD>
__device__ __forceinline__ float2 cap_tanh2(float2 y, float2 &f) {
    if constexpr (MODE == kSigmoidTanh) {
        const float2 t = f2(tanh_approx(y.x), tanh_approx(y.y));
        if constexpr (GRAD) f = fma2(mul2(t, f2(-1.0f, -1.0f)), t, f2(1.0f, 1.0f));
        return t;
    } else {
        const float2 e = f2(ex2_approx(-2.0f * kLog2e * fabsf(y.x)), ex2_approx(-2.0f * kLog2e * fabsf(y.y)));
        const float2 r = f2(rcp_approx(1.0f + e.x), rcp_approx(1.0f + e.y));
        const float2 t = mul2(fma2(e, f2(-1.0f, -1.0f), f2(1.0f, 1.0f)), r);
        if constexpr (GRAD) f = mul2(mul2(f2(4.0f, 4.0f), e), mul2(r, r));
        return f2(copysignf(t.x, y.x), copysignf(t.y, y.y));
    }
}

// P of two neighbouring columns from their raw products.
template <int MODE, int SCORE>
__device__ __forceinline__ float2 score_p2(float s0, float s1, const ScoreCoef &cf, float rel) {
    const float2 add = score_addend<SCORE>(cf, rel);
    float2 y;
    if constexpr (SCORE & kScoreCap) {
        float2 f;
        const float2 t = cap_tanh2<MODE, false>(mul2(f2(s0, s1), f2(cf.a, cf.a)), f);
        y = fma2(t, f2(cf.cap, cf.cap), add);
    } else {
        y = fma2(f2(s0, s1), f2(cf.a, cf.a), add);
    }
    return sigma2<MODE>(y);
}

// P and g = dP/d(alpha s) of two neighbouring columns.
template <int MODE, int SCORE>
__device__ __forceinline__ void score_pg2(float s0, float s1, const ScoreCoef &cf, float rel, float2 &p,
                                          float2 &g) {
    const float2 add = score_addend<SCORE>(cf, rel);
    if constexpr (SCORE & kScoreCap) {
        float2 f;
        const float2 t = cap_tanh2<MODE, true>(mul2(f2(s0, s1), f2(cf.a, cf.a)), f);
        sigma_grad2<MODE>(fma2(t, f2(cf.cap, cf.cap), add), p, g);
        g = mul2(g, f);
    } else {
        sigma_grad2<MODE>(fma2(f2(s0, s1), f2(cf.a, cf.a), add), p, g);
    }
}

// ------------------------------------------------------------------ spans

// Where the kernels take a batch's masks from.  spans null: every row of a
// sample sees all its keys.
struct SpanSource {
    const int2 *spans;     // [Z][L] {lo, hi}
    const int *seqlens;    // [Z]
    int L;
    int *status;
};

// Tokens of sample z, clamped to [0, L].
__device__ __forceinline__ int span_tokens(const SpanSource &s, int z) {
    int n = s.seqlens[z];
    if (n < 0 || n > s.L) {
        if ((threadIdx.x & 31) == 0) record_status(s.status, kStatusSeqlenRange);
        n = min(max(n, 0), s.L);
    }
    return n;
}

// Keys that row i of sample z (n tokens) sees; (0, 0) when there are none.
__device__ __forceinline__ int2 row_span(const SpanSource &s, int z, int i, int n) {
    if (i >= n) return make_int2(0, 0);
    int2 r = make_int2(0, n);
    if (s.spans != nullptr) {
        r = s.spans[static_cast<size_t>(z) * s.L + i];
        r.x = max(r.x, 0);
        r.y = min(r.y, n);
    }
    return r.x < r.y ? r : make_int2(0, 0);
}

// Bits [a, b) of a 32-bit word, for any a, b.
__device__ __forceinline__ uint32_t bit_range(int a, int b) {
    const uint32_t below_b = b >= 32 ? 0xffffffffu : (b <= 0 ? 0u : (1u << b) - 1u);
    const uint32_t below_a = a >= 32 ? 0xffffffffu : (a <= 0 ? 0u : (1u << a) - 1u);
    return below_b & ~below_a;
}

// Keeps the packed bf16 pairs (columns 2 i, 2 i + 1) whose bit is set.
template <int N>
__device__ __forceinline__ void keep_bits(uint32_t (&pk)[N], uint32_t bits) {
    static_assert(N <= 16, "one word of bits");
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t lo = (bits >> (2 * i)) & 1u ? 0x0000FFFFu : 0u;
        const uint32_t hi = (bits >> (2 * i + 1)) & 1u ? 0xFFFF0000u : 0u;
        pk[i] &= lo | hi;
    }
}

// Zeroes rows [r0, 128) of a [128][64 NSUB] bf16 operand tile in shared memory
// (a row is 128 contiguous bytes of each 64-column atom; the swizzle permutes
// chunks inside them), by one warp, and makes the zeros visible to the MMA.
// Rows of padding are multiplied by weights of exactly zero; NaN or infinities
// in them would still spoil the product.
template <int NSUB>
__device__ __forceinline__ void zero_tile_rows(uint8_t *tile, int r0) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int s = 0; s < NSUB; ++s) {
        uint4 *rows = reinterpret_cast<uint4 *>(tile + s * (128 * 64 * 2));
        for (int e = r0 * 8 + lane; e < 128 * 8; e += 32) rows[e] = make_uint4(0u, 0u, 0u, 0u);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}

}  // namespace sigattn
