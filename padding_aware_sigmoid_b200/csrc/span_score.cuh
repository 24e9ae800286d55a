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

// SCORE: which terms a kernel instance evaluates.  kScoreFar goes with a cap above
// kCapFar, in the EXP form only (cap_tanh2).
enum ScoreTerms : int { kScoreCap = 1, kScoreSlope = 2, kScoreFar = 4 };
constexpr float kCapFar = 64.0f;
inline int score_terms(float cap, const float *slopes) {
    return (cap > 0.0f ? kScoreCap : 0) | (cap > kCapFar ? kScoreFar : 0) | (slopes != nullptr ? kScoreSlope : 0);
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Coefficients of one (sample, head); arguments are kept times log2 e, as ex2
// wants them.
struct ScoreCoef {
    float a;    // on the raw product: alpha log2 e, or alpha / cap with a cap
    float c;    // b log2 e
    float cap;  // cap log2 e
    float m;    // -m_h log2 e
    // the cap as a polynomial of the raw product s (see cap_poly2)
    float k0, k1, k2;
    int most;   // s^2 up to which it holds, as bits
};
// tanh(y) / y as a0 + a1 y^2 + a2 y^4 on |y| <= 3/4: minimax fit in relative error,
// fitted for this library by iteratively reweighted least squares (maximum 2.2e-4;
// the hardware tanh has 4.9e-4).
constexpr float kCapA0 = 0.9997852f, kCapA1 = -0.32629665f, kCapA2 = 0.09735532f, kCapMost = 0.75f;

template <int SCORE>
__device__ __forceinline__ ScoreCoef make_score(float alpha, float bias, float cap, float slope) {
    ScoreCoef r;
    r.a = SCORE & kScoreCap ? alpha / cap : kLog2e * alpha;
    r.c = kLog2e * bias;
    r.cap = kLog2e * cap;
    r.m = -kLog2e * slope;
    r.k0 = r.k1 = r.k2 = 0.0f;
    r.most = 0;
    if constexpr (SCORE & kScoreCap) {
        const float a2 = r.a * r.a, k = kLog2e * alpha, most = kCapMost / r.a;
        r.k0 = k * kCapA0;
        r.k1 = k * kCapA1 * a2;
        r.k2 = k * kCapA2 * a2 * a2;
        r.most = __float_as_int(most * most);
    }
    return r;
}

// Additive part of the arguments of two neighbouring columns; `rel` is this
// row's position less the first column's.  (A second copy of the loops with the
// straight line that |i - j| is away from the diagonal, one FMA in place of five
// operations, ran 3 to 9% slower in five of six cases.)
template <int SCORE>
__device__ __forceinline__ float2 score_addend(const ScoreCoef &cf, float rel) {
    if constexpr (SCORE & kScoreSlope)
        return fma2(f2(fabsf(rel), fabsf(rel - 1.0f)), f2(cf.m, cf.m), f2(cf.c, cf.c));
    else
        return f2(cf.c, cf.c);
}

// tanh of two capped scores, and 1 - tanh^2.  TANH mode takes the hardware
// tanh (relative error 2^-11, so the capped score moves by at most 2^-11 of
// itself).  EXP mode forms (1 - e) / (1 + e) with e = exp(-2 |y|), and 4 e / (1 +
// e)^2, in which nothing cancels.  Below |y| = 1/4 the former does: an absolute error
// of about 2^-21, which the cap multiplies: a score is off by 2^-15 at kCapFar.  FAR, above
// that, takes tanh(y) / y there as a polynomial in y^2 (minimax fit in relative error,
// fitted for this library as the one above, maximum 4e-7).  Either side is then within
// 2^-20 of tanh, relatively, and so is a capped score, whatever the cap.  For every cap
// that would be 9 to 15% of the EXP mode's time (cap 30, forward of 2 x 4001, 16 over 4
// heads, D = 128: 275 -> 314 us, backward 695 -> 799; D = 64, full 4K forward 405 -> 441) and 3 to
// 5% of the paged attention's (32 x 4 drafts 53.6 -> 55.6).
constexpr float kTanh0 = 0.999999583f, kTanh1 = -0.333219081f, kTanh2 = 0.128416136f, kTanhMost = 0.25f;
template <int MODE, bool GRAD, bool FAR>
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
        if constexpr (!FAR) return f2(copysignf(t.x, y.x), copysignf(t.y, y.y));
        const float2 z = mul2(y, y);
        const float2 n = mul2(y, fma2(z, fma2(z, f2(kTanh2, kTanh2), f2(kTanh1, kTanh1)), f2(kTanh0, kTanh0)));
        return f2(fabsf(y.x) < kTanhMost ? n.x : copysignf(t.x, y.x), fabsf(y.y) < kTanhMost ? n.y : copysignf(t.y, y.y));
    }
}

// x log2 e of two neighbouring columns from their raw products and the additive
// part; with GRAD and a cap also the cap's derivative.
template <int MODE, int SCORE, bool GRAD>
__device__ __forceinline__ float2 score_arg2(float s0, float s1, const ScoreCoef &cf, float2 add, float2 &f) {
    if constexpr (SCORE & kScoreCap) {
        const float2 t = cap_tanh2<MODE, GRAD, (SCORE & kScoreFar) != 0>(mul2(f2(s0, s1), f2(cf.a, cf.a)), f);
        return fma2(t, f2(cf.cap, cf.cap), add);
    } else {
        return fma2(f2(s0, s1), f2(cf.a, cf.a), add);
    }
}

// The same with the cap as a polynomial: four FMA operations more than without a
// cap, where a tanh doubles the MUFU's work.
//   q = k alpha (a0 + a1 (a s)^2 + a2 (a s)^4),  x = s q + ..
__device__ __forceinline__ float2 cap_poly2(float s0, float s1, const ScoreCoef &cf, float2 add, int &largest) {
    const float2 s = f2(s0, s1), z = mul2(s, s);
    largest = __vimax3_s32(largest, __float_as_int(z.x), __float_as_int(z.y));
    const float2 q = fma2(z, fma2(z, f2(cf.k2, cf.k2), f2(cf.k1, cf.k1)), f2(cf.k0, cf.k0));
    return fma2(s, q, add);
}

// How the chunks of a warp are evaluated in TANH mode: counts of chunks that skip a
// form which did not fit before.
struct ScorePause {
    int tail, poly;
};
constexpr int kPause = 31, kNever = 1 << 30;
constexpr int kTailMost = 0x3D000000;    // u = 1/32 as bits
constexpr float kTailBias = -11.5f;      // b log2 e: rows of about 2900 tokens
__device__ __forceinline__ ScorePause score_pause(const ScoreCoef &cf) {
    // the polynomial's coefficients stay in range for any sane alpha / cap
    return ScorePause{cf.c <= kTailBias ? 0 : kNever, fabsf(cf.a) < 1e4f ? 0 : kNever};
}

// P (packed bf16) of 32 neighbouring columns of this thread's row, and with GRAD g
// = dP/d(alpha s), in TANH mode with the forms POLY (of the cap) and TAIL (of
// sigma); returns whether both hold for all 32 x 32 scores of the warp (bit 0: the
// cap's does not, bit 1: the tail's).  A lane whose row is not there (`live`) has no
// say.
//
// TAIL: in the left tail, u = e^x <= 1/32, p = u - u^2 stands for sigma and p - p^2 for
// sigma' from one ex2: as many MUFU and FMA operations as the tanh form, but a
// relative error of -u^2 (either one; the next term is u^3), at most 1e-3, where 0.5 +
// 0.5 tanh cancels (up to 1.4%).  (u - 2 u^2 for sigma' would have -3 u^2.)
template <int SCORE, bool GRAD, bool POLY, bool TAIL>
__device__ __forceinline__ int score_form(const uint32_t *r, const ScoreCoef &cf, float rel, uint32_t *pk, float2 *g,
                                          bool live) {
    ScoreCoef cx = cf;
    if constexpr (!TAIL) {     // tanh wants x / 2
        constexpr float kHalfLn2 = 0.34657359f;
        if constexpr (!(SCORE & kScoreCap)) cx.a *= kHalfLn2;
        cx.c *= kHalfLn2;
        cx.cap *= kHalfLn2;
        cx.m *= kHalfLn2;
        cx.k0 *= kHalfLn2;
        cx.k1 *= kHalfLn2;
        cx.k2 *= kHalfLn2;
    }
    int largest = 0, top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float s0 = __uint_as_float(r[2 * i]), s1 = __uint_as_float(r[2 * i + 1]);
        const float2 add = score_addend<SCORE>(cx, rel - static_cast<float>(2 * i));
        float2 f, p, y;
        if constexpr (POLY) y = cap_poly2(s0, s1, cx, add, largest);
        else y = score_arg2<kSigmoidTanh, SCORE, GRAD>(s0, s1, cx, add, f);
        if constexpr (TAIL) {
            const float2 u = f2(ex2_approx(y.x), ex2_approx(y.y)), n = f2(-u.x, -u.y);
            top = __vimax3_s32(top, __float_as_int(u.x), __float_as_int(u.y));
            p = fma2(n, u, u);
            if constexpr (GRAD) g[i] = fma2(f2(-p.x, -p.y), p, p);
        } else if constexpr (GRAD) {
            sigma_grad2<kSigmoidTanh>(y, p, g[i]);
        } else {
            p = sigma2<kSigmoidTanh>(y);
        }
        if constexpr (GRAD && (SCORE & kScoreCap)) g[i] = mul2(g[i], f);
        pk[i] = pack_bf16x2(p.x, p.y);
    }
    int bad = 0;
    if constexpr (POLY) bad |= __any_sync(0xffffffffu, live && largest > cf.most) ? 1 : 0;
    if constexpr (TAIL) bad |= __any_sync(0xffffffffu, live && top > kTailMost) ? 2 : 0;
    return bad;
}

// P (packed bf16) of 32 neighbouring columns of this thread's row, and with GRAD g
// = dP/d(alpha s); `rel` is the row's position less the first column's.
//
// In TANH mode a chunk is tried with the forms that usually hold and looked at
// afterwards (the largest s^2 and u, as integers, which order like positive
// floats); where one does not hold, the chunk is done again without it, and the
// next kPause chunks of the warp skip it, so that rows of large scores do not pay
// twice.  Chunks of which some pair is masked (not `whole`) are not tried: what a masked
// key or a row of padding holds must not choose the form, and with it the last bits,
// of the pairs that count.
//
// The tail form is for b = -ln n of long rows, where nearly every chunk fits:
// 2-norm error of O 3.3e-3 -> 2.3e-3 at n = 16384 (at n = 2048 the tanh alone has
// 2.4e-3: biases above kTailBias do not try), for 5% of the time (causal forward, H =
// 16, L = 16384, D = 128: 1003 us with the tanh alone, 1054 us so; with a degree-2
// polynomial and a look at the arguments first 1178 us).  Chunks that hold a
// larger weight keep the tanh: there the weights that cancel are the small ones.
//
// FWD: the cap as a polynomial, in the forward and without slopes (D = 64, full 4K:
// 280 -> 222 us).  With slopes it gained nothing (D = 128 193 -> 194 us, D = 64 packed 56 ->
// 62 us), though no pipe is full there (with the tanh, D = 128: MUFU 71%, FMA 24%, ALU
// 17%, issue 40%): a warp's load of scores, its arithmetic and its store follow one
// another, and more instructions make that chain longer.  The backward's registers do
// not hold its operands (D = 128 547 -> 663 us).
//
// P, and in the backward dS, is rounded to bf16, half a step of 2^-8 at most: the type
// of the tensor pipe's operands.  It is the larger part of a bf16 result's error (2-norm
// of O, dQ, dK, dV 2.35e-3 of the definition's in 64 bits, 1.66e-3 with P in 32 bits
// and one rounding at the end), as in the padding-only kernels.  A second bf16 part
// would double the products that are the bound at D = 128; the paged tile kernel, whose
// few rows leave them room, keeps two.
template <int MODE, int SCORE, bool GRAD, bool FWD = false>
__device__ __forceinline__ void score_chunk(const uint32_t *r, const ScoreCoef &cf, float rel, uint32_t *pk,
                                            float2 *g, ScorePause &pause, bool whole, bool live = true) {
    if constexpr (MODE == kSigmoidExp) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float2 p, f;
            const float2 y =
                score_arg2<MODE, SCORE, GRAD>(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]), cf,
                                              score_addend<SCORE>(cf, rel - static_cast<float>(2 * i)), f);
            if constexpr (GRAD) {
                sigma_grad2<MODE>(y, p, g[i]);
                if constexpr (SCORE & kScoreCap) g[i] = mul2(g[i], f);
            } else {
                p = sigma2<MODE>(y);
            }
            pk[i] = pack_bf16x2(p.x, p.y);
        }
    } else if constexpr (FWD && SCORE == kScoreCap) {
        if (whole && pause.poly == 0) {
            int bad = 2;
            if (pause.tail == 0) {
                if ((bad = score_form<SCORE, GRAD, true, true>(r, cf, rel, pk, g, live)) == 0) return;
                pause.tail = kPause + 1;
            }
            --pause.tail;
            if (!(bad & 1) && score_form<SCORE, GRAD, true, false>(r, cf, rel, pk, g, live) == 0) return;
            pause.poly = kPause + 1;
        }
        pause.poly = max(pause.poly - 1, 0);
        score_form<SCORE, GRAD, false, false>(r, cf, rel, pk, g, live);
    } else {
        if (whole && pause.tail == 0) {
            if (score_form<SCORE, GRAD, false, true>(r, cf, rel, pk, g, live) == 0) return;
            pause.tail = kPause + 1;
        }
        pause.tail = max(pause.tail - 1, 0);
        score_form<SCORE, GRAD, false, false>(r, cf, rel, pk, g, live);
    }
}
// P of two neighbouring columns, for kernels whose scores are few: one ex2 and one
// reciprocal, e^-|x| keeping both tails.  Relative error about 2^-20, and what the
// argument's own error moves: 2^-23 of x without a cap, that of cap_tanh2 with one.
template <int SCORE>
__device__ __forceinline__ float2 score_p2(float s0, float s1, const ScoreCoef &cf, float rel) {
    float2 f;
    const float2 y = score_arg2<kSigmoidExp, SCORE, false>(
        s0, s1, cf, score_addend<SCORE>(cf, rel), f);
    const float2 u = f2(ex2_approx(-fabsf(y.x)), ex2_approx(-fabsf(y.y)));
    const float2 g = f2(rcp_approx(1.0f + u.x), rcp_approx(1.0f + u.y));
    return mul2(g, f2(y.x >= 0.0f ? 1.0f : u.x, y.y >= 0.0f ? 1.0f : u.y));
}

// Lets the next kernel of the stream start, and waits until the one before has
// finished (both do nothing where the launch did not ask for it).
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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

// The sample of grid position r: samples start by decreasing length (ranks_before,
// up to kMaxRankedSamples of them; above that in index order).  Every warp finds it
// by itself.
__device__ __forceinline__ int span_sample(const int *seqlens, int Z, int r) {
    if (Z > kMaxRankedSamples || Z == 1) return r;
    const int lane = threadIdx.x & 31;
    int w[2], rank[2] = {0, 0};
#pragma unroll
    for (int c = 0; c < 2; ++c) w[c] = lane + 32 * c < Z ? seqlens[lane + 32 * c] : 0;
    for (int j = 0; j < Z; ++j) {
        const int wj = __shfl_sync(0xffffffffu, j < 32 ? w[0] : w[1], j & 31);
#pragma unroll
        for (int c = 0; c < 2; ++c) rank[c] += ranks_before(wj, j, w[c], lane + 32 * c);
    }
    const unsigned a = __ballot_sync(0xffffffffu, lane < Z && rank[0] == r);
    const unsigned b = __ballot_sync(0xffffffffu, lane + 32 < Z && rank[1] == r);
    return a != 0 ? __ffs(a) - 1 : 31 + __ffs(b);
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

// Keeps the packed bf16 pairs (columns 2 i, 2 i + 1) whose bit is set.  Bit k of
// the word is the sign bit of a byte of bits << (7 - k % 8), and PRMT can spread
// the sign of a byte: one PRMT makes a pair's mask out of two of the eight
// shifted words, 39 instructions a chunk where selects by bit take about 110.
__device__ __forceinline__ void keep_bits(uint32_t (&pk)[16], uint32_t bits) {
    uint32_t t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = bits << k;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int byte = i / 4, k = (2 * i) % 8;
        // low half: sign of `byte` of the first word, high half: of the second
        const uint32_t sel = (8u | byte) * 0x11u | (8u | 4u | byte) * 0x1100u;
        uint32_t m;
        asm("prmt.b32 %0, %1, %2, %3;" : "=r"(m) : "r"(t[7 - k]), "r"(t[6 - k]), "r"(sel));
        pk[i] &= m;
    }
}

// Bit i of lane j's word against bit j of lane i's: the 32 x 32 bits of a warp
// transposed.
__device__ __forceinline__ uint32_t warp_transpose(uint32_t x) {
    const int lane = threadIdx.x & 31;
    uint32_t m = 0x0000FFFFu;
#pragma unroll
    for (int j = 16; j > 0; j >>= 1, m ^= m << j) {
        const uint32_t y = __shfl_xor_sync(0xffffffffu, x, j);
        x = lane & j ? (x & ~m) | ((y & ~m) >> j) : (x & m) | ((y & m) << j);
    }
    return x;
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
