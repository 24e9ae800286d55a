// Launchers of the masked-attention kernels, one file per kernel so that their
// instances (head dimension x sigma form x score terms) compile side by side.
#pragma once

#include "host.cuh"
#include "span_bwd_sm100.cuh"
#include "span_fwd_sm100.cuh"

namespace sigattn {

struct SpanKind {
    int D, mode, score;   // 64 or 128; SigmoidMode; ScoreTerms
};

sigattn_status launch_span_fwd(const SpanKind &kind, dim3 grid, const CUtensorMap &mq, const CUtensorMap &mk,
                               const CUtensorMap &mv, const SpanFwdParams &p, cudaStream_t st);
sigattn_status launch_span_dq(const SpanKind &kind, dim3 grid, const CUtensorMap &mq, const CUtensorMap &mk,
                              const CUtensorMap &mv, const CUtensorMap &mdo, const SpanBwdParams &p,
                              cudaStream_t st);
sigattn_status launch_span_dkdv(const SpanKind &kind, dim3 grid, const CUtensorMap &mq, const CUtensorMap &mk,
                                const CUtensorMap &mv, const CUtensorMap &mdo, const SpanBwdParams &p,
                                cudaStream_t st);

// Calls f.template operator()<D, MODE, SCORE>() for the instance `kind` names.
template <int D, int MODE, typename F>
sigattn_status with_score(int score, F &&f) {
    switch (score) {
        case 0: return f.template operator()<D, MODE, 0>();
        case kScoreCap: return f.template operator()<D, MODE, kScoreCap>();
        case kScoreSlope: return f.template operator()<D, MODE, kScoreSlope>();
        case kScoreCap | kScoreSlope: return f.template operator()<D, MODE, kScoreCap | kScoreSlope>();
    }
    constexpr int kFar = MODE == kSigmoidExp ? kScoreFar : 0;     // the hardware tanh has no such form
    return score & kScoreSlope ? f.template operator()<D, MODE, kScoreCap | kScoreSlope | kFar>()
                               : f.template operator()<D, MODE, kScoreCap | kFar>();
}
template <typename F>
sigattn_status with_kind(const SpanKind &k, F &&f) {
    if (k.D == 64)
        return k.mode == kSigmoidTanh ? with_score<64, kSigmoidTanh>(k.score, f)
                                      : with_score<64, kSigmoidExp>(k.score, f);
    return k.mode == kSigmoidTanh ? with_score<128, kSigmoidTanh>(k.score, f)
                                  : with_score<128, kSigmoidExp>(k.score, f);
}

}  // namespace sigattn
