#include "span_launch.cuh"

namespace sigattn {

sigattn_status launch_span_fwd(const SpanKind &kind, dim3 grid, const CUtensorMap &mq, const CUtensorMap &mk,
                               const CUtensorMap &mv, const SpanFwdParams &p, cudaStream_t st) {
    return with_kind(kind, [&]<int D, int MODE, int SCORE>() {
        return launch(span_fwd_kernel<D, MODE, SCORE>, grid, dim3(SpanTiles<D>::kThreads), SpanFwdLayout<D>::SMEM_ALLOC, st, mq, mk, mv, p);
    });
}

}  // namespace sigattn
