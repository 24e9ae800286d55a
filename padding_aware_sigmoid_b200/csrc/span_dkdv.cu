#include "span_launch.cuh"

namespace sigattn {

sigattn_status launch_span_dkdv(const SpanKind &kind, dim3 grid, const CUtensorMap &mq, const CUtensorMap &mk,
                               const CUtensorMap &mv, const CUtensorMap &mdo, const SpanBwdParams &p, cudaStream_t st) {
    return with_kind(kind, [&]<int D, int MODE, int SCORE>() {
        constexpr int kSmem = SpanBwdLayout<D, false>::SMEM_ALLOC;
        return launch_with(span_dkdv_kernel<D, MODE, SCORE>, grid, dim3(SpanBwdShape<D, false>::kThreads), kSmem, kSmem, true, st, mq, mk, mv, mdo, p);
    });
}

}  // namespace sigattn
