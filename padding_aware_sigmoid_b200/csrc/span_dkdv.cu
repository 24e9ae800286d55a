#include "span_launch.cuh"

namespace sigattn {

sigattn_status launch_span_dkdv(const SpanKind &kind, dim3 grid, const CUtensorMap &mq, const CUtensorMap &mk,
                               const CUtensorMap &mv, const CUtensorMap &mdo, const SpanBwdParams &p, cudaStream_t st) {
    return with_kind(kind, [&]<int D, int MODE, int SCORE>() {
        constexpr int kSmem = SpanBwdLayout<D, false>::SMEM_ALLOC;
        auto run = [&](auto kernel) {
            return launch_with(kernel, grid, dim3(SpanBwdShape<D, false>::kThreads), kSmem, kSmem, true, p.split, st, mq, mk, mv, mdo, p);
        };
        return p.split > 1 ? run(span_dkdv_kernel<D, MODE, SCORE, true>) : run(span_dkdv_kernel<D, MODE, SCORE, false>);
    });
}

}  // namespace sigattn
