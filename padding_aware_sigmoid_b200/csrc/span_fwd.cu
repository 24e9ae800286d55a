#include "span_launch.cuh"

namespace sigattn {

sigattn_status launch_span_fwd(const SpanKind &kind, dim3 grid, const CUtensorMap &mq, const CUtensorMap &mk,
                               const CUtensorMap &mv, const SpanFwdParams &p, cudaStream_t st) {
    return with_kind(kind, [&]<int D, int MODE, int SCORE>() {
        constexpr int kSmem = SpanFwdLayout<D>::SMEM_ALLOC;
        auto run = [&](auto kernel) {
            return launch_with(kernel, grid, dim3(SpanTiles<D>::kThreads), kSmem, kSmem, false, p.split, st, mq, mk, mv, p);
        };
        return p.split > 1 ? run(span_fwd_kernel<D, MODE, SCORE, true>) : run(span_fwd_kernel<D, MODE, SCORE, false>);
    });
}

}  // namespace sigattn
