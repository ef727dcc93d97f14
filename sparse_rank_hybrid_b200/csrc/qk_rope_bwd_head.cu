// The backward kernels of qk_rope.cuh with a norm per head.
#include "qk_rope.cuh"

namespace slra {

cudaError_t launch_qk_rope_bwd_head(const QkRopeArgs& a, const RowPlan& p, cudaStream_t st) {
    return rope_launch_all<true, kQkNormHead, true>(a, p, st);
}

}  // namespace slra
