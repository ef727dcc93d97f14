// The backward kernels of qk_rope.cuh without a norm, not every pair rotated.
#include "qk_rope.cuh"

namespace slra {

cudaError_t launch_qk_rope_bwd_none_some(const QkRopeArgs& a, const RowPlan& p, cudaStream_t st) {
    return rope_launch_all<true, kQkNormNone, false>(a, p, st);
}

}  // namespace slra
