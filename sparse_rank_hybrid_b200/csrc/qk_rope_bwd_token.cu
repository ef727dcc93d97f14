// The backward kernels of qk_rope.cuh with a norm over a token's heads.
#include "qk_rope.cuh"

namespace slra {

cudaError_t launch_qk_rope_bwd_token(const QkRopeArgs& a, const RowPlan& p, cudaStream_t st) {
    return rope_launch_all<true, kQkNormToken, true>(a, p, st);
}

}  // namespace slra
