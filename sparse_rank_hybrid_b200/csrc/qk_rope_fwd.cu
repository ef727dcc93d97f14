// QK norm and rotary positions: forward (qk_rope.cuh).
#include "qk_rope.cuh"

namespace slra {

cudaError_t launch_qk_rope_fwd(const QkRopeArgs& a, const RowPlan& p, cudaStream_t st) {
    return rope_launch_all<false, -1, true>(a, p, st);
}

}  // namespace slra
