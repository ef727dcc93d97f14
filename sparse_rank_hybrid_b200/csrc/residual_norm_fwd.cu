// Gated residual and modulated norm: forward, a modulation row for several rows (residual_norm.cuh).
#include "residual_norm.cuh"

namespace slra {

cudaError_t launch_residual_norm_fwd(const ResidualNormArgs& a, const RowPlan& p, cudaStream_t st) {
    return launch_rows<false, false>(a, p, st);
}

}  // namespace slra
