// Gated residual and modulated norm: backward, a modulation row for several rows (residual_norm.cuh).
#include "residual_norm.cuh"

namespace slra {

cudaError_t launch_residual_norm_bwd(const ResidualNormArgs& a, const RowPlan& p, cudaStream_t st) {
    return launch_rows<true, false>(a, p, st);
}

}  // namespace slra
