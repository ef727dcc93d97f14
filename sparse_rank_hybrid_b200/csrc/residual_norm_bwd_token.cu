// Gated residual and modulated norm: backward, a modulation row for each row (residual_norm.cuh).
#include "residual_norm.cuh"

namespace slra {

cudaError_t launch_residual_norm_bwd_token(const ResidualNormArgs& a, const RowPlan& p, cudaStream_t st) {
    return launch_rows<true, true>(a, p, st);
}

}  // namespace slra
