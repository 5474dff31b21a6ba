// flce_norm_fp8_left.cu — the norm's forward with an 8-bit output, where products
// of h and the weights are rounded and what that leaves is carried along.
#include "flce_norm_fwd.cuh"

namespace flce {

cudaError_t launch_norm_fwd_fp8_left(const NormParams& p, int32_t dt, int32_t rdt, const RowPlan& pl, int grid,
                                     cudaStream_t st) {
  return launch_fwd_any<kFp8Left>(p, dt, rdt, pl, grid, st);
}

}  // namespace flce
