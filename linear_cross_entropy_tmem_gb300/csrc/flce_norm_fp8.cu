// flce_norm_fp8.cu — the norm's forward with an 8-bit output, where products of
// h and the weights are exact.
#include "flce_norm_fwd.cuh"

namespace flce {

cudaError_t launch_norm_fwd_fp8_exact(const NormParams& p, int32_t dt, int32_t rdt, const RowPlan& pl, int grid,
                                      cudaStream_t st) {
  return launch_fwd_any<kFp8Exact>(p, dt, rdt, pl, grid, st);
}

}  // namespace flce
