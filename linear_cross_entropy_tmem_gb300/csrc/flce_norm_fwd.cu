// flce_norm_fwd.cu — the norm's forward.
#include "flce_norm_fwd.cuh"

namespace flce {

cudaError_t launch_norm_fwd(const NormParams& p, int32_t dt, int32_t rdt, const RowPlan& pl, int grid, cudaStream_t st) {
  return launch_fwd_any<kSameBits>(p, dt, rdt, pl, grid, st);
}

}  // namespace flce
