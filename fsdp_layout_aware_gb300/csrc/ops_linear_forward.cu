// y = f(x W^T + b) + r: both operands K-major.
#include "gemm_tc.cuh"

namespace tide {

cudaError_t launch_forward(const TcArgs& p, TcTile t, int grid, bool after, cudaStream_t stream) {
  return launch_layout<false, false, EPI_FORWARD>(p, t, grid, after, stream);
}

}  // namespace tide
