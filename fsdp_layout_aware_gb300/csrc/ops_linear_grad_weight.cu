// dW = dy^T X: the summed axis (tokens) outermost in both.
#include "gemm_tc.cuh"

namespace tide {

cudaError_t launch_grad_weight(const TcArgs& p, TcTile t, int grid, bool after, cudaStream_t stream) {
  return launch_layout<true, true, EPI_PLAIN>(p, t, grid, after, stream);
}

}  // namespace tide
