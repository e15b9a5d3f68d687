// dx = (dy W) * f'(z): dy K-major, W with the summed axis outermost.
#include "gemm_tc.cuh"

namespace tide {

cudaError_t launch_grad_input(const TcArgs& p, TcTile t, int grid, bool after, cudaStream_t stream) {
  return launch_layout<false, true, EPI_GRAD_INPUT>(p, t, grid, after, stream);
}

}  // namespace tide
