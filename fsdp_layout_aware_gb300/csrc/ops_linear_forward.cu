// y = f(x W^T + b) + r: both operands K-major.
#include "gemm_tc.cuh"

namespace tide {

cudaError_t launch_forward(const TcArgs& p, const TcLaunch& l, bool partial, cudaStream_t stream) {
  return launch_layout<false, false, EPI_FORWARD>(p, l, partial, stream);
}

}  // namespace tide
