// ragged_i8.cu -- ragged_kernel on 8-bit integer operands.
#include "ragged_launch.cuh"

namespace sgemm_gb300 {
namespace ragged {

cudaError_t launch_i8(int dev, int bq, int grid, const Params& p, const CUtensorMap& mp,
                      const CUtensorMap& mq, cudaStream_t stream) {
  switch (bq) {
    case 32: return launch_one<kI8, 32>(dev, grid, p, mp, mq, stream);
    case 64: return launch_one<kI8, 64>(dev, grid, p, mp, mq, stream);
    case 128: return launch_one<kI8, 128>(dev, grid, p, mp, mq, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace ragged
}  // namespace sgemm_gb300
