// ragged_k16.cu -- ragged_kernel on BF16 and F16 operands.
#include "ragged_launch.cuh"

namespace sgemm_gb300 {
namespace ragged {

cudaError_t launch_k16(int dev, int bq, int grid, const Params& p, const CUtensorMap& mp,
                       const CUtensorMap& mq, cudaStream_t stream) {
  switch (bq) {
    case 32: return launch_one<k16, 32>(dev, grid, p, mp, mq, stream);
    case 64: return launch_one<k16, 64>(dev, grid, p, mp, mq, stream);
    case 128: return launch_one<k16, 128>(dev, grid, p, mp, mq, stream);
    case 256: return launch_one<k16, 256>(dev, grid, p, mp, mq, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace ragged
}  // namespace sgemm_gb300
