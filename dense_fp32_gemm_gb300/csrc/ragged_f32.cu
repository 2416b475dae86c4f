// ragged_f32.cu -- ragged_kernel on FP32 operands (three BF16 parts each).
#include "ragged_launch.cuh"

namespace sgemm_gb300 {
namespace ragged {

cudaError_t launch_f32(int dev, int bq, int grid, const Params& p, const CUtensorMap& mp,
                       const CUtensorMap& mq, cudaStream_t stream) {
  switch (bq) {
    case 32: return launch_one<kF32, 32>(dev, grid, p, mp, mq, stream);
    case 64: return launch_one<kF32, 64>(dev, grid, p, mp, mq, stream);
    case 128: return launch_one<kF32, 128>(dev, grid, p, mp, mq, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace ragged
}  // namespace sgemm_gb300
