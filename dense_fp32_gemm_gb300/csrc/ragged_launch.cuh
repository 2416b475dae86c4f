// ragged_launch.cuh -- host side of ragged_kernel shared by its entry points:
// tensor maps, copies of operands that TMA cannot read in place, attributes
// and the launch.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "../../include/sgemm_gb300.h"
#include "ragged_gemm.cuh"

namespace sgemm_gb300 {

// Provided by api.cu.
int library_workspace(int dev, cudaStream_t stream, size_t floats, size_t nflags, float** scratch,
                      int** status, uint32_t** flags, uint32_t* epoch);
int library_device_sms(int dev, int* sms);
void note_last_config(const char* text);
long long library_wait_timeout_ns();

namespace ragged {

// A stored operand: `batch` matrices of rows x cols elements (cols is the
// unit-stride dimension), pitch ld, `stride` between matrices.
struct Operand {
  const void* ptr;
  int elem;                 // bytes per element
  long long rows, cols, ld, stride;
  int batch;
  // TMA reads it in place: 16-byte aligned rows and matrices
  bool direct() const {
    return ((reinterpret_cast<uintptr_t>(ptr) & 15u) == 0) && (ld * elem) % 16 == 0 &&
           (batch <= 1 || (stride * elem) % 16 == 0);
  }
  long long packed_ld() const { return (cols * elem + 15) / 16 * 16 / elem; }
  size_t packed_bytes() const {
    return direct() ? 0 : ((size_t)batch * rows * packed_ld() * elem + 255) / 256 * 256;
  }
};

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encode();
// Copies `op` to `dst` with 16-byte aligned rows and describes the copy.
cudaError_t pack_operand(Operand* op, void* dst, int sms, cudaStream_t stream);
// The 3-D map of an operand with boxes of box_rows rows of row_bytes bytes.
bool encode_operand(CUtensorMap* map, const Operand& op, CUtensorMapDataType type, int row_bytes,
                    int box_rows);

// One launch of ragged_kernel<SRC, BQ>; bq must be one of the built widths.
cudaError_t launch_k16(int dev, int bq, int grid, const Params& p, const CUtensorMap& mp,
                       const CUtensorMap& mq, cudaStream_t stream);
cudaError_t launch_f32(int dev, int bq, int grid, const Params& p, const CUtensorMap& mp,
                       const CUtensorMap& mq, cudaStream_t stream);
cudaError_t launch_i8(int dev, int bq, int grid, const Params& p, const CUtensorMap& mp,
                      const CUtensorMap& mq, cudaStream_t stream);

constexpr int kMaxDevices = 64;

template <int SRC, int BQ>
cudaError_t launch_one(int dev, int grid, const Params& p, const CUtensorMap& mp,
                       const CUtensorMap& mq, cudaStream_t stream) {
  static std::mutex mutex;
  static bool ready[kMaxDevices];
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mutex);
    if (!ready[dev]) {
      const cudaError_t e = cudaFuncSetAttribute(
          ragged_kernel<SRC, BQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
      if (e != cudaSuccess) return e;
      ready[dev] = true;
    }
  }
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  lc.gridDim = dim3((unsigned)grid);
  lc.blockDim = dim3(Geo<SRC, BQ>::kThreads);
  lc.dynamicSmemBytes = kSmemBytes;
  lc.stream = stream;
  lc.attrs = la;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, ragged_kernel<SRC, BQ>, p, mp, mq);
}

}  // namespace ragged
}  // namespace sgemm_gb300
