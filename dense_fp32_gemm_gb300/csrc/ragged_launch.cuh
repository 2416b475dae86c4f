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
std::unique_lock<std::mutex> library_lock();
int library_workspace(int dev, cudaStream_t stream, size_t floats, size_t nflags, float** scratch,
                      int** status, uint32_t** flags, uint32_t* epoch, uint32_t** counters);
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
  // The copy's row pitch and size in bytes; `widen`: 8-bit integers as F16
  // (always copied).
  long long packed_pitch(bool widen) const { return (cols * (widen ? 2 : elem) + 15) / 16 * 16; }
  size_t packed_bytes(bool widen) const {
    if (direct() && !widen) return 0;
    return ((size_t)batch * rows * packed_pitch(widen) + 255) / 256 * 256;
  }
};

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encode();
// Copies the operands that have a destination there, with 16-byte aligned rows
// (widen: as F16), in one launch, and describes the copies.
cudaError_t pack_operands(Operand* a, void* dst_a, Operand* b, void* dst_b, bool widen, int sms,
                          cudaStream_t stream);
// The 3-D map of an operand with boxes of box_rows rows of row_bytes bytes.
bool encode_operand(CUtensorMap* map, const Operand& op, CUtensorMapDataType type, int row_bytes,
                    int box_rows);

// A built kernel: source, tile width, CTAs per worker (1, or 2: pairs).
struct Form {
  int src, bq, cl;
};
// One entry of the table of built kernels (a translation unit per source):
// makes the kernel ready on the current device and gives the workers that are
// resident at once (0: pairs cannot run); launches it.
struct FormEntry {
  Form form;
  cudaError_t (*prepare)(int sms, int* workers);
  cudaError_t (*launch)(int workers, const Params& p, const CUtensorMap& mp, const CUtensorMap& mq,
                        cudaStream_t stream);
};
extern const FormEntry kForms16[], kFormsF32[], kFormsI8[];
extern const int kNumForms16, kNumFormsF32, kNumFormsI8;

template <int SRC, int BQ, int CL>
struct FormOf {
  using G = Geo<SRC, BQ, CL>;
  static cudaLaunchConfig_t config(int workers, cudaLaunchAttribute (&la)[2], cudaStream_t stream) {
    la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    la[0].val.programmaticStreamSerializationAllowed = 1;
    la[1].id = cudaLaunchAttributeClusterDimension;
    la[1].val.clusterDim.x = CL;
    la[1].val.clusterDim.y = 1;
    la[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)(workers * CL));
    lc.blockDim = dim3(G::kThreads);
    lc.dynamicSmemBytes = kSmemBytes;
    lc.stream = stream;
    lc.attrs = la;
    lc.numAttrs = CL == 2 ? 2 : 1;
    return lc;
  }
  static cudaError_t prepare(int sms, int* workers) {
    const cudaError_t e = cudaFuncSetAttribute(
        ragged_kernel<SRC, BQ, CL>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    *workers = sms;
    if (e != cudaSuccess || CL == 1) return e;
    // pairs that fit at once (SMs pair up within a GPC, so it can be below sms / 2)
    cudaLaunchAttribute la[2];
    cudaLaunchConfig_t lc = config(sms / 2 > 0 ? sms / 2 : 1, la, nullptr);
    lc.attrs = la + 1;
    lc.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, ragged_kernel<SRC, BQ, CL>, &lc) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    *workers = n;
    return cudaSuccess;
  }
  static cudaError_t launch(int workers, const Params& p, const CUtensorMap& mp,
                            const CUtensorMap& mq, cudaStream_t stream) {
    cudaLaunchAttribute la[2];
    const cudaLaunchConfig_t lc = config(workers, la, stream);
    return cudaLaunchKernelEx(&lc, ragged_kernel<SRC, BQ, CL>, p, mp, mq);
  }
};

#define SGEMM_GB300_FORM(SRC, BQ, CL) \
  { {SRC, BQ, CL}, &FormOf<SRC, BQ, CL>::prepare, &FormOf<SRC, BQ, CL>::launch }

}  // namespace ragged
}  // namespace sgemm_gb300
