// i8_quantize.cu -- sgemm_i8_quantize: rows of a matrix to 8-bit integers with
// one scale a row.
//
// scale = amax / 127, q = rint(x / scale) in [-127, 127], both quotients
// rounded to nearest FP32 (so q is a defined integer, ties to even). A row of
// zeros has scale 0 and q 0; a row that holds an infinity or a NaN has that
// for its scale, so the products of the row come out as NaN, never as
// plausible numbers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/sgemm_gb300.h"
#include "ptx.cuh"

#define SGEMM_API extern "C" __attribute__((visibility("default")))

namespace sgemm_gb300 {

int library_device_sms(int dev, int* sms);

namespace {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

constexpr int kThreads = 256;

template <typename E>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(int M, int K, const E* __restrict__ X, long long ldx,
                    signed char* __restrict__ Q, long long ldq, float* __restrict__ scale) {
  __shared__ uint32_t warp_max[kThreads / 32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  for (int m = blockIdx.x; m < M; m += gridDim.x) {
    const E* x = X + m * ldx;
    // magnitudes compared as bit patterns: a NaN is above infinity, so either
    // survives the maximum
    uint32_t most = 0;
    for (int k = threadIdx.x; k < K; k += kThreads)
      most = max(most, __float_as_uint(to_f32(x[k])) & 0x7FFFFFFFu);
    most = __reduce_max_sync(0xffffffffu, most);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) most = max(most, warp_max[w]);
    const float s = __fdiv_rn(__uint_as_float(most), 127.f);
    if (threadIdx.x == 0) scale[m] = s;
    for (int k = threadIdx.x; k < K; k += kThreads) {
      const float v = s > 0.f ? __fdiv_rn(to_f32(x[k]), s) : 0.f;   // (NaN scale: 0)
      const int q = __float2int_rn(fminf(fmaxf(v, -127.f), 127.f));
      Q[m * ldq + k] = (signed char)(v == v ? q : 0);
    }
  }
}

template <typename E>
cudaError_t quantize(int M, int K, const void* X, int ldx, signed char* Q, int ldq, float* scale,
                     int sms, cudaStream_t stream) {
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  lc.gridDim = dim3((unsigned)(M < sms * 8 ? M : sms * 8));
  lc.blockDim = dim3(kThreads);
  lc.stream = stream;
  lc.attrs = la;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, quantize_kernel<E>, M, K, static_cast<const E*>(X),
                            (long long)ldx, Q, (long long)ldq, scale);
}

}  // namespace
}  // namespace sgemm_gb300

using namespace sgemm_gb300;

SGEMM_API int sgemm_i8_quantize(int M, int K, int type, const void* X, int ldx, signed char* Q,
                                int ldq, float* scale, void* stream_) {
  if (type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16 && type != SGEMM_TYPE_F16)
    return SGEMM_ERR_INVALID_VALUE;
  if (M < 0 || K < 0) return SGEMM_ERR_INVALID_DIM;
  if (ldx < (K > 1 ? K : 1) || ldq < (K > 1 ? K : 1)) return SGEMM_ERR_INVALID_LD;
  if (M == 0) return SGEMM_OK;
  if (scale == nullptr || (K > 0 && (X == nullptr || Q == nullptr))) return SGEMM_ERR_NULL_PTR;
  const uintptr_t mask = type == SGEMM_TYPE_F32 ? 3u : 1u;
  if ((reinterpret_cast<uintptr_t>(X) & mask) || (reinterpret_cast<uintptr_t>(scale) & 3u))
    return SGEMM_ERR_MISALIGNED;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return SGEMM_ERR_LAUNCH;
  }
  const int st = library_device_sms(dev, &sms);
  if (st != SGEMM_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const cudaError_t e =
      type == SGEMM_TYPE_F32    ? quantize<float>(M, K, X, ldx, Q, ldq, scale, sms, stream)
      : type == SGEMM_TYPE_BF16 ? quantize<__nv_bfloat16>(M, K, X, ldx, Q, ldq, scale, sms, stream)
                                : quantize<__half>(M, K, X, ldx, Q, ldq, scale, sms, stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return SGEMM_ERR_LAUNCH;
  }
  return SGEMM_OK;
}
