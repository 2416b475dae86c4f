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

// 16 values of a row at a time: from any address (V: 16-byte aligned), and as 8-bit
// integers to any address.
template <typename E, bool V>
__device__ __forceinline__ void load_16(const E* x, int n, float (&v)[16]) {
  if (V && n >= 16) {
    constexpr int W = sizeof(E);      // 16-byte vectors of the 16 values
    uint4 raw[W];
#pragma unroll
    for (int i = 0; i < W; ++i) raw[i] = __ldg(reinterpret_cast<const uint4*>(x) + i);
    const E* e = reinterpret_cast<const E*>(raw);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = to_f32(e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = i < n ? to_f32(x[i]) : 0.f;
  }
}

// rint(x / s), the quotient rounded to FP32 first. x * (1 / s) is within 2^-22
// of it (relative), so the two round to the same integer unless the product
// lies that near to the middle of two integers; only then the division runs.
__device__ __forceinline__ int quotient(float x, float s, float inv) {
  float v = x * inv;
  const float r = rintf(v);
  if (!(fabsf(fabsf(v - r) - 0.5f) >= 1e-4f) || !(inv < 1e37f)) {   // (or no number)
    v = __fdiv_rn(x, s);
    if (!(v == v)) return 0;
    return __float2int_rn(fminf(fmaxf(v, -127.f), 127.f));
  }
  return __float2int_rn(fminf(fmaxf(r, -127.f), 127.f));
}

template <typename E, bool V>
__device__ __forceinline__ uint32_t magnitude(const float (&v)[16], uint32_t most) {
#pragma unroll
  for (int i = 0; i < 16; ++i) most = max(most, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return most;
}

// One row per block of `threads` = blockDim.x. Up to 16 * kHeld values a thread
// stay in registers between the two passes (the maximum, the quotients); of a
// longer row the rest is read again. One read of X and one write of Q are all
// that a call has to move: at 4096 x 4096 bf16 it is bound by them.
template <typename E, bool V>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(int M, int K, const E* __restrict__ X, long long ldx,
                    signed char* __restrict__ Q, long long ldq, float* __restrict__ scale) {
  __shared__ uint32_t warp_max[kThreads / 32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int step = 16 * blockDim.x, k0 = 16 * threadIdx.x;
  constexpr int kHeld = 2;
  for (int m = blockIdx.x; m < M; m += gridDim.x) {
    const E* x = X + m * ldx;
    // magnitudes compared as bit patterns: a NaN is above infinity, so either
    // survives the maximum
    uint32_t most = 0;
    float held[kHeld][16];
#pragma unroll
    for (int h = 0; h < kHeld; ++h) load_16<E, V>(x + k0 + h * step, K - k0 - h * step, held[h]);
#pragma unroll
    for (int h = 0; h < kHeld; ++h) most = magnitude<E, V>(held[h], most);
    for (int k = k0 + kHeld * step; k < K; k += step) {
      float v[16];
      load_16<E, V>(x + k, K - k, v);
      most = magnitude<E, V>(v, most);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = most;
    __syncthreads();
    for (int w = 0; w < (int)blockDim.x / 32; ++w) most = max(most, warp_max[w]);
    const float s = __fdiv_rn(__uint_as_float(most), 127.f);
    if (threadIdx.x == 0) scale[m] = s;
    const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
    auto put = [&](const float (&v)[16], int k) {
      const int n = K - k;
      uint32_t w[4] = {0u, 0u, 0u, 0u};
      if (s > 0.f) {     // (a NaN scale: zeros)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w[i >> 2] |= (uint32_t)(quotient(v[i], s, inv) & 255) << (8 * (i & 3));
      }
      signed char* q = Q + m * ldq + k;
      if (n >= 16 && (reinterpret_cast<uintptr_t>(q) & 15u) == 0) {
        *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i < n) q[i] = (signed char)(w[i >> 2] >> (8 * (i & 3)));
      }
    };
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
      if (k0 + h * step < K) put(held[h], k0 + h * step);
    for (int k = k0 + kHeld * step; k < K; k += step) {
      float v[16];
      load_16<E, V>(x + k, K - k, v);
      put(v, k);
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
  // as many threads as the row has 16-value pieces: short rows take few
  int threads = (K + 15) / 16;
  threads = threads < 32 ? 32 : (threads + 31) / 32 * 32;
  if (threads > kThreads) threads = kThreads;
  const int fit = sms * (2048 / kThreads) * (kThreads / threads);
  lc.gridDim = dim3((unsigned)(M < fit ? M : fit));
  lc.blockDim = dim3((unsigned)threads);
  lc.stream = stream;
  lc.attrs = la;
  lc.numAttrs = 1;
  const bool aligned = (reinterpret_cast<uintptr_t>(X) & 15u) == 0 &&
                       ((long long)ldx * (int)sizeof(E)) % 16 == 0;
  return cudaLaunchKernelEx(&lc, aligned ? quantize_kernel<E, true> : quantize_kernel<E, false>, M,
                            K, static_cast<const E*>(X), (long long)ldx, Q, (long long)ldq, scale);
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
