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

// 16 values of a row as they are stored: from a 16-byte aligned address (V) or
// any; what lies past the row's end reads as zeros.
template <typename E>
struct Raw {
  uint4 v[sizeof(E)];
};
template <typename E, bool V>
__device__ __forceinline__ Raw<E> load_16(const E* x, int n) {
  Raw<E> r;
  if (V && n >= 16) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(E); ++i) r.v[i] = __ldg(reinterpret_cast<const uint4*>(x) + i);
  } else {
    E* e = reinterpret_cast<E*>(r.v);
#pragma unroll
    for (int i = 0; i < 16; ++i) e[i] = i < n ? x[i] : (E)0.f;
  }
  return r;
}
template <typename E>
__device__ __forceinline__ float value(const Raw<E>& r, int i) {
  return to_f32(reinterpret_cast<const E*>(r.v)[i]);
}

// The largest magnitude, as bits: a NaN is above infinity, so either survives.
template <typename E>
__device__ __forceinline__ uint32_t magnitude(const Raw<E>& r, uint32_t most) {
#pragma unroll
  for (int i = 0; i < 16; ++i) most = max(most, __float_as_uint(value(r, i)) & 0x7FFFFFFFu);
  return most;
}

// rint(x / s), the quotient rounded to FP32 first, in [-127, 127]; 0 for a NaN.
__device__ __forceinline__ uint32_t quotient(float x, float s) {
  const float d = __fdiv_rn(x, s);
  return d == d ? (uint32_t)__float2int_rn(fminf(fmaxf(d, -127.f), 127.f)) : 0u;
}

// The quotients of 16 values (r, also at x in memory), written to q (n of them).
// x * inv, inv = 1 / s, is within 2^-22 of the quotient (relative; |x / s| <=
// 127), so the two round to the same integer unless the product lies that near
// to the middle of two. Adding 1.5 * 2^23 rounds to the nearest integer, ties
// to even, and leaves it in the sum's low byte. Where one of the 16 lies near a
// middle (or 1 / s is no number to multiply by), all are divided.
template <typename E>
__device__ __forceinline__ void put_16(const Raw<E>& r, const E* x, float s, float inv,
                                       signed char* q, int n) {
  constexpr float kMagic = 12582912.f;
  if (!(s > 0.f)) {     // a row of zeros, or a NaN scale
    for (int i = 0; i < min(n, 16); ++i) q[i] = 0;
    return;
  }
  uint32_t w[4];
  bool near = !(inv < 1e37f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = value(r, 4 * i + j) * inv, t = v + kMagic;
      // (also for no number)
      near = near || !(fabsf(v - (t - kMagic)) <= 0.5f - 1e-4f);
      b[j] = __float_as_uint(t);
    }
    w[i] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  }
  if (near) {
#pragma unroll 1
    for (int i = 0; i < min(n, 16); ++i) q[i] = (signed char)quotient(to_f32(x[i]), s);
    return;
  }
  if (n >= 16 && (reinterpret_cast<uintptr_t>(q) & 15u) == 0) {
    *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) q[i] = (signed char)(w[i >> 2] >> (8 * (i & 3)));
  }
}

// A row per block. Of a row up to kHeld groups of 16 values a thread stay in
// registers between the two passes (the maximum, the quotients); the rest of a
// longer row is read again. A call has to read X and write Q once: 50 MB for
// 4096 x 4096 BF16 values, 18 us under the profiler (14 instructions a value, a
// third of the issue slots; the row's chain of load, maximum and store is the
// rest). Fewer registers a thread for more rows in flight spill: 22.2 against
// 23.8 us for 133 x 1000 with its product. A row per warp took 37 us.
constexpr int kHeld = 2;
template <typename E, bool V>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(int M, int K, const E* __restrict__ X, long long ldx,
                    signed char* __restrict__ Q, long long ldq, float* __restrict__ scale) {
  __shared__ uint32_t warp_max[kThreads / 32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int step = 16 * blockDim.x, k0 = 16 * threadIdx.x;
  // (row numbers and places in a row pass 32 bits before they end their loops)
  for (long long m = blockIdx.x; m < M; m += gridDim.x) {
    const E* x = X + m * ldx;
    uint32_t most = 0;
    Raw<E> h[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) h[i] = load_16<E, V>(x + k0 + i * step, K - k0 - i * step);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) most = magnitude(h[i], most);
    for (long long k = k0 + kHeld * step; k < K; k += step)
      most = magnitude(load_16<E, V>(x + k, (int)(K - k)), most);
    most = __reduce_max_sync(0xffffffffu, most);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = most;
    __syncthreads();
    for (int w = 0; w < (int)blockDim.x / 32; ++w) most = max(most, warp_max[w]);
    const float s = __fdiv_rn(__uint_as_float(most), 127.f);
    if (threadIdx.x == 0) scale[m] = s;
    const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
    signed char* q = Q + m * ldq;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (k0 + i * step < K)
        put_16(h[i], x + k0 + i * step, s, inv, q + k0 + i * step, K - k0 - i * step);
    for (long long k = k0 + kHeld * step; k < K; k += step)
      put_16(load_16<E, V>(x + k, (int)(K - k)), x + k, s, inv, q + k, (int)(K - k));
  }
}

template <typename E>
cudaError_t quantize(int M, int K, const void* X, int ldx, signed char* Q, int ldq, float* scale,
                     int sms, cudaStream_t stream) {
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  // Few rows: as many threads as the row has groups, for its latency. Rows that
  // fill the SMs: half as many, so that twice the rows are in flight (a row is
  // a chain of a load, a block-wide maximum and a store).
  const int groups = K / 16 + (K % 16 != 0), want = M < 4 * sms ? groups : (groups + 1) / 2;
  int threads = want < 32 ? 32 : (want + 31) / 32 * 32;
  if (threads > kThreads) threads = kThreads;
  const int fit = sms * (2048 / threads < 32 ? 2048 / threads : 32);
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
