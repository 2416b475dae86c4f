// mx4_quantize.cu -- sgemm_mx4_quantize and sgemm_mx4_dequantize: rows of a matrix
// to 4-bit floating point in blocks of 32 values with a power of two each, and
// back.
//
// A block's power is floor(log2(max|x|)) - 2, so that its largest value lies in
// 4 .. 8 units; values are rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6
// units (ties to the even code), beyond 6 to 6. Multiplying by a power of two is
// exact, so the codes are defined bit by bit.
#include <cuda_fp4.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/sgemm_gb300.h"
#include "elements.cuh"
#include "ptx.cuh"

#define SGEMM_API extern "C" __attribute__((visibility("default")))

namespace sgemm_gb300 {

int library_device_sms(int dev, int* sms);

namespace mx4 {
namespace {

using rows::from_f32;
using rows::to_f32;

constexpr int kThreads = 256;
constexpr uint32_t kAll = 0xffffffffu;

// The byte of block b's scale of row m: tiles of 128 rows x 4 blocks, 512 bytes
// each, in a tile 32 lines of the 4 rows r, r + 32, r + 64, r + 96.
__device__ __forceinline__ long long scale_place(long long m, int b, int block_tiles) {
  return ((m >> 7) * block_tiles + (b >> 2)) * 512 + (m & 31) * 16 + ((m >> 5) & 3) * 4 + (b & 3);
}

struct Args {
  int M, K, blocks, block_tiles;
  const void* x;
  long long ldx;
  unsigned char* q;
  long long ldq;
  unsigned char* scale;
};

// VW neighbours a thread (16 bytes of X, or one element), so a block of 32 is 32
// / VW lanes, and a warp takes VW blocks at a time. All of the scales' tiles are
// written: zeros where they belong to no block.
template <typename E, int VW>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const Args a) {
  constexpr int kLanes = 32 / VW;          // of a block
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  // groups of 4 blocks, 128 values, of the rows and of those that fill up their tiles
  const long long groups = (long long)a.block_tiles * ((a.M + 127ll) / 128 * 128);
  constexpr int kAtOnce = VW > 1 ? 32 / (4 * kLanes) : 1;       // groups of a warp
  const long long warps = (long long)gridDim.x * (kThreads / 32);
  for (long long g0 = (blockIdx.x * (long long)(kThreads / 32) + (threadIdx.x >> 5)) * kAtOnce;
       g0 < groups; g0 += warps * kAtOnce) {
    if constexpr (VW > 1) {
      const long long g = g0 + lane / (4 * kLanes);
      const bool in = g < groups;
      const long long m = in ? g / a.block_tiles : 0;
      const int tile = in ? (int)(g - m * a.block_tiles) : 0;
      const int l = lane & (4 * kLanes - 1);                    // within the group
      const long long k = tile * 128ll + l * VW;
      float v[VW];
#pragma unroll
      for (int i = 0; i < VW; ++i) v[i] = 0.f;
      // (K is a multiple of VW here)
      if (in && m < a.M && k < a.K)
        rows::unpack(rows::load<E, VW>(static_cast<const E*>(a.x) + m * a.ldx + k), v);
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < VW; ++i) most = max(most, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
      for (int d = 1; d < kLanes; d <<= 1) most = max(most, __shfl_xor_sync(kAll, most, d));
      const int e = (int)(most >> 23);                          // 255: no number among them
      const uint32_t s = e == 255 ? 255u : (uint32_t)max(e - 2, 0);
      const float unit = __uint_as_float((254u - min(s, 252u)) << 23);   // 1 / 2^(s - 127)
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < VW; i += 2)
        w |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(v[i] * unit, v[i + 1] * unit), __NV_E2M1,
                                                cudaRoundNearest) << (4 * i);
      // the row's blocks are whole: past its end there are zeros
      if (in && m < a.M && k < a.blocks * 32ll) {
        unsigned char* q = a.q + m * a.ldq + k / 2;
        if constexpr (VW == 8)
          *reinterpret_cast<uint32_t*>(q) = w;
        else
          *reinterpret_cast<uint16_t*>(q) = (uint16_t)w;
      }
      // the group's four bytes, by its first lane (past the row's end: 0)
      uint32_t word = s & 0xffu;
      word = m < a.M && tile * 4 + l / kLanes < a.blocks ? word : 0u;
      const int first = lane & ~(4 * kLanes - 1);
      const uint32_t b1 = __shfl_sync(kAll, word, first + kLanes),
                     b2 = __shfl_sync(kAll, word, first + 2 * kLanes),
                     b3 = __shfl_sync(kAll, word, first + 3 * kLanes);
      if (in && l == 0)
        *reinterpret_cast<uint32_t*>(a.scale + scale_place(m, tile * 4, a.block_tiles)) =
            word | b1 << 8 | b2 << 16 | b3 << 24;
    } else {
      const long long m = g0 / a.block_tiles;
      const int tile = (int)(g0 - m * a.block_tiles);
      const E* x = static_cast<const E*>(a.x) + m * a.ldx;
      uint32_t word = 0;
      float v[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const long long k = (tile * 4ll + b) * 32 + lane;
        v[b] = m < a.M && k < a.K ? to_f32(x[k]) : 0.f;
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const long long k = (tile * 4ll + b) * 32 + lane;
        const int e = (int)(__reduce_max_sync(kAll, __float_as_uint(v[b]) & 0x7fffffffu) >> 23);
        const uint32_t s = e == 255 ? 255u : (uint32_t)max(e - 2, 0);
        const float unit = __uint_as_float((254u - min(s, 252u)) << 23);
        const float next = __shfl_down_sync(kAll, v[b], 1);
        if (m < a.M && tile * 4 + b < a.blocks) {
          word |= s << (8 * b);
          if (!(lane & 1))
            a.q[m * a.ldq + k / 2] = (unsigned char)__nv_cvt_float2_to_fp4x2(
                make_float2(v[b] * unit, next * unit), __NV_E2M1, cudaRoundNearest);
        }
      }
      if (lane == 0)
        *reinterpret_cast<uint32_t*>(a.scale + scale_place(m, tile * 4, a.block_tiles)) = word;
    }
  }
}

// Values of a block: the code's value times the block's power, rounded to E. A
// scale of 255 makes them NaN. Eight codes (4 bytes) a thread.
template <typename E>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(const Args a, E* x, long long ldx, int wide) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const long long pieces = (a.K + 7ll) / 8, all = pieces * a.M;
  for (long long i = blockIdx.x * (long long)kThreads + threadIdx.x; i < all;
       i += (long long)gridDim.x * kThreads) {
    const long long m = i / pieces, k = (i - m * pieces) * 8;
    const unsigned char* q = a.q + m * a.ldq + k / 2;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(q);     // (rows are whole blocks)
    const uint32_t s = a.scale[scale_place(m, (int)(k / 32), a.block_tiles)];
    // 2^(s - 127): below the normal numbers for s = 0, NaN for 255
    const float unit = s == 0 ? 0x1p-127f : __uint_as_float(s == 255 ? 0x7fc00000u : s << 23);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t c = w >> (4 * j) & 15u, e = c >> 1 & 3u, f = c & 1u;
      // E2M1: 0 and 0.5, then (1 + f / 2) 2^(e - 1)
      const float mag = e == 0 ? 0.5f * (float)f : __uint_as_float((126u + e) << 23 | f << 22);
      v[j] = (c & 8u ? -mag : mag) * unit;
    }
    E* o = x + m * ldx + k;
    if (wide && k + 8 <= a.K) {
      constexpr int VW = 16 / (int)sizeof(E);
#pragma unroll
      for (int j = 0; j < 8; j += VW)
        rows::store<E, VW>(o + j, rows::pack<E, VW>(*reinterpret_cast<const float(*)[VW]>(v + j)));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (k + j < a.K) o[j] = from_f32<E>(v[j]);
    }
  }
}

template <typename... A>
cudaError_t start(void (*kernel)(A...), long long blocks, int sms, cudaStream_t stream,
                  std::common_type_t<A>... args) {
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  lc.gridDim = dim3((unsigned)(blocks < sms * 8ll ? blocks : sms * 8ll));
  lc.blockDim = dim3(kThreads);
  lc.stream = stream;
  lc.attrs = la;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, args...);
}

template <typename E>
cudaError_t quantize(const Args& a, int sms, cudaStream_t stream) {
  constexpr int VW = 16 / (int)sizeof(E);
  const long long groups = (long long)a.block_tiles * ((a.M + 127ll) / 128 * 128);
  const bool vec = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && a.ldx * sizeof(E) % 16 == 0 &&
                   a.K % VW == 0;
  const long long per_block = (kThreads / 32) * (vec ? VW / 4 : 1);
  return start(vec ? quantize_kernel<E, VW> : quantize_kernel<E, 1>,
               (groups + per_block - 1) / per_block, sms, stream, a);
}

template <typename E>
cudaError_t dequantize(const Args& a, void* x, long long ldx, int sms, cudaStream_t stream) {
  const bool wide = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && ldx * sizeof(E) % 16 == 0;
  return start(dequantize_kernel<E>, ((a.K + 7ll) / 8 * a.M + kThreads - 1) / kThreads, sms, stream,
               a, static_cast<E*>(x), ldx, (int)wide);
}

bool type_ok(int type) {
  return type == SGEMM_TYPE_F32 || type == SGEMM_TYPE_BF16 || type == SGEMM_TYPE_F16;
}

// Checks of both calls; X's are the same whichever way it goes.
int check(int M, int K, int type, const void* X, int ldx, const void* Q, int ldq, const void* scale) {
  if (!type_ok(type)) return SGEMM_ERR_INVALID_VALUE;
  if (M < 0 || K < 0) return SGEMM_ERR_INVALID_DIM;
  const long long bytes = (K + 31ll) / 32 * 16;
  if (ldx < (K > 1 ? K : 1) || ldq < bytes || ldq % 16 != 0) return SGEMM_ERR_INVALID_LD;
  if (M == 0 || K == 0) return SGEMM_OK;
  if (X == nullptr || Q == nullptr || scale == nullptr) return SGEMM_ERR_NULL_PTR;
  const uintptr_t mask = type == SGEMM_TYPE_F32 ? 3u : 1u;
  if ((reinterpret_cast<uintptr_t>(X) & mask) || (reinterpret_cast<uintptr_t>(Q) & 15u) ||
      (reinterpret_cast<uintptr_t>(scale) & 15u))
    return SGEMM_ERR_MISALIGNED;
  return SGEMM_OK;
}

Args args_of(int M, int K, const void* X, int ldx, const unsigned char* Q, int ldq,
             const unsigned char* scale) {
  Args a = {};
  a.M = M;
  a.K = K;
  a.blocks = (int)((K + 31ll) / 32);
  a.block_tiles = (a.blocks + 3) / 4;
  a.x = X;
  a.ldx = ldx;
  a.q = const_cast<unsigned char*>(Q);
  a.ldq = ldq;
  a.scale = const_cast<unsigned char*>(scale);
  return a;
}

int device(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return SGEMM_ERR_LAUNCH;
  }
  return library_device_sms(dev, sms);
}

int done(cudaError_t e) {
  if (e == cudaSuccess) return SGEMM_OK;
  cudaGetLastError();
  return SGEMM_ERR_LAUNCH;
}

}  // namespace
}  // namespace mx4
}  // namespace sgemm_gb300

using namespace sgemm_gb300;

SGEMM_API int sgemm_mx4_quantize(int M, int K, int type, const void* X, int ldx, unsigned char* Q,
                                 int ldq, unsigned char* scale, void* stream_) {
  int st = mx4::check(M, K, type, X, ldx, Q, ldq, scale);
  if (st != SGEMM_OK || M == 0 || K == 0) return st;
  int sms = 0;
  st = mx4::device(&sms);
  if (st != SGEMM_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const mx4::Args a = mx4::args_of(M, K, X, ldx, Q, ldq, scale);
  return mx4::done(type == SGEMM_TYPE_F32    ? mx4::quantize<float>(a, sms, stream)
                   : type == SGEMM_TYPE_BF16 ? mx4::quantize<__nv_bfloat16>(a, sms, stream)
                                             : mx4::quantize<__half>(a, sms, stream));
}

SGEMM_API int sgemm_mx4_dequantize(int M, int K, const unsigned char* Q, int ldq,
                                   const unsigned char* scale, int type, void* X, int ldx,
                                   void* stream_) {
  int st = mx4::check(M, K, type, X, ldx, Q, ldq, scale);
  if (st != SGEMM_OK || M == 0 || K == 0) return st;
  int sms = 0;
  st = mx4::device(&sms);
  if (st != SGEMM_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const mx4::Args a = mx4::args_of(M, K, nullptr, 0, Q, ldq, scale);
  return mx4::done(type == SGEMM_TYPE_F32    ? mx4::dequantize<float>(a, X, ldx, sms, stream)
                   : type == SGEMM_TYPE_BF16 ? mx4::dequantize<__nv_bfloat16>(a, X, ldx, sms, stream)
                                             : mx4::dequantize<__half>(a, X, ldx, sms, stream));
}
