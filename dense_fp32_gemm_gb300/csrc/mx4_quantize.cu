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

// A warp's share: a piece of a row (whole groups of 4 blocks), whose loads are
// all in flight before the first is used. Numbered row by row; the division is
// done in 32 bits where the numbers allow it (in 64 it took most of the time).
struct Share {
  long long m;
  int piece;
};
__device__ __forceinline__ Share share_of(long long i, int pieces) {
  if (i <= 0xffffffffll) {
    const unsigned m = (unsigned)i / (unsigned)pieces;
    return {m, (int)((unsigned)i - m * (unsigned)pieces)};
  }
  const long long m = i / pieces;
  return {m, (int)(i - m * pieces)};
}

// The byte of a block whose largest magnitude has these bits (255: no number
// among them), and the factor that brings its values to units.
__device__ __forceinline__ uint32_t power_of(uint32_t most) {
  const int e = (int)(most >> 23);
  return e == 255 ? 255u : (uint32_t)max(e - 2, 0);
}
__device__ __forceinline__ float units_of(uint32_t s) {
  return __uint_as_float((254u - min(s, 252u)) << 23);   // 1 / 2^(s - 127)
}

// VW neighbours a thread (16 bytes of X, or one element), so a block of 32 is 32
// / VW lanes, and a warp takes VW blocks at a time. All of the scales' tiles are
// written: zeros where they belong to no block.
constexpr int kAhead = 4;                              // pieces of a thread
constexpr int values_of(int vw) { return vw > 1 ? 32 * vw * kAhead : 128; }   // of a warp's share
template <typename E, int VW>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const Args a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  constexpr int kValues = values_of(VW);
  const int pieces = (int)((a.block_tiles * 128ll + kValues - 1) / kValues);
  // (the rows that fill up the scales' tiles have zeros, too)
  const long long all = (a.M + 127ll) / 128 * 128 * pieces;
  const long long warps = (long long)gridDim.x * (kThreads / 32);
  for (long long i = blockIdx.x * (long long)(kThreads / 32) + (threadIdx.x >> 5); i < all; i += warps) {
    const Share sh = share_of(i, pieces);
    const bool row = sh.m < a.M;
    const E* x = static_cast<const E*>(a.x) + sh.m * a.ldx;
    unsigned char* q = a.q + sh.m * a.ldq;
    const long long k0 = (long long)sh.piece * kValues;
    if constexpr (VW > 1) {
      constexpr int kLanes = 32 / VW;                  // of a block
      rows::Piece<E, VW> in[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const long long k = k0 + j * (32 * VW) + lane * VW;
        if (row && k < a.K) in[j] = rows::load<E, VW>(x + k);   // (K is a multiple of VW here)
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const long long k = k0 + j * (32 * VW) + lane * VW;
        if (k - lane * VW >= a.block_tiles * 128ll) break;      // (the whole warp)
        float v[VW];
#pragma unroll
        for (int c = 0; c < VW; ++c) v[c] = 0.f;
        if (row && k < a.K) rows::unpack(in[j], v);
        uint32_t most = 0;
#pragma unroll
        for (int c = 0; c < VW; ++c) most = max(most, __float_as_uint(v[c]) & 0x7fffffffu);
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) most = max(most, __shfl_xor_sync(kAll, most, d));
        const uint32_t s = power_of(most);
        const float unit = units_of(s);
        uint32_t w = 0;
#pragma unroll
        for (int c = 0; c < VW; c += 2)
          w |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(v[c] * unit, v[c + 1] * unit),
                                                  __NV_E2M1, cudaRoundNearest) << (4 * c);
        // the row's blocks are whole: past its end there are zeros
        const bool block = row && k < a.blocks * 32ll;
        if (block) {
          if constexpr (VW == 8)
            *reinterpret_cast<uint32_t*>(q + k / 2) = w;
          else
            *reinterpret_cast<uint16_t*>(q + k / 2) = (uint16_t)w;
        }
        // a group's four bytes, by its first lane
        const uint32_t byte = block ? s : 0u;
        const int first = lane & ~(4 * kLanes - 1);
        const uint32_t word = byte | __shfl_sync(kAll, byte, first + kLanes) << 8 |
                              __shfl_sync(kAll, byte, first + 2 * kLanes) << 16 |
                              __shfl_sync(kAll, byte, first + 3 * kLanes) << 24;
        if (lane == first && k < a.block_tiles * 128ll)
          *reinterpret_cast<uint32_t*>(a.scale + scale_place(sh.m, (int)(k / 32), a.block_tiles)) = word;
      }
    } else {
      uint32_t word = 0;
      float v[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const long long k = k0 + b * 32 + lane;
        v[b] = row && k < a.K ? to_f32(x[k]) : 0.f;
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const long long k = k0 + b * 32 + lane;
        const uint32_t s = power_of(__reduce_max_sync(kAll, __float_as_uint(v[b]) & 0x7fffffffu));
        const float unit = units_of(s);
        const float next = __shfl_down_sync(kAll, v[b], 1);
        if (row && k - lane < a.blocks * 32ll) {
          word |= s << (8 * b);
          if (!(lane & 1))
            q[k / 2] = (unsigned char)__nv_cvt_float2_to_fp4x2(make_float2(v[b] * unit, next * unit),
                                                               __NV_E2M1, cudaRoundNearest);
        }
      }
      if (lane == 0)
        *reinterpret_cast<uint32_t*>(a.scale + scale_place(sh.m, sh.piece * 4, a.block_tiles)) = word;
    }
  }
}

// Values of a block: the code's value times the block's power, rounded to E. A
// scale of 255 makes them NaN. Eight codes (4 bytes) a thread at a time.
template <typename E>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(const Args a, E* x, long long ldx, int wide) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  constexpr int kValues = 32 * 8 * kAhead;
  const int lane = threadIdx.x & 31, pieces = (int)((a.K + (long long)kValues - 1) / kValues);
  const long long all = (long long)a.M * pieces, warps = (long long)gridDim.x * (kThreads / 32);
  for (long long i = blockIdx.x * (long long)(kThreads / 32) + (threadIdx.x >> 5); i < all; i += warps) {
    const Share sh = share_of(i, pieces);
    const long long k0 = (long long)sh.piece * kValues + lane * 8;
    const unsigned char* q = a.q + sh.m * a.ldq;
    uint32_t w[kAhead], s[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const long long k = k0 + j * 256;
      if (k >= a.K) continue;
      w[j] = __ldcs(reinterpret_cast<const uint32_t*>(q + k / 2));   // (rows are whole blocks)
      s[j] = a.scale[scale_place(sh.m, (int)(k / 32), a.block_tiles)];
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const long long k = k0 + j * 256;
      if (k >= a.K) continue;
      // 2^(s - 127): below the normal numbers for s = 0, NaN for 255
      const float unit =
          s[j] == 0 ? 0x1p-127f : __uint_as_float(s[j] == 255 ? 0x7fc00000u : s[j] << 23);
      float v[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint32_t code = w[j] >> (4 * c) & 15u, e = code >> 1 & 3u, f = code & 1u;
        // E2M1: 0 and 0.5, then (1 + f / 2) 2^(e - 1)
        const float mag = e == 0 ? 0.5f * (float)f : __uint_as_float((126u + e) << 23 | f << 22);
        v[c] = (code & 8u ? -mag : mag) * unit;
      }
      E* o = x + sh.m * ldx + k;
      if (wide && k + 8 <= a.K) {
        constexpr int VW = 16 / (int)sizeof(E);
#pragma unroll
        for (int c = 0; c < 8; c += VW) {
          float part[VW];
#pragma unroll
          for (int d = 0; d < VW; ++d) part[d] = v[c + d];
          rows::store<E, VW>(o + c, rows::pack<E, VW>(part));
        }
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (k + c < a.K) o[c] = from_f32<E>(v[c]);
      }
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
  const bool vec = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && a.ldx * sizeof(E) % 16 == 0 &&
                   a.K % VW == 0;
  const int values = values_of(vec ? VW : 1);
  const long long shares = (a.M + 127ll) / 128 * 128 * ((a.block_tiles * 128ll + values - 1) / values);
  return start(vec ? quantize_kernel<E, VW> : quantize_kernel<E, 1>,
               (shares + kThreads / 32 - 1) / (kThreads / 32), sms, stream, a);
}

template <typename E>
cudaError_t dequantize(const Args& a, void* x, long long ldx, int sms, cudaStream_t stream) {
  const bool wide = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && ldx * sizeof(E) % 16 == 0;
  constexpr int kValues = 32 * 8 * kAhead;
  const long long shares = (a.K + (long long)kValues - 1) / kValues * a.M;
  return start(dequantize_kernel<E>, (shares + kThreads / 32 - 1) / (kThreads / 32), sms, stream, a,
               static_cast<E*>(x), ldx, (int)wide);
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
