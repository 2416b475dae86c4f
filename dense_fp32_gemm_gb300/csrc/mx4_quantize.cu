// mx4_quantize.cu -- sgemm_mx4_quantize and sgemm_mx4_dequantize: rows of a matrix
// to 4-bit floating point in blocks of 32 values with a power of two each, and
// back.
//
// A block's power is floor(log2(max|x|)) - 2, so that its largest value lies in
// 4 .. 8 units; values are rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6
// units (ties to the even code), beyond 6 to 6. Multiplying by a power of two is
// exact, so the codes are defined bit by bit.
//
// Bound by DRAM, the 16-bit form by its instructions (13 a value, 75 % of the issue
// slots). Measured on GB300: 8192 x 4096 FP32 21.4 us, 7.1 TB/s with a part of it
// still in L2; BF16 16.2 us, 5.2 TB/s; back to FP32 25.5 us, 6.0 TB/s. (Numbers of
// the rows by 64-bit divisions, one load at a time: 36, 31 and 31 us.) One row of
// 4096: 2 us.
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

// Eight neighbours of a row, as they are stored: what the kernel needs of them.
// The largest magnitude as the bits of an FP32 value, a NaN above all numbers.
template <typename E>
struct Eight {
  uint4 w;
  __device__ __forceinline__ void load(const E* p) { w = __ldcs(reinterpret_cast<const uint4*>(p)); }
  // from the 32 bytes around them, `skip` bytes on; the first n of them (the rest: zeros)
  static constexpr int kChunks = 2;
  __device__ __forceinline__ void extract(const uint4 (&from)[kChunks], unsigned skip, unsigned n) {
    uint32_t c[8] = {from[0].x, from[0].y, from[0].z, from[0].w, from[1].x, from[1].y, from[1].z, from[1].w};
#pragma unroll
    for (int i = 0; i < 6; ++i) c[i] = skip & 8u ? c[i + 2] : c[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) c[i] = skip & 4u ? c[i + 1] : c[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = __funnelshift_r(c[i], c[i + 1], (skip & 2u) * 8u);
      if (2 * i + 1 >= n) c[i] = 2 * i >= n ? 0u : c[i] & 0xffffu;
    }
    w = make_uint4(c[0], c[1], c[2], c[3]);
  }
  __device__ __forceinline__ void clear() { w = make_uint4(0u, 0u, 0u, 0u); }
  // (the bits of 16-bit magnitudes are in the order of the magnitudes)
  __device__ __forceinline__ uint32_t most() const {
    const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
    const uint16_t h = (uint16_t)max(m & 0xffffu, m >> 16);
    return __float_as_uint(to_f32(*reinterpret_cast<const E*>(&h)));
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = rows::unpack2(in[i], E{});
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  static constexpr int kChunks = 3;
  __device__ __forceinline__ void extract(const uint4 (&from)[kChunks], unsigned skip, unsigned n) {
    uint32_t c[12] = {from[0].x, from[0].y, from[0].z, from[0].w, from[1].x, from[1].y,
                      from[1].z, from[1].w, from[2].x, from[2].y, from[2].z, from[2].w};
#pragma unroll
    for (int i = 0; i < 9; ++i) c[i] = skip & 8u ? c[i + 2] : c[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = skip & 4u ? c[i + 1] : c[i];
      if (i >= n) c[i] = 0u;
    }
    a = make_float4(__uint_as_float(c[0]), __uint_as_float(c[1]), __uint_as_float(c[2]), __uint_as_float(c[3]));
    b = make_float4(__uint_as_float(c[4]), __uint_as_float(c[5]), __uint_as_float(c[6]), __uint_as_float(c[7]));
  }
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ uint32_t most() const {
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

// The codes of eight values, the first in the lowest bits.
__device__ __forceinline__ uint32_t codes_of(const float (&v)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return w;
}

// The 16-byte chunks around the values k .. k + 7 of a row (of K) that may start
// anywhere: those that hold one of the row's. What is beside the row is read with them
// where that is the matrix's (`inner`).
template <typename E>
__device__ __forceinline__ void load_around(const E* row, unsigned k, unsigned K, unsigned skip, bool inner,
                                            uint4 (&c)[Eight<E>::kChunks]) {
  constexpr unsigned VW = 16 / sizeof(E);
  const unsigned first = k - skip / (unsigned)sizeof(E);       // (below 0 in front of the row)
  const E* p = row + k - skip / sizeof(E);
#pragma unroll
  for (unsigned i = 0; i < Eight<E>::kChunks; ++i) {
    c[i] = make_uint4(0u, 0u, 0u, 0u);
    if (i > 0 && first + i * VW >= K) continue;
    if (inner) {
      c[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    } else {
      E* e = reinterpret_cast<E*>(&c[i]);
#pragma unroll
      for (unsigned j = 0; j < VW; ++j)
        if (first + i * VW + j < K) e[j] = p[i * VW + j];
    }
  }
}

// Eight neighbours a thread, so a block of 32 is 4 lanes, and a warp takes 8 blocks
// at a time. SHIFT: rows that do not start on 16 bytes, or do not end after a multiple
// of 8 values; the values are taken out of the chunks around them (8192 x 4097: BF16
// 31 us, FP32 47, by single elements 59 each). All of the scales' tiles are
// written: zeros where they belong to no block.
constexpr int kAhead = 4;                              // pieces of a thread
constexpr int kValues = 256 * kAhead;                  // of a warp's share
template <typename E, bool SHIFT>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const Args a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const unsigned lane = threadIdx.x & 31, K = (unsigned)a.K;
  const unsigned row_end = (unsigned)a.blocks * 32u, tile_end = (unsigned)a.block_tiles * 128u;
  const int pieces = (int)((tile_end + kValues - 1) / kValues);
  // (the rows that fill up the scales' tiles have zeros, too)
  const long long all = (a.M + 127ll) / 128 * 128 * pieces;
  const long long warps = (long long)gridDim.x * (kThreads / 32);
  for (long long i = blockIdx.x * (long long)(kThreads / 32) + (threadIdx.x >> 5); i < all; i += warps) {
    const Share sh = share_of(i, pieces);
    const bool row = sh.m < a.M;
    const E* x = static_cast<const E*>(a.x) + sh.m * a.ldx;
    unsigned char* q = a.q + sh.m * a.ldq;
    unsigned char* scale = a.scale + scale_place(sh.m, 0, a.block_tiles);   // the row's: 512 bytes a tile
    const unsigned k0 = (unsigned)sh.piece * kValues;
    const unsigned skip = SHIFT ? (unsigned)(reinterpret_cast<uintptr_t>(x) & 15u) : 0u;
    const bool inner = SHIFT && rows::inner_row(sh.m, a.M, a.K, 16 / (int)sizeof(E));
    Eight<E> in[kAhead];
    uint4 around[SHIFT ? kAhead : 1][Eight<E>::kChunks];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const unsigned k = k0 + j * 256u + lane * 8u;
      in[j].clear();
      if (!row || k >= K) continue;
      if constexpr (SHIFT)
        load_around<E>(x, k, K, skip, inner, around[j]);
      else
        in[j].load(x + k);                             // (K is a multiple of 8 here)
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const unsigned k = k0 + j * 256u + lane * 8u;
      if (k0 + j * 256u >= tile_end) break;            // (the whole warp)
      if constexpr (SHIFT)
        if (row && k < K) in[j].extract(around[j], skip, K - k);
      uint32_t most = in[j].most();
      most = max(most, __shfl_xor_sync(kAll, most, 1));
      most = max(most, __shfl_xor_sync(kAll, most, 2));
      const uint32_t s = power_of(most);
      const float unit = units_of(s);
      float v[8];
      in[j].values(v);
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] *= unit;
      // the row's blocks are whole: past its end there are zeros
      const bool block = row && k < row_end;
      if (block) *reinterpret_cast<uint32_t*>(q + k / 2) = codes_of(v);
      // four blocks' bytes, by the first of their 16 lanes
      uint32_t word = block ? s << (lane * 2 & 24u) : 0u;
      word |= __shfl_xor_sync(kAll, word, 4);
      word |= __shfl_xor_sync(kAll, word, 8);
      if ((lane & 15u) == 0 && k < tile_end)
        *reinterpret_cast<uint32_t*>(scale + (size_t)(k / 128) * 512) = word;
    }
  }
}

// 2^(s - 127): below the normal numbers for s = 0, NaN for 255.
__device__ __forceinline__ float power(uint32_t s) {
  return s == 0 ? 0x1p-127f : __uint_as_float(s == 255 ? 0x7fc00000u : s << 23);
}
__device__ __forceinline__ uint32_t codes_at(const unsigned char* q, int word, unsigned K) {
  return word >= 0 && (unsigned)word * 8u < K ? __ldcs(reinterpret_cast<const uint32_t*>(q) + word) : 0u;
}

// Values of a block: the code's value times the block's power, rounded to E. A
// scale of 255 makes them NaN. A thread writes 16 bytes at a time (4 or 8 values).
// SHIFT: rows of X that do not start on 16 bytes; places count from the boundary
// before the row, and a thread's codes lie in two words and up to two blocks (8192 x
// 4097: BF16 23 us, FP32 33; by single elements 90 and 44).
template <typename E, bool SHIFT>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const Args a, E* x, long long ldx) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  constexpr int VW = 16 / (int)sizeof(E), kPieces = 8 * kAhead / VW;
  const unsigned lane = threadIdx.x & 31, K = (unsigned)a.K;
  const int pieces = (int)((K + (SHIFT ? VW - 1u : 0u) + kValues - 1) / kValues);
  const long long all = (long long)a.M * pieces, warps = (long long)gridDim.x * (kThreads / 32);
  for (long long i = blockIdx.x * (long long)(kThreads / 32) + (threadIdx.x >> 5); i < all; i += warps) {
    const Share sh = share_of(i, pieces);
    const unsigned first = SHIFT ? rows::start_of<E>(x, sh.m, ldx) : 0u, end = K + first;
    const unsigned c0 = (unsigned)sh.piece * kValues + lane * VW;
    const unsigned char* q = a.q + sh.m * a.ldq;
    const unsigned char* scale = a.scale + scale_place(sh.m, 0, a.block_tiles);
    E* o = x + sh.m * ldx;
    auto scale_of = [&](unsigned block) { return (uint32_t)__ldg(scale + (size_t)(block / 4) * 512 + block % 4); };
    uint32_t w[kPieces], more[kPieces], s[kPieces], t[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const unsigned c = c0 + j * (32u * VW);
      if (c >= end) continue;
      const int k = (int)(c - first);                  // (below 0 in front of the row)
      // (rows are whole blocks)
      if constexpr (SHIFT) {
        w[j] = codes_at(q, k >> 3, K);
        more[j] = codes_at(q, (k >> 3) + 1, K);
        const unsigned k1 = (unsigned)max(k, 0);
        s[j] = scale_of(k1 / 32);
        t[j] = scale_of(min((k1 + VW - 1) / 32, (unsigned)a.blocks - 1u));
      } else {
        if constexpr (VW == 8)
          w[j] = __ldcs(reinterpret_cast<const uint32_t*>(q + k / 2));
        else
          w[j] = __ldcs(reinterpret_cast<const uint16_t*>(q + k / 2));
        s[j] = scale_of((unsigned)k / 32);
      }
    }
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const unsigned c = c0 + j * (32u * VW);
      if (c >= end) continue;
      const int k = (int)(c - first);
      if (SHIFT) w[j] = __funnelshift_r(w[j], more[j], 4u * (k & 7));
      const float unit = power(s[j]), unit1 = SHIFT ? power(t[j]) : unit;
      const int in_first = SHIFT ? 32 - (k & 31) : VW;   // values of the first block
      float v[VW];
#pragma unroll
      for (int i = 0; i < VW; i += 2) {
        const __half2_raw h =
            __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(w[j] >> (4 * i) & 0xffu), __NV_E2M1);
        const float2 f = __half22float2(__half2(h));
        v[i] = f.x * (i < in_first ? unit : unit1);
        v[i + 1] = f.y * (i + 1 < in_first ? unit : unit1);
      }
      if (k >= 0 && c + VW <= end) {
        rows::store<E, VW>(o + k, rows::pack<E, VW>(v));
      } else {
#pragma unroll
        for (int i = 0; i < VW; ++i)
          if (k + i >= 0 && c + i < end) o[k + i] = from_f32<E>(v[i]);
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
  lc.gridDim = dim3((unsigned)(blocks < sms * 64ll ? blocks : sms * 64ll));
  lc.blockDim = dim3(kThreads);
  lc.stream = stream;
  lc.attrs = la;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, args...);
}

template <typename E>
cudaError_t quantize(const Args& a, int sms, cudaStream_t stream) {
  const bool whole = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && a.ldx * sizeof(E) % 16 == 0 &&
                     a.K % 8 == 0;
  const long long shares = (a.M + 127ll) / 128 * 128 * ((a.block_tiles * 128ll + kValues - 1) / kValues);
  return start(whole ? quantize_kernel<E, false> : quantize_kernel<E, true>,
               (shares + kThreads / 32 - 1) / (kThreads / 32), sms, stream, a);
}

template <typename E>
cudaError_t dequantize(const Args& a, void* x, long long ldx, int sms, cudaStream_t stream) {
  const bool whole = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && ldx * sizeof(E) % 16 == 0;
  const long long places = a.K + (whole ? 0ll : 16 / (int)sizeof(E) - 1ll);
  const long long shares = (places + kValues - 1) / kValues * a.M;
  return start(whole ? dequantize_kernel<E, false> : dequantize_kernel<E, true>,
               (shares + kThreads / 32 - 1) / (kThreads / 32), sms, stream, a, static_cast<E*>(x), ldx);
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
