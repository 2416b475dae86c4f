// elements.cuh -- element types of the row-wise operators, and pieces of a row:
// 16 bytes at a time where everything is aligned for that, else one element.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace sgemm_gb300 {
namespace rows {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename E>
__device__ __forceinline__ E from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// VW neighbouring elements of a row.
template <typename E, int VW>
struct __align__(VW * sizeof(E)) Piece {
  E e[VW];
};

// Loads that are read once; the memory may be written later in the same kernel.
template <typename E, int VW>
__device__ __forceinline__ Piece<E, VW> load(const E* p) {
  constexpr int kBytes = VW * (int)sizeof(E);
  static_assert(kBytes == 16 || VW == 1, "pieces of 16 bytes or of one element");
  Piece<E, VW> r;
  if constexpr (kBytes == 16)
    *reinterpret_cast<uint4*>(&r) = __ldcs(reinterpret_cast<const uint4*>(p));
  else
    r.e[0] = *p;
  return r;
}
template <typename E, int VW>
__device__ __forceinline__ void store(E* p, const Piece<E, VW>& r) {
  if constexpr (VW * sizeof(E) == 16)
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(&r);
  else
    *p = r.e[0];
}
// VW values of a vector that no kernel of the call writes, as FP32; 16-byte
// aligned where VW > 1.
template <typename W, int VW>
__device__ __forceinline__ void load_vector(const W* p, float (&v)[VW]) {
  if constexpr (VW == 1) {
    v[0] = to_f32(__ldg(p));
  } else {
    constexpr int kWords = VW * (int)sizeof(W) / 4;
    uint32_t w[kWords];
    if constexpr (kWords == 2) {
      const uint2 a = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = a.x;
      w[1] = a.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(p) + i / 4);
        w[i] = a.x;
        w[i + 1] = a.y;
        w[i + 2] = a.z;
        w[i + 3] = a.w;
      }
    }
    const W* e = reinterpret_cast<const W*>(w);
#pragma unroll
    for (int i = 0; i < VW; ++i) v[i] = to_f32(e[i]);
  }
}

}  // namespace rows
}  // namespace sgemm_gb300
