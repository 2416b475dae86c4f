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

// VW neighbouring elements of a row, as 32-bit words where there are several
// (two 16-bit elements a word; element by element the compiler took twice the
// registers).
template <typename E, int VW>
struct Piece {
  static constexpr int kWords = VW * (int)sizeof(E) / 4;
  static_assert(kWords == 4, "pieces of 16 bytes or of one element");
  uint4 w;
};
template <typename E>
struct Piece<E, 1> {
  E e;
};

// Loads that are read once; the memory may be written later in the same kernel.
template <typename E, int VW>
__device__ __forceinline__ Piece<E, VW> load(const E* p) {
  Piece<E, VW> r;
  if constexpr (VW == 1)
    r.e = *p;
  else
    r.w = __ldcs(reinterpret_cast<const uint4*>(p));
  return r;
}
template <typename E, int VW>
__device__ __forceinline__ void store(E* p, const Piece<E, VW>& r) {
  if constexpr (VW == 1)
    *p = r.e;
  else
    *reinterpret_cast<uint4*>(p) = r.w;
}

__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The elements as FP32, and FP32 values rounded to elements.
template <typename E, int VW>
__device__ __forceinline__ void unpack(const Piece<E, VW>& p, float (&v)[VW]) {
  if constexpr (VW == 1) {
    v[0] = to_f32(p.e);
  } else {
    const uint32_t w[4] = {p.w.x, p.w.y, p.w.z, p.w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (VW == 4) {
        v[i] = __uint_as_float(w[i]);
      } else {
        const float2 f = unpack2(w[i], E{});
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
}
template <typename E, int VW>
__device__ __forceinline__ Piece<E, VW> pack(const float (&v)[VW]) {
  Piece<E, VW> p;
  if constexpr (VW == 1) {
    p.e = from_f32<E>(v[0]);
  } else if constexpr (VW == 4) {
    p.w = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                     __float_as_uint(v[3]));
  } else {
    p.w = make_uint4(pack2(v[0], v[1], E{}), pack2(v[2], v[3], E{}), pack2(v[4], v[5], E{}),
                     pack2(v[6], v[7], E{}));
  }
  return p;
}

// Elements between the 16-byte boundary before row m and its start.
template <typename E>
__device__ __forceinline__ unsigned start_of(const void* p, long long m, long long ld) {
  return (unsigned)((reinterpret_cast<uintptr_t>(p) + m * ld * sizeof(E)) & 15u) / (unsigned)sizeof(E);
}
// Whether the whole pieces of row m are within the matrix, whose pitch is N at least.
__device__ __forceinline__ bool inner_row(long long m, int M, int N, int vw) {
  return m * N >= vw && (M - 1 - m) * N >= vw;
}
// The piece at place c of a row whose elements are at first .. end - 1 (SHIFT: places
// count from the 16-byte boundary before the row, else first is 0 and pieces are
// whole). Beside the row it holds whatever is there, until clean() has made that
// zeros: a load that nothing waits for. `inner`: the matrix has rows before and after
// this one, so that what is beside it is the matrix's (else it is not read).
template <typename E, int VW, bool SHIFT>
__device__ __forceinline__ Piece<E, VW> load_at(const E* row, unsigned c, unsigned first, unsigned end,
                                                bool inner) {
  if constexpr (SHIFT) {
    if (!inner && (c < first || c + VW > end)) {
      Piece<E, VW> p;
      p.w = make_uint4(0u, 0u, 0u, 0u);
      E* e = reinterpret_cast<E*>(&p.w);
#pragma unroll
      for (int j = 0; j < VW; ++j)
        if (c + j >= first && c + j < end) e[j] = row[c + j];
      return p;
    }
  }
  return load<E, VW>(row + c);
}
template <typename E, int VW, bool SHIFT>
__device__ __forceinline__ Piece<E, VW> clean(Piece<E, VW> p, unsigned c, unsigned first, unsigned end) {
  if constexpr (SHIFT) {
    if (c < first || c + VW > end) {
      E* e = reinterpret_cast<E*>(&p.w);
#pragma unroll
      for (int j = 0; j < VW; ++j)
        if (c + j < first || c + j >= end) e[j] = from_f32<E>(0.f);
    }
  }
  return p;
}
// (what is outside the row is not written)
template <typename E, int VW, bool SHIFT>
__device__ __forceinline__ void store_at(E* row, unsigned c, unsigned first, unsigned end,
                                         const Piece<E, VW>& p) {
  if constexpr (SHIFT) {
    if (c < first || c + VW > end) {
      const E* e = reinterpret_cast<const E*>(&p.w);
#pragma unroll
      for (int j = 0; j < VW; ++j)
        if (c + j >= first && c + j < end) row[c + j] = e[j];
      return;
    }
  }
  store<E, VW>(row + c, p);
}

// VW values of a vector that no kernel of the call writes, as FP32; 16-byte
// aligned where VW > 1. SHARED: in shared memory.
template <typename W, int VW, bool SHARED = false>
__device__ __forceinline__ void load_vector(const W* p, float (&v)[VW]) {
  auto get = [](auto* q) {
    if constexpr (SHARED)
      return *q;
    else
      return __ldg(q);
  };
  if constexpr (VW == 1) {
    v[0] = to_f32(get(p));
  } else {
    constexpr int kWords = VW * (int)sizeof(W) / 4;
    uint32_t w[kWords];
    if constexpr (kWords == 2) {
      const uint2 a = get(reinterpret_cast<const uint2*>(p));
      w[0] = a.x;
      w[1] = a.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 a = get(reinterpret_cast<const uint4*>(p) + i / 4);
        w[i] = a.x;
        w[i + 1] = a.y;
        w[i + 2] = a.z;
        w[i + 3] = a.w;
      }
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(W) == 4) {
        v[i] = __uint_as_float(w[i]);
      } else {
        const float2 f = unpack2(w[i], W{});
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
}

}  // namespace rows
}  // namespace sgemm_gb300
