// grad_clip.cu -- sgemm_grad_clip: the 2-norm of many tensors taken together,
// and every tensor scaled so that the norm stays below a bound.
//
//   norm = sqrt(sum over all tensors of g^2)
//   coef = min(1, max_norm / (norm + 1e-6)),  out = g * coef
//
// Two launches a list of up to kTable tensors: the squares, then the scaling.
// The tensors are cut into pieces of 16 or 32 KB that start on 16-byte addresses
// (the elements before a tensor's first such address form its first, shorter
// vector), dealt to the CTAs in turn. Squares are summed in FP32 over at most
// four vectors of a thread's share of a piece (16 FP32 or 32 16-bit values) and
// in FP64 beyond; every CTA of the second launch adds the first one's per-CTA
// sums in the same order, so the result does not depend on timing.
//
// Bound by HBM: the gradients are read twice (the norm is not known before all of
// them have been) and written once, or read once where nothing is clipped.
// 400 M BF16 values: 396 us, 6.1 TB/s of 2.4 GB (measured copy: 6.78 TB/s);
// 60 M FP32 values below the bound: 47 us, 5.1 TB/s; 48 tensors of 1 M FP32
// values in all: 10.8 us a call, the two launches. Gradients of zeros only, whose
// sums have to be told from squares that vanish: 268 MB in 56 us, others in 48.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cstring>
#include <mutex>

#include "../../include/sgemm_gb300.h"
#include "ptx.cuh"

#define SGEMM_API extern "C" __attribute__((visibility("default")))

namespace sgemm_gb300 {

std::unique_lock<std::mutex> library_lock();
int library_workspace(int dev, cudaStream_t stream, size_t floats, size_t nflags, float** scratch,
                      int** status, uint32_t** flags, uint32_t* epoch, uint32_t** counters);
int library_device_sms(int dev, int* sms);

namespace {

constexpr int kThreads = 256;
// A piece is `vecs` 16-byte vectors a thread: 4 (16 KB), or, in the first pass
// over at least kLarge bytes, 8: twice the bytes in flight (60 M FP32 values 44
// against 50 us). In the second pass 8 need more registers than its CTAs have
// (150 M values 312 against 306 us).
constexpr long long kLarge = 64 << 20;
constexpr int piece_bytes(int vecs) { return vecs * 16 * kThreads; }
// CTAs resident per SM (64 and 51 registers a thread)
constexpr int ctas_per_sm(int vecs) { return vecs == 8 ? 4 : 5; }
constexpr int kTable = 1000;            // tensors per launch (they are kernel parameters)

struct Entry {
  const void* in;
  void* out;
  long long n;     // elements
};
template <int CAP>
struct Table {
  int count;
  unsigned pieces;
  bool in_place;              // every tensor is its own output
  Entry e[CAP];
  unsigned first[CAP];        // number of the tensor's first piece
  unsigned char type[CAP];
};
static_assert(sizeof(Table<kTable>) + 64 <= 32764, "kernel parameters");

__device__ __forceinline__ float elem_f32(const void* p, long long i, int type) {
  if (type == SGEMM_TYPE_F32) return static_cast<const float*>(p)[i];
  if (type == SGEMM_TYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void put_elem(void* p, long long i, int type, float v) {
  if (type == SGEMM_TYPE_F32)
    static_cast<float*>(p)[i] = v;
  else if (type == SGEMM_TYPE_BF16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// The values of a 16-byte vector (4 FP32, or 8 of 16 bits) as FP32.
__device__ __forceinline__ void unpack(const uint4& v, int type, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (type == SGEMM_TYPE_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = __uint_as_float(w[i]);
      x[i + 4] = 0.f;
    }
  } else if (type == SGEMM_TYPE_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}
__device__ __forceinline__ uint4 pack(const float (&x)[8], int type) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (type == SGEMM_TYPE_F32) {
      w[i] = __float_as_uint(x[i]);
    } else if (type == SGEMM_TYPE_BF16) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The tensor of piece `at` and the piece's place in it, in vectors counted
// from the 16-byte address at or below the tensor's start.
template <int CAP>
__device__ __forceinline__ int find(const Table<CAP>& t, unsigned at, int last) {
  // (most often that of the piece before)
  if (last >= 0 && t.first[last] <= at && (last + 1 == t.count || at < t.first[last + 1]))
    return last;
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= at) lo = mid; else hi = mid - 1;
  }
  return lo;
}
__device__ __forceinline__ int elem_size(int type) { return type == SGEMM_TYPE_F32 ? 4 : 2; }

// Sum of a block's values in FP64 (the same order every time), in thread 0.
__device__ __forceinline__ double block_sum(double v, double* buf) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_down_sync(0xffffffffu, v, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < kThreads / 32; ++w) s += buf[w];
  return s;
}

template <int CAP, int VECS>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(VECS))
    squares_kernel(const __grid_constant__ Table<CAP> t, double* sums) {
  __shared__ double buf[kThreads / 32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  double total = 0.0;
  int i = -1;
  for (unsigned at = blockIdx.x; at < t.pieces; at += gridDim.x) {
    i = find(t, at, i);
    const int type = t.type[i], es = elem_size(type), per = 16 / es;
    const char* in = static_cast<const char*>(t.e[i].in);
    const int head = (int)(reinterpret_cast<uintptr_t>(in) & 15u) / es;
    const long long n = t.e[i].n;
    const long long v0 = (long long)(at - t.first[i]) * (VECS * kThreads) + threadIdx.x;
    uint4 raw[VECS];
    bool whole[VECS];
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const long long lo = (v0 + j * kThreads) * per - head;   // first element of the vector
      whole[j] = lo >= 0 && lo + per <= n;
      if (whole[j]) raw[j] = __ldg(reinterpret_cast<const uint4*>(in + lo * es));
    }
    float part[VECS / 4] = {};
    float x[8];
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      float& s = part[j / 4];
      if (whole[j]) {
        unpack(raw[j], type, x);
#pragma unroll
        for (int k = 0; k < 8; ++k) s = fmaf(x[k], x[k], s);
      } else {
        const long long lo = (v0 + j * kThreads) * per - head;
        for (int k = 0; k < per; ++k)
          if (lo + k >= 0 && lo + k < n) {
            const float e = elem_f32(in, lo + k, type);
            s = fmaf(e, e, s);
          }
      }
    }
    bool plain[VECS / 4], all = true;
#pragma unroll
    for (int q = 0; q < VECS / 4; ++q) {
      plain[q] = part[q] > 1e-30f && part[q] < 1e37f;
      if (plain[q]) total += (double)part[q];
      all = all && plain[q];
    }
    if (!all) {
      // squares near the ends of FP32's range, or below it (or no numbers): in
      // FP64, but for vectors of zeros and those beyond the tensor
      const uint32_t value_bits = type == SGEMM_TYPE_F32 ? 0x7fffffffu : 0x7fff7fffu;
      unsigned left = 0;
#pragma unroll
      for (int j = 0; j < VECS; ++j)
        if (!plain[j / 4] &&
            (whole[j] ? ((raw[j].x | raw[j].y | raw[j].z | raw[j].w) & value_bits) != 0u
                      : (v0 + j * kThreads) * per - head < n))
          left |= 1u << j;
      for (; left != 0u; left &= left - 1) {
        const long long lo = (v0 + (__ffs(left) - 1) * kThreads) * per - head;
        for (int k = 0; k < per; ++k)
          if (lo + k >= 0 && lo + k < n) {
            const double e = (double)elem_f32(in, lo + k, type);
            total += e * e;
          }
      }
    }
  }
  const double s = block_sum(total, buf);
  if (threadIdx.x == 0) sums[blockIdx.x] = s;
}

template <int CAP, int VECS>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(VECS))
    scale_kernel(const __grid_constant__ Table<CAP> t, const double* sums, int nsums,
                 float max_norm, float* norm) {
  __shared__ double buf[kThreads / 32];
  __shared__ float coef_s;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  // from the end: what the first pass read last is still in L2 (1 % of the call
  // at 400 M bf16 values)
  int i = -1;
  uint4 raw[VECS];
  bool whole[VECS];
  // loads the whole vectors of the piece that is `left` from the end
  auto load = [&](unsigned left) {
    const unsigned at = t.pieces - 1 - left;
    i = find(t, at, i);
    const int es = elem_size(t.type[i]), per = 16 / es;
    const char* in = static_cast<const char*>(t.e[i].in);
    const int head = (int)(reinterpret_cast<uintptr_t>(in) & 15u) / es;
    const long long v0 = (long long)(at - t.first[i]) * (VECS * kThreads) + threadIdx.x;
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const long long lo = (v0 + j * kThreads) * per - head;
      whole[j] = lo >= 0 && lo + per <= t.e[i].n;
      if (whole[j]) raw[j] = *reinterpret_cast<const uint4*>(in + lo * es);
    }
  };
  // the first piece is on its way while the norm is formed
  const bool writes = t.count > 0 && t.e[0].out != nullptr;
  if (writes && blockIdx.x < t.pieces) load(blockIdx.x);
  double v = 0.0;
  for (int k = threadIdx.x; k < nsums; k += kThreads) v += __ldcg(sums + k);
  v = block_sum(v, buf);
  if (threadIdx.x == 0) {
    const float nrm = (float)sqrt(v);
    float c = max_norm / (nrm + 1e-6f);
    if (c > 1.f) c = 1.f;      // (a NaN stays)
    coef_s = c;
    if (blockIdx.x == 0 && norm != nullptr) *norm = nrm;
  }
  __syncthreads();
  const float coef = coef_s;
  if (!writes || (coef == 1.f && t.in_place)) return;
  for (unsigned left = blockIdx.x; left < t.pieces; left += gridDim.x) {
    if (left != blockIdx.x) load(left);
    const unsigned at = t.pieces - 1 - left;
    const int type = t.type[i], es = elem_size(type), per = 16 / es;
    const char* in = static_cast<const char*>(t.e[i].in);
    char* out = static_cast<char*>(t.e[i].out);
    if (coef == 1.f && out == in) continue;
    const int head = (int)(reinterpret_cast<uintptr_t>(in) & 15u) / es;
    const bool same = ((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
    const long long n = t.e[i].n;
    const long long v0 = (long long)(at - t.first[i]) * (VECS * kThreads) + threadIdx.x;
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const long long lo = (v0 + j * kThreads) * per - head;
      if (whole[j]) {
        float x[8];
        unpack(raw[j], type, x);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] *= coef;
        if (same) {
          *reinterpret_cast<uint4*>(out + lo * es) = pack(x, type);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < per) put_elem(out, lo + k, type, x[k]);
        }
      } else {
        for (int k = 0; k < per; ++k)
          if (lo + k >= 0 && lo + k < n)
            put_elem(out, lo + k, type, elem_f32(in, lo + k, type) * coef);
      }
    }
  }
}

template <int CAP>
Table<CAP> fill(int vecs, int from, int to, const void* const* in, void* const* out, const long long* sizes,
                const int* types) {
  Table<CAP> t;
  t.count = 0;
  t.in_place = true;
  unsigned pieces = 0;
  for (int i = from; i < to; ++i) {
    if (sizes[i] == 0) continue;
    const int es = types[i] == SGEMM_TYPE_F32 ? 4 : 2;
    const long long bytes = sizes[i] * es + (long long)(reinterpret_cast<uintptr_t>(in[i]) & 15u);
    t.e[t.count] = Entry{in[i], out == nullptr ? nullptr : out[i], sizes[i]};
    t.in_place = t.in_place && out != nullptr && out[i] == in[i];
    t.first[t.count] = pieces;
    t.type[t.count] = (unsigned char)types[i];
    pieces += (unsigned)((bytes + piece_bytes(vecs) - 1) / piece_bytes(vecs));
    ++t.count;
  }
  t.pieces = pieces;
  return t;
}

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), int grid, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  lc.gridDim = dim3((unsigned)grid);
  lc.blockDim = dim3(kThreads);
  lc.stream = stream;
  lc.attrs = la;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, static_cast<KArgs>(args)...);
}

}  // namespace
}  // namespace sgemm_gb300

using namespace sgemm_gb300;

SGEMM_API int sgemm_grad_clip(int n, const void* const* grads, void* const* out,
                              const long long* sizes, const int* types, float max_norm, float* norm,
                              void* stream_) {
  if (n < 0) return SGEMM_ERR_INVALID_DIM;
  if (!(max_norm >= 0.f)) return SGEMM_ERR_INVALID_VALUE;
  if (n > 0 && (grads == nullptr || sizes == nullptr || types == nullptr))
    return SGEMM_ERR_NULL_PTR;
  if (norm == nullptr && out == nullptr) return SGEMM_ERR_NULL_PTR;
  long long bytes = 0;
  for (int i = 0; i < n; ++i) {
    if (types[i] != SGEMM_TYPE_F32 && types[i] != SGEMM_TYPE_BF16 && types[i] != SGEMM_TYPE_F16)
      return SGEMM_ERR_INVALID_VALUE;
    if (sizes[i] < 0 || sizes[i] > (1LL << 40)) return SGEMM_ERR_INVALID_DIM;
    if (sizes[i] == 0) continue;
    if (grads[i] == nullptr || (out != nullptr && out[i] == nullptr)) return SGEMM_ERR_NULL_PTR;
    const uintptr_t mask = types[i] == SGEMM_TYPE_F32 ? 3u : 1u;
    if ((reinterpret_cast<uintptr_t>(grads[i]) & mask) ||
        (out != nullptr && (reinterpret_cast<uintptr_t>(out[i]) & mask)))
      return SGEMM_ERR_MISALIGNED;
    bytes += sizes[i] * (types[i] == SGEMM_TYPE_F32 ? 4 : 2) + piece_bytes(4);
    if (bytes > (1LL << 44)) return SGEMM_ERR_INVALID_DIM;   // the piece numbers are 32 bits
  }
  if (reinterpret_cast<uintptr_t>(norm) & 3u) return SGEMM_ERR_MISALIGNED;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return SGEMM_ERR_LAUNCH;
  }
  int st = library_device_sms(dev, &sms);
  if (st != SGEMM_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);

  const int lists = n > 0 ? (n + kTable - 1) / kTable : 1;
  const int wide = bytes >= kLarge ? 8 : 4;   // vectors a piece of the first pass
  const size_t most = (size_t)lists * sms * ctas_per_sm(4);
  float* ws = nullptr;
  int* status = nullptr;
  const std::unique_lock<std::mutex> lock = library_lock();   // to the last launch
  st = library_workspace(dev, stream, most * 2, 0, &ws, &status, nullptr, nullptr,
                         nullptr);
  if (st != SGEMM_OK) return st;
  double* sums = reinterpret_cast<double*>(ws);
  // the first launches write their sums one list after another
  int nsums = 0;
  auto grid_of = [&](unsigned pieces, int vecs) {
    const unsigned fit = (unsigned)(sms * ctas_per_sm(vecs));
    return pieces < 1 ? 1 : (int)(pieces < fit ? pieces : fit);
  };
  auto squares = [&](const auto& t, auto* kernel) {
    const int grid = grid_of(t.pieces, wide);
    const cudaError_t r = launch(kernel, grid, stream, t, sums + nsums);
    nsums += grid;
    return r;
  };
  auto scale = [&](const auto& t, auto* kernel) {
    return launch(kernel, out == nullptr ? 1 : grid_of(t.pieces, 4), stream, t,
                  (const double*)sums, nsums, max_norm, norm);
  };
  cudaError_t e = cudaSuccess;
  for (int pass = 0; pass < 2; ++pass)
    for (int l = 0; l < lists && e == cudaSuccess; ++l) {
      const int from = l * kTable, to = from + kTable < n ? from + kTable : n;
      const int vecs = pass == 0 ? wide : 4;
      if (to - from <= 64) {
        const auto t = fill<64>(vecs, from, to, grads, out, sizes, types);
        e = pass == 0 ? squares(t, wide == 8 ? squares_kernel<64, 8> : squares_kernel<64, 4>)
                      : scale(t, scale_kernel<64, 4>);
      } else {
        const auto t = fill<kTable>(vecs, from, to, grads, out, sizes, types);
        e = pass == 0
                ? squares(t, wide == 8 ? squares_kernel<kTable, 8> : squares_kernel<kTable, 4>)
                : scale(t, scale_kernel<kTable, 4>);
      }
    }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return SGEMM_ERR_LAUNCH;
  }
  return SGEMM_OK;
}
