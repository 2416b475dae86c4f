// rms_norm.cu -- sgemm_rms_norm, sgemm_rms_norm_i8 and sgemm_rms_norm_grad:
// the residual's addition and the root-mean-square norm of its rows, with an
// output in the input's type or in 8-bit integers with a scale a row, and the
// gradients.
//
// Mathematics, a row of N values at a time:
//   h = x + r, rounded to the type of x (the sum that the next layer adds to)
//   rstd = 1 / sqrt(mean(h^2) + eps),  n = h rstd
//   y = n w
//   8 bits: u = h w in FP32, step = max|u| / 127, q = rint(u / step), scale =
//     step rstd. The factor rstd is common to a row, so q does not depend on
//     it (nor on the order of its sum), and one pass over the row gives both
//     the sum of squares and the maximum.
//   gradients of y and h (dy, dh):  dn = dy w,  c = mean(dn n),
//     dx = dr = rstd (dn - n c) + dh,  dw = sum over rows of dy n.
//
// Bound by DRAM, less what a row's chain of loads, block-wide sum and stores leaves
// idle. Measured on GB300, 8192 x 4096 BF16 with a residual (a copy runs at 6.8
// TB/s): y 43.7 us, 6.1 TB/s; 8 bits 43.3 us, 5.4 TB/s (a value takes 29
// instructions, 61 % of the issue slots); gradients 48.4 us, 5.5 TB/s, the sum of
// dw's parts 5 of them. One row of 4096: 4.2 us. Of the forms tried: element by
// element instead of words 70 us (8 bits); no row ahead 118; rows of 16-byte copies
// three deep in shared memory 57 (8 bits), 46 (y), 70 (gradients, whose weight then
// no longer stays in L1); 256 threads a row at 64 registers 55, 43.6.
#include <cuda_runtime.h>
#include <cmath>
#include <mutex>
#include <stdint.h>

#include "../../include/sgemm_gb300.h"
#include "elements.cuh"
#include "ptx.cuh"

#define SGEMM_API extern "C" __attribute__((visibility("default")))

namespace sgemm_gb300 {

int library_device_sms(int dev, int* sms);
std::unique_lock<std::mutex> library_lock();
int library_workspace(int dev, cudaStream_t stream, size_t floats, size_t nflags, float** scratch,
                      int** status, uint32_t** flags, uint32_t* epoch, uint32_t** counters);

namespace rows {
namespace {

constexpr int kMaxThreads = 512;
// Pieces of a row that a thread holds: of 16 bytes, or single elements.
__host__ __device__ constexpr int held_of(int vw) { return vw > 1 ? 4 : 8; }
constexpr uint32_t kAll = 0xffffffffu;

struct NormArgs {
  int M, N;
  const void *x, *r, *w;   // r: null without a residual
  long long ldx, ldr;
  void* h;                 // null: not stored (then r is null)
  long long ldh;
  void* y;                 // E, or signed char (8 bits)
  long long ldy;
  float* rstd;             // may be null
  float* scale;            // 8 bits
  float eps;
  int wide_q;              // 8 bits: rows of q aligned to a piece's integers
};

// Sum and maximum over the block, the same in every thread and in a fixed
// order. `buf` alternates between the two halves of the array from one call to
// the next, so one barrier a call is enough.
struct Reduced {
  float sum;
  uint32_t most;
};
template <bool MOST>
__device__ __forceinline__ Reduced reduce(float sum, uint32_t most, float2 (*part)[kMaxThreads / 32],
                                          int& buf) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
  if (MOST) most = __reduce_max_sync(kAll, most);
  const int warps = (int)blockDim.x >> 5;
  if (warps == 1) return {sum, most};
  if ((threadIdx.x & 31) == 0)
    part[buf][threadIdx.x >> 5] = make_float2(sum, __uint_as_float(most));
  __syncthreads();
  sum = 0.f;
  most = 0;
  for (int i = 0; i < warps; ++i) {
    const float2 p = part[buf][i];
    sum += p.x;
    if (MOST) most = max(most, __float_as_uint(p.y));
  }
  buf ^= 1;
  return {sum, most};
}

// q = rint(u / step), the quotient rounded to FP32 first, in the low bytes of
// b. u * inv, inv = 1 / step, is within 2^-22 of the quotient (relative; |u /
// step| <= 127), so the two round to the same integer unless the product lies
// that near to the middle of two. Adding 1.5 * 2^23 rounds to the nearest
// integer, ties to even, and leaves it in the sum's low byte. Where one value of
// the piece lies near a middle (or 1 / step is no number to multiply by, or u
// is none), all are divided.
template <int VW>
__device__ __forceinline__ void quotients(const float (&u)[VW], float step, float inv,
                                          uint32_t (&b)[VW]) {
  constexpr float kMagic = 12582912.f;
  bool near = false;
#pragma unroll
  for (int j = 0; j < VW; ++j) {
    const float v = u[j] * inv, t = v + kMagic;
    near = near || !(fabsf(v - (t - kMagic)) <= 0.5f - 1e-4f);
    b[j] = __float_as_uint(t);
  }
  if (near) {
#pragma unroll
    for (int j = 0; j < VW; ++j)
      // (a step below FP32's normal numbers may be far below max|u| / 127)
      b[j] = (uint32_t)__float2int_rn(fminf(fmaxf(__fdiv_rn(u[j], step), -127.f), 127.f));
  }
}

// Factor of the values of rows whose squares FP32 does not hold (a sum above 3e38). The
// largest, below 2^128, have squares below 2^76 with it, 2^31 of which still add up; the
// smallest such row, 2^31 values of 4e14, has squares of 1e-25. (With 2^-70 rows of 4096
// values of 3e38 were beyond FP32 once more.)
constexpr float kDown = 0x1p-90f;

// What a row's integers are divided by.
struct Step {
  float step, inv;     // 1 / step, where that is a number to multiply by (else no number)
  bool none;           // a row of zeros, or with no numbers: its integers are 0
};
__device__ __forceinline__ Step step_of(uint32_t most) {
  Step s;
  s.step = __fdiv_rn(__uint_as_float(most), 127.f);
  s.inv = s.step > 1e-37f ? __frcp_rn(s.step) : __uint_as_float(0x7fc00000u);
  s.none = !(s.step > 0.f && s.step <= 3e38f);
  return s;
}

// The integers of a piece; `wide`: q is aligned to as many bytes. Of the VW those
// from `first` on and before `end` are the row's.
template <int VW>
__device__ __forceinline__ void put_quotients(const float (&u)[VW], const Step& s, signed char* q,
                                              int wide, int first = 0, int end = VW) {
  uint32_t b[VW];
#pragma unroll
  for (int j = 0; j < VW; ++j) b[j] = 0u;
  if (!s.none) quotients<VW>(u, s.step, s.inv, b);
  if (VW > 1 && wide) {
    uint32_t o[VW / 4 > 0 ? VW / 4 : 1];
#pragma unroll
    for (int j = 0; j < VW / 4; ++j)
      o[j] = __byte_perm(__byte_perm(b[4 * j], b[4 * j + 1], 0x0040),
                         __byte_perm(b[4 * j + 2], b[4 * j + 3], 0x0040), 0x5410);
    if constexpr (VW == 8)
      *reinterpret_cast<uint2*>(q) = make_uint2(o[0], o[1]);
    else
      *reinterpret_cast<uint32_t*>(q) = o[0];
  } else {
#pragma unroll
    for (int j = 0; j < VW; ++j)
      if (j >= first && j < end) q[j] = (signed char)(b[j] & 0xffu);
  }
}

// Rows that do not start on 16 bytes (SHIFT), all of the call's matrices alike: the
// places of a row count from the boundary before it, so that all of its pieces but
// the first and the last are whole. The rows of a block (of a group of lanes, in the
// kernels for short rows) start at the same place after a boundary, as the
// host takes rows that are a multiple of 16 bytes apart; so a block's weights are
// laid out once, in shared memory, the way its pieces lie. 8192 x 4097 BF16: y 55 us,
// 8 bits 72, gradients 93; by single elements 124, 161 and 200.
template <typename W>
__device__ __forceinline__ const W* lay_out(const W* w, unsigned first, unsigned end, unsigned places) {
  extern __shared__ uint4 weights[];
  W* out = reinterpret_cast<W*>(weights);
  for (unsigned c = threadIdx.x; c < places; c += blockDim.x)
    out[c] = c >= first && c < end ? w[c - first] : from_f32<W>(0.f);
  __syncthreads();
  return out;
}

// Brings n elements of a row into L2 (but for parts of 16 bytes at its ends), for
// a thread to call: of the rows that a block takes next what it has no registers to
// load ahead. 4096 x 12288 FP32: y 154 to 126 us, 8 bits 148 to 116; gradients of 8192 x
// 7168, FP32 157 to 139 and BF16 95 to 83.
template <typename E>
__device__ __forceinline__ void to_l2(const E* row, unsigned n) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(row), from = (at + 15) & ~(uintptr_t)15,
                  to = (at + (unsigned long long)n * sizeof(E)) & ~(uintptr_t)15;
  if (to > from) ptx::prefetch_l2(reinterpret_cast<const void*>(from), (uint32_t)(to - from));
}

// A row per block, in pieces of VW elements (16 bytes, or one element where
// something is not aligned). Up to HELD pieces a thread stay in registers between
// the pass that sums and the pass that writes, and those of the block's next row
// are loaded ahead; what is left of a longer row is read again (the thread's own
// h, or x).
template <typename E, typename W, int VW, bool I8, bool SHIFT>
__global__ void __launch_bounds__(kMaxThreads) norm_kernel(const NormArgs a) {
  constexpr int HELD = held_of(VW);
  __shared__ float2 part[2][kMaxThreads / 32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const E* x = static_cast<const E*>(a.x);
  const E* r = static_cast<const E*>(a.r);
  const W* w = static_cast<const W*>(a.w);
  E* h = static_cast<E*>(a.h);
  // the row's elements are at places s .. N - 1
  // (places in a row pass 2^31 before they end their loops, not 2^32)
  const unsigned s = SHIFT ? start_of<E>(a.x, blockIdx.x, a.ldx) : 0u;
  const unsigned step_c = blockDim.x * VW, c0 = threadIdx.x * VW, N = (unsigned)a.N + s;
  if (SHIFT) w = lay_out(w, s, N, (N + VW - 1) / VW * VW);
  const float inv_n = 1.f / (float)a.N;
  int buf = 0;
  Piece<E, VW> held[HELD], ahead[HELD];      // x, then h; the residual
  auto inner = [&](long long m) { return inner_row(m, a.M, a.N, VW); };
  auto cleaned = [&](const Piece<E, VW>& p, unsigned c) { return clean<E, VW, SHIFT>(p, c, s, N); };
  auto fetch = [&](long long m) {
    const bool in = inner(m);
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const unsigned c = c0 + i * step_c;
      if (c >= N) continue;
      held[i] = load_at<E, VW, SHIFT>(x + m * a.ldx - s, c, s, N, in);
      if (r != nullptr) ahead[i] = load_at<E, VW, SHIFT>(r + m * a.ldr - s, c, s, N, in);
    }
  };
  auto sum_of = [&](const Piece<E, VW>& p, const Piece<E, VW>& q) {
    float f[VW], g[VW];
    unpack(p, f);
    unpack(q, g);
#pragma unroll
    for (int j = 0; j < VW; ++j) f[j] += g[j];
    return pack<E, VW>(f);
  };
  fetch(blockIdx.x);
  for (long long m = blockIdx.x; m < a.M; m += gridDim.x) {
    float sum = 0.f;
    uint32_t most = 0;
    auto add = [&](const Piece<E, VW>& p, unsigned c) {
      if (h != nullptr) store_at<E, VW, SHIFT>(h + m * a.ldh - s, c, s, N, p);
      float f[VW], t = 0.f;
      unpack(p, f);
#pragma unroll
      for (int j = 0; j < VW; ++j) t = fmaf(f[j], f[j], t);
      sum += t;
      if (I8) {
        float v[VW];
        load_vector<W, VW, SHIFT>(w + c, v);
        // as bits: a NaN is above infinity, so either survives
#pragma unroll
        for (int j = 0; j < VW; ++j)
          most = max(most, __float_as_uint(f[j] * v[j]) & 0x7fffffffu);
      }
    };
    Piece<E, VW> row[HELD];
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      row[i] = cleaned(r != nullptr ? sum_of(held[i], ahead[i]) : held[i], c0 + i * step_c);
    const long long next = m + gridDim.x;
    if (next < a.M) {
      fetch(next);
      // (what is not held; for rows that are, a second one ahead cost up to 5 %)
      if (HELD * step_c < N && threadIdx.x < 2 && (threadIdx.x == 0 || r != nullptr))
        to_l2((threadIdx.x == 0 ? x + next * a.ldx : r + next * a.ldr) + (HELD * step_c - s),
              N - HELD * step_c);
    }
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (c0 + i * step_c < N) add(row[i], c0 + i * step_c);
    for (unsigned c = c0 + HELD * step_c; c < N; c += step_c) {
      Piece<E, VW> p = load_at<E, VW, SHIFT>(x + m * a.ldx - s, c, s, N, inner(m));
      if (r != nullptr) p = sum_of(p, load_at<E, VW, SHIFT>(r + m * a.ldr - s, c, s, N, inner(m)));
      add(cleaned(p, c), c);
    }
    // the row's values once more: those that were not held from h, or x
    auto each = [&](auto&& f) {
#pragma unroll
      for (int i = 0; i < HELD; ++i)
        if (c0 + i * step_c < N) f(row[i], c0 + i * step_c);
      for (unsigned c = c0 + HELD * step_c; c < N; c += step_c)
        f(cleaned(load_at<E, VW, SHIFT>((h != nullptr ? h + m * a.ldh : x + m * a.ldx) - s, c, s, N,
                                        inner(m)), c), c);
    };
    Reduced t = reduce<I8>(sum, most, part, buf);
    // Squares beyond FP32's range (values above 1e19): once more on values that
    // are scaled down. eps is at least 1e-30, so squares below the range do not count.
    float down = 1.f;
    if (!(t.sum <= 3e38f)) {
      down = kDown;
      sum = 0.f;
      each([&](const Piece<E, VW>& p, unsigned) {
        float f[VW];
        unpack(p, f);
#pragma unroll
        for (int j = 0; j < VW; ++j) sum = fmaf(f[j] * down, f[j] * down, sum);
      });
      t.sum = reduce<false>(sum, 0, part, buf).sum;
    }
    // (below FP32's normal numbers where the values are above 8e37: 21 bits are left)
    const float rstd = rsqrtf(t.sum * inv_n + a.eps * down * down) * down;
    if (threadIdx.x == 0 && a.rstd != nullptr) a.rstd[m] = rstd;
    if (!I8) {
      E* y = static_cast<E*>(a.y) + m * a.ldy - s;
      each([&](const Piece<E, VW>& p, unsigned c) {
        float v[VW], f[VW];
        load_vector<W, VW, SHIFT>(w + c, v);
        unpack(p, f);
#pragma unroll
        for (int j = 0; j < VW; ++j) f[j] = f[j] * rstd * v[j];
        store_at<E, VW, SHIFT>(y, c, s, N, pack<E, VW>(f));
      });
    } else {
      const Step step = step_of(t.most);
      if (threadIdx.x == 0) a.scale[m] = step.step * rstd;
      signed char* q = static_cast<signed char*>(a.y) + m * a.ldy - s;
      each([&](const Piece<E, VW>& p, unsigned c) {
        float u[VW], f[VW];
        load_vector<W, VW, SHIFT>(w + c, u);
        unpack(p, f);
#pragma unroll
        for (int j = 0; j < VW; ++j) u[j] *= f[j];
        put_quotients<VW>(u, step, q + c, a.wide_q, SHIFT ? (int)(s - c) : 0, SHIFT ? (int)(N - c) : VW);
      });
    }
  }
}

struct GradArgs {
  int M, N;
  const void *dy, *h, *w, *dh;   // dh: may be null
  long long lddy, ldh, lddh;
  const float* rstd;
  void* dx;                      // may be null
  long long lddx;
  float* partial;                // gridDim.x rows of N sums for dw; null: not formed here
};

// A row per block at a time, every thread at the same places in each, so that
// its part of dw stays in registers over all rows of the block. DW: the row
// fits into HELD pieces a thread and dw's parts are formed.
// HELD 2 (rows of at most 512 pieces): the next row's loads are ahead, on 256
// threads; more pieces, and their sums, leave no registers for that, and the next
// row comes into L2. (Rows over the blocks of a cluster, two pieces a thread and two
// ahead: 2048 x 16384 BF16 84 us, this way 60.)
template <typename E, typename W, int VW, int HELD, bool DW, bool SHIFT>
__global__ void __launch_bounds__(HELD == 2 ? 256 : kMaxThreads, HELD == 2 ? 2 : 1)
    norm_grad_kernel(const GradArgs a) {
  constexpr bool kAhead = HELD == 2;
  __shared__ float2 part[2][kMaxThreads / 32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const E* dy = static_cast<const E*>(a.dy);
  const E* h = static_cast<const E*>(a.h);
  const E* dh = static_cast<const E*>(a.dh);
  const W* w = static_cast<const W*>(a.w);
  E* dx = static_cast<E*>(a.dx);
  const unsigned s = SHIFT ? start_of<E>(a.dy, blockIdx.x, a.lddy) : 0u;   // as in norm_kernel
  const unsigned step_c = blockDim.x * VW, c0 = threadIdx.x * VW, N = (unsigned)a.N + s;
  if (SHIFT) w = lay_out(w, s, N, (N + VW - 1) / VW * VW);
  const float inv_n = 1.f / (float)a.N;
  int buf = 0;
  float dw[DW ? HELD : 1][VW];
#pragma unroll
  for (int i = 0; i < (DW ? HELD : 1); ++i)
#pragma unroll
    for (int j = 0; j < VW; ++j) dw[i][j] = 0.f;
  Piece<E, VW> g1[HELD], v1[HELD], d1[HELD];
  float rstd1 = 0.f;
  auto get = [&](const E* p, long long ld, long long m, unsigned c) {
    return load_at<E, VW, SHIFT>(p + m * ld - s, c, s, N, inner_row(m, a.M, a.N, VW));
  };
  auto cleaned = [&](const Piece<E, VW>& p, unsigned c) { return clean<E, VW, SHIFT>(p, c, s, N); };
  auto fetch = [&](long long m) {
    rstd1 = a.rstd[m];
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const unsigned c = c0 + i * step_c;
      if (c >= N) continue;
      g1[i] = get(dy, a.lddy, m, c);
      v1[i] = get(h, a.ldh, m, c);
      if (dh != nullptr) d1[i] = get(dh, a.lddh, m, c);
    }
  };
  if (kAhead) fetch(blockIdx.x);
  for (long long m = blockIdx.x; m < a.M; m += gridDim.x) {
    if (!kAhead) fetch(m);
    const float rstd = rstd1;
    Piece<E, VW> g[HELD], v[HELD], d[HELD];
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      g[i] = cleaned(g1[i], c0 + i * step_c);
      v[i] = cleaned(v1[i], c0 + i * step_c);
      d[i] = d1[i];
    }
    const long long next = m + gridDim.x;
    if (next < a.M) {
      if (kAhead) {
        fetch(next);
      } else if (threadIdx.x < 3 && (threadIdx.x < 2 || dh != nullptr)) {
        to_l2(threadIdx.x == 0   ? dy + next * a.lddy
              : threadIdx.x == 1 ? h + next * a.ldh
                                 : dh + next * a.lddh,
              (unsigned)a.N);
      }
    }
    float sum = 0.f;
    auto add = [&](const Piece<E, VW>& g, const Piece<E, VW>& v, unsigned c) {
      float wv[VW], gf[VW], vf[VW], t = 0.f;
      load_vector<W, VW, SHIFT>(w + c, wv);
      unpack(g, gf);
      unpack(v, vf);
#pragma unroll
      for (int j = 0; j < VW; ++j) t = fmaf(gf[j] * wv[j], vf[j] * rstd, t);
      sum += t;
    };
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const unsigned c = c0 + i * step_c;
      if (c >= N) continue;
      add(g[i], v[i], c);
      if (DW) {
        float gf[VW], vf[VW];
        unpack(g[i], gf);
        unpack(v[i], vf);
#pragma unroll
        for (int j = 0; j < VW; ++j) dw[i][j] = fmaf(gf[j], vf[j] * rstd, dw[i][j]);
      }
    }
    if (!DW)
      for (unsigned c = c0 + HELD * step_c; c < N; c += step_c)
        add(cleaned(get(dy, a.lddy, m, c), c), cleaned(get(h, a.ldh, m, c), c), c);
    if (dx == nullptr) continue;
    const float mean = reduce<false>(sum, 0, part, buf).sum * inv_n;
    auto put = [&](const Piece<E, VW>& g, const Piece<E, VW>& v, const Piece<E, VW>& d, unsigned c) {
      float wv[VW], gf[VW], vf[VW], df[VW];
      load_vector<W, VW, SHIFT>(w + c, wv);
      unpack(g, gf);
      unpack(v, vf);
      unpack(d, df);
#pragma unroll
      for (int j = 0; j < VW; ++j) {
        const float t = rstd * fmaf(-mean, vf[j] * rstd, gf[j] * wv[j]);
        gf[j] = dh != nullptr ? t + df[j] : t;
      }
      store_at<E, VW, SHIFT>(dx + m * a.lddx - s, c, s, N, pack<E, VW>(gf));
    };
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (c0 + i * step_c < N) put(g[i], v[i], d[i], c0 + i * step_c);
    if (!DW)
      for (unsigned c = c0 + HELD * step_c; c < N; c += step_c)
        put(get(dy, a.lddy, m, c), get(h, a.ldh, m, c),
            dh != nullptr ? get(dh, a.lddh, m, c) : Piece<E, VW>{}, c);
  }
  if (DW && a.partial != nullptr) {
    float* p = a.partial + (long long)blockIdx.x * a.N;
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const unsigned c = c0 + i * step_c;
      if (c >= N) continue;
      if constexpr (VW == 1) {
        p[c] = dw[i][0];
      } else if constexpr (SHIFT) {
#pragma unroll
        for (int j = 0; j < VW; ++j)
          if (c + j >= s && c + j < N) p[c + j - s] = dw[i][j];
      } else {
#pragma unroll
        for (int j = 0; j < VW; j += 4)
          *reinterpret_cast<float4*>(p + c + j) =
              make_float4(dw[i][j], dw[i][j + 1], dw[i][j + 2], dw[i][j + 3]);
      }
    }
  }
}

// Short rows, of at most 32 pieces of 16 bytes: a row is one piece each of `lanes`
// (8, 16 or 32) neighbouring threads, and its sums go over them alone. (1048576
// rows of 128 BF16: 104 us, back 178, of 79 and 118 that the bytes take; by a block
// a row 324 and 330. 8192 rows of 64: 1.9 and 4.0 us instead of 4.4 and 11.5.)
constexpr int kSmallThreads = 256;
__device__ __forceinline__ float sum_over(float v, int lanes) {
  for (int d = lanes >> 1; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}
template <typename E, typename W, int VW, bool I8, bool SHIFT>
__global__ void __launch_bounds__(kSmallThreads) small_norm_kernel(const NormArgs a, int lanes) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int rows = kSmallThreads / lanes, l = threadIdx.x & (lanes - 1), group = threadIdx.x / lanes;
  // (a group's rows are a multiple of 8 apart: all start at the same place)
  const unsigned s = SHIFT ? start_of<E>(a.x, (long long)blockIdx.x * rows + group, a.ldx) : 0u;
  const unsigned c = l * VW, N = (unsigned)a.N + s;
  const float inv_n = 1.f / (float)a.N;
  float w[VW];
#pragma unroll
  for (int j = 0; j < VW; ++j) w[j] = 0.f;
  if constexpr (SHIFT) {
#pragma unroll
    for (int j = 0; j < VW; ++j)
      if (c + j >= s && c + j < N) w[j] = to_f32(__ldg(static_cast<const W*>(a.w) + (c + j - s)));
  } else if (c < N) {
    load_vector<W, VW>(static_cast<const W*>(a.w) + c, w);
  }
  // (the same number of steps for every thread: they exchange sums)
  for (long long m0 = (long long)blockIdx.x * rows; m0 < a.M; m0 += (long long)gridDim.x * rows) {
    const long long m = m0 + group;
    const bool live = m < a.M && c < N, inner = inner_row(m, a.M, a.N, VW);
    float f[VW], u[VW];
#pragma unroll
    for (int j = 0; j < VW; ++j) f[j] = 0.f;
    if (live) {
      Piece<E, VW> p = load_at<E, VW, SHIFT>(static_cast<const E*>(a.x) + m * a.ldx - s, c, s, N, inner);
      p = clean<E, VW, SHIFT>(p, c, s, N);
      unpack(p, f);
      if (a.r != nullptr) {
        unpack(clean<E, VW, SHIFT>(
            load_at<E, VW, SHIFT>(static_cast<const E*>(a.r) + m * a.ldr - s, c, s, N, inner), c, s, N), u);
#pragma unroll
        for (int j = 0; j < VW; ++j) f[j] += u[j];
        p = pack<E, VW>(f);
        unpack(p, f);
        store_at<E, VW, SHIFT>(static_cast<E*>(a.h) + m * a.ldh - s, c, s, N, p);
      }
    }
    float sum = 0.f;
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < VW; ++j) {
      sum = fmaf(f[j], f[j], sum);
      u[j] = f[j] * w[j];
      if (I8 && live) most = max(most, __float_as_uint(u[j]) & 0x7fffffffu);
    }
    sum = sum_over(sum, lanes);
    if (I8)
      for (int d = lanes >> 1; d > 0; d >>= 1) most = max(most, __shfl_xor_sync(kAll, most, d));
    // (squares beyond FP32's range: as in norm_kernel)
    float down = 1.f;
    if (__any_sync(kAll, !(sum <= 3e38f))) {
      float scaled = 0.f;
#pragma unroll
      for (int j = 0; j < VW; ++j) scaled = fmaf(f[j] * kDown, f[j] * kDown, scaled);
      scaled = sum_over(scaled, lanes);
      if (!(sum <= 3e38f)) {
        sum = scaled;
        down = kDown;
      }
    }
    const float rstd = rsqrtf(sum * inv_n + a.eps * down * down) * down;
    if (m < a.M && l == 0 && a.rstd != nullptr) a.rstd[m] = rstd;
    if (!I8) {
      if (!live) continue;
#pragma unroll
      for (int j = 0; j < VW; ++j) f[j] = f[j] * rstd * w[j];
      store_at<E, VW, SHIFT>(static_cast<E*>(a.y) + m * a.ldy - s, c, s, N, pack<E, VW>(f));
    } else {
      const Step step = step_of(most);
      if (m < a.M && l == 0) a.scale[m] = step.step * rstd;
      if (!live) continue;
      put_quotients<VW>(u, step, static_cast<signed char*>(a.y) + m * a.ldy - s + c, a.wide_q,
                        SHIFT ? (int)(s - c) : 0, SHIFT ? (int)(N - c) : VW);
    }
  }
}

template <typename E, typename W, int VW, bool SHIFT>
__global__ void __launch_bounds__(kSmallThreads) small_grad_kernel(const GradArgs a, int lanes) {
  __shared__ float part[kSmallThreads][VW + 1];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int rows = kSmallThreads / lanes, l = threadIdx.x & (lanes - 1), group = threadIdx.x / lanes;
  // (a group's rows are a multiple of 8 apart: all start at the same place)
  const unsigned s = SHIFT ? start_of<E>(a.dy, (long long)blockIdx.x * rows + group, a.lddy) : 0u;
  const unsigned c = l * VW, N = (unsigned)a.N + s;
  const float inv_n = 1.f / (float)a.N;
  float w[VW], dw[VW];
#pragma unroll
  for (int j = 0; j < VW; ++j) w[j] = dw[j] = 0.f;
  if constexpr (SHIFT) {
#pragma unroll
    for (int j = 0; j < VW; ++j)
      if (c + j >= s && c + j < N) w[j] = to_f32(__ldg(static_cast<const W*>(a.w) + (c + j - s)));
  } else if (c < N) {
    load_vector<W, VW>(static_cast<const W*>(a.w) + c, w);
  }
  for (long long m0 = (long long)blockIdx.x * rows; m0 < a.M; m0 += (long long)gridDim.x * rows) {
    const long long m = m0 + group;
    const bool live = m < a.M && c < N, inner = inner_row(m, a.M, a.N, VW);
    float g[VW], n[VW], d[VW], sum = 0.f, rstd = 0.f;
#pragma unroll
    for (int j = 0; j < VW; ++j) g[j] = n[j] = d[j] = 0.f;
    if (live) {
      rstd = a.rstd[m];
      unpack(clean<E, VW, SHIFT>(
          load_at<E, VW, SHIFT>(static_cast<const E*>(a.dy) + m * a.lddy - s, c, s, N, inner), c, s, N), g);
      unpack(clean<E, VW, SHIFT>(
          load_at<E, VW, SHIFT>(static_cast<const E*>(a.h) + m * a.ldh - s, c, s, N, inner), c, s, N), n);
      if (a.dh != nullptr) unpack(load_at<E, VW, SHIFT>(static_cast<const E*>(a.dh) + m * a.lddh - s, c, s, N, inner), d);
#pragma unroll
      for (int j = 0; j < VW; ++j) {
        n[j] *= rstd;
        dw[j] = fmaf(g[j], n[j], dw[j]);
        g[j] *= w[j];
        sum = fmaf(g[j], n[j], sum);
      }
    }
    if (a.dx == nullptr) continue;
    const float mean = sum_over(sum, lanes) * inv_n;
    if (!live) continue;
#pragma unroll
    for (int j = 0; j < VW; ++j) g[j] = rstd * fmaf(-mean, n[j], g[j]) + d[j];
    store_at<E, VW, SHIFT>(static_cast<E*>(a.dx) + m * a.lddx - s, c, s, N, pack<E, VW>(g));
  }
  if (a.partial == nullptr) return;
#pragma unroll
  for (int j = 0; j < VW; ++j) part[threadIdx.x][j] = dw[j];
  __syncthreads();
  for (int i = threadIdx.x; i < a.N; i += kSmallThreads) {
    float sum = 0.f;
    for (int r = 0; r < rows; ++r) {
      const unsigned at = i + (SHIFT ? start_of<E>(a.dy, (long long)blockIdx.x * rows + r, a.lddy) : 0u);
      sum += part[r * lanes + at / VW][at % VW];
    }
    a.partial[(long long)blockIdx.x * a.N + i] = sum;
  }
}

// Rows too long for registers: dw's parts a column a thread, over the rows of a
// slab (slab s has the rows s, s + slabs, ...).
constexpr int kColumnThreads = 256;
template <typename E>
__global__ void __launch_bounds__(kColumnThreads) column_kernel(const GradArgs a, int slabs) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const long long columns = (a.N + kColumnThreads - 1ll) / kColumnThreads;
  for (long long b = blockIdx.x; b < columns * slabs; b += gridDim.x) {
    const long long slab = b / columns, c = (b - slab * columns) * kColumnThreads + threadIdx.x;
    if (c >= a.N) continue;
    const E* dy = static_cast<const E*>(a.dy) + c;
    const E* h = static_cast<const E*>(a.h) + c;
    float sum = 0.f;
#pragma unroll 4
    for (long long m = slab; m < a.M; m += slabs)
      sum = fmaf(to_f32(dy[m * a.lddy]), to_f32(h[m * a.ldh]) * a.rstd[m], sum);
    a.partial[slab * a.N + c] = sum;
  }
}

// dw[c] = sum of the parts in an order of their own: 32 columns a block, 32
// threads a column, each the parts of its residue.
constexpr int kSumLanes = 32;
template <typename W>
__global__ void __launch_bounds__(32 * kSumLanes)
    sum_kernel(const float* partial, int parts, int N, W* dw) {
  __shared__ float s[kSumLanes][32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
  for (long long c0 = blockIdx.x * 32ll; c0 < N; c0 += gridDim.x * 32ll) {
    const long long c = c0 + lane;
    float sum = 0.f;
    if (c < N) {
#pragma unroll 8
      for (int p = group; p < parts; p += kSumLanes) sum += __ldcg(partial + (long long)p * N + c);
    }
    s[group][lane] = sum;
    __syncthreads();
    if (group == 0 && c < N) {
#pragma unroll 8
      for (int g = 1; g < kSumLanes; ++g) sum += s[g][lane];
      dw[c] = from_f32<W>(sum);
    }
    __syncthreads();
  }
}

// Bytes of shared memory for the weights of shifted rows; longer ones are taken by
// single elements.
constexpr int kMostShared = 96 << 10;

// (the limit that is set belongs to the kernel, whoever calls: always the most that any
// call takes, so that no call lowers it between another's setting and its launch)
template <typename... A>
cudaError_t launch(void (*kernel)(A...), long long blocks, int threads, int shared_bytes,
                   cudaStream_t stream, std::common_type_t<A>... args) {
  if (shared_bytes > (32 << 10)) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t lc = {};
  lc.dynamicSmemBytes = (size_t)shared_bytes;
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  lc.gridDim = dim3((unsigned)blocks);
  lc.blockDim = dim3((unsigned)threads);
  lc.stream = stream;
  lc.attrs = la;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, args...);
}

// Threads of a row: a piece each while that leaves SMs idle otherwise (few
// rows: latency), else as many pieces as are held, and what the blocks that fit
// leave (8192 x 4097 FP32 gradients on 288 threads, one block an SM, 173 us; on 512, 151).
int threads_of(long long pieces, int held, bool few) {
  const long long want = few ? pieces : (pieces + held - 1) / held;
  const long long t = (want + 31) / 32 * 32;
  const int n = (int)(t < 32 ? 32 : (t > kMaxThreads ? kMaxThreads : t));
  return few ? n : kMaxThreads / (kMaxThreads / n) / 32 * 32;
}
// Blocks: a row each, or as many as fill the SMs (`threads_per_sm` resident).
int blocks_of(int M, int threads, int sms, int threads_per_sm) {
  const int fit = sms * (threads_per_sm / threads < 32 ? threads_per_sm / threads : 32);
  return M < fit ? M : fit;
}

// Threads of a short row, and blocks of such rows.
int small_lanes(long long pieces) { return pieces <= 8 ? 8 : (pieces <= 16 ? 16 : 32); }
int small_blocks(int M, int lanes, int sms) {
  const int rows = kSmallThreads / lanes;
  const long long blocks = (M + rows - 1ll) / rows;
  return (int)(blocks < sms * 6ll ? blocks : sms * 6ll);
}

bool aligned(const void* p, long long ld, int elem, int bytes) {
  return p == nullptr ||
         ((reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0 && ld * elem % bytes == 0);
}
// Every row of p starts at the same place after a 16-byte boundary as that of x.
bool alike(const void* p, long long ld, const void* x, long long ldx, int elem) {
  return p == nullptr || (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(x)) & 15u) == 0 &&
                          (ld - ldx) * elem % 16 == 0);
}

// How a call's rows are taken: in 16-byte pieces that start with the row, in
// pieces that start at a boundary before it, or by single elements.
enum Access { kPieces, kShifted, kSingle };
// Shifted, unless the weights take too much, or the call is a few rows that threads
// hold by single elements: laying out the weights, and the first and the last row,
// whose ends are read by themselves, take 1 to 2 us (16 x 1001 BF16: 4.0 us, single 2.4;
// 16 x 16383: 10.3 and 15.1).
bool shift(int M, int N, int vw, int weight_bytes, int sms) {
  return (N + 2ll * vw) * weight_bytes <= kMostShared &&
         (M >= 2 * sms || N > held_of(1) * kMaxThreads);
}
// Places of a row in the worst case, in pieces of vw.
long long pieces_of(Access access, int N, int vw) {
  return access == kSingle ? N : (N + (access == kShifted ? vw - 1ll : 0ll) + vw - 1) / vw;
}
int shared_of(Access access, int N, int vw, int weight_bytes) {
  return access == kShifted ? (int)(pieces_of(access, N, vw) * vw * weight_bytes) : 0;
}
// Rows that the 32 threads of a block hold by single elements (up to 256 values) and
// shifted in one more piece than the threads have turns for, most of which are then
// idle: from `from` pieces on, to `to`. y from 33 pieces on: 255 values, 72 MB each of x,
// r, h and y, BF16 shifted 125 us, single 90 (257 values 124 and 166); FP32 129 78 and 62,
// 255 58 and 49. 8 bits to 48: BF16 255 150 and 120, FP32 129 99 and 93, 189 71 and 70,
// 197 68 and 71. Gradients from 65 on: FP32 255 79 and 62 (245 61 and 63, BF16 255 115 and 123).
bool one_warp(int N, int vw, long long from, long long to) {
  const long long pieces = pieces_of(kShifted, N, vw);
  return N <= 32 * held_of(1) && pieces >= from && pieces <= to;
}
// Blocks so that the rows of one, where there are several, are a multiple of 16
// bytes apart.
int spaced(Access access, int M, long long row_bytes, int blocks) {
  int rows = 1;
  while (row_bytes * rows % 16 != 0) rows *= 2;
  if (access != kShifted || blocks >= M) return blocks;
  return blocks >= rows ? blocks / rows * rows : (M < rows ? M : rows);
}

template <typename E, typename W, bool I8>
cudaError_t forward(NormArgs a, int sms, cudaStream_t stream) {
  constexpr int VW = 16 / (int)sizeof(E);
  const bool whole = aligned(a.x, a.ldx, sizeof(E), 16) && aligned(a.r, a.ldr, sizeof(E), 16) &&
                     aligned(a.h, a.ldh, sizeof(E), 16) && aligned(a.w, 0, sizeof(W), 16) &&
                     a.N % VW == 0 && (I8 || aligned(a.y, a.ldy, sizeof(E), 16));
  const bool shifted = alike(a.r, a.ldr, a.x, a.ldx, sizeof(E)) && alike(a.h, a.ldh, a.x, a.ldx, sizeof(E)) &&
                       (I8 || alike(a.y, a.ldy, a.x, a.ldx, sizeof(E))) &&
                       shift(a.M, a.N, VW, sizeof(W), sms) && !one_warp(a.N, VW, 33, I8 ? 48 : 256);
  const Access access = whole ? kPieces : shifted ? kShifted : kSingle;
  a.wide_q = I8 && access != kShifted && aligned(a.y, a.ldy, 1, VW);
  const bool few = a.M < 2 * sms;
  const long long pieces = pieces_of(access, a.N, VW);
  if (access != kSingle && pieces <= 32) {
    const int lanes = small_lanes(pieces);
    return launch(whole ? small_norm_kernel<E, W, VW, I8, false> : small_norm_kernel<E, W, VW, I8, true>,
                  small_blocks(a.M, lanes, sms), kSmallThreads, 0, stream, a, lanes);
  }
  const int t = threads_of(pieces, held_of(access != kSingle ? VW : 1), few);
  return launch(access == kPieces    ? norm_kernel<E, W, VW, I8, false>
                : access == kShifted ? norm_kernel<E, W, VW, I8, true>
                                     : norm_kernel<E, W, 1, I8, false>,
                spaced(access, a.M, a.ldx * (int)sizeof(E), blocks_of(a.M, t, sms, 512)), t,
                shared_of(access, a.N, VW, sizeof(W)), stream, a);
}

// `blocks` make a part of dw each: of norm_grad_kernel where a row is `held` (in so
// many pieces a thread; 1: short rows of `threads` lanes), else (0) slabs of
// column_kernel.
template <typename E, typename W>
cudaError_t backward(GradArgs a, W* dw, float* partial, int blocks, int sms, cudaStream_t stream,
                     int threads, Access access, int held) {
  constexpr int VW = 16 / (int)sizeof(E);
  a.partial = partial;
  cudaError_t e = cudaSuccess;
  if (held == 1) {
    e = launch(access == kShifted ? small_grad_kernel<E, W, VW, true> : small_grad_kernel<E, W, VW, false>,
               blocks, kSmallThreads, 0, stream, a, threads);
  } else if (held != 0) {
    e = launch(access == kSingle    ? norm_grad_kernel<E, W, 1, 8, true, false>
               : access == kPieces ? (held == 2 ? norm_grad_kernel<E, W, VW, 2, true, false>
                                                : norm_grad_kernel<E, W, VW, 4, true, false>)
                                   : (held == 2 ? norm_grad_kernel<E, W, VW, 2, true, true>
                                                : norm_grad_kernel<E, W, VW, 4, true, true>),
               blocks, threads, shared_of(access, a.N, VW, sizeof(W)), stream, a);
  } else {
    // (dw's parts first: dx may take the place of what they are made of)
    if (dw != nullptr) {
      const long long all = (a.N + kColumnThreads - 1ll) / kColumnThreads * blocks;
      e = launch(column_kernel<E>, all < sms * 8ll ? all : sms * 8ll, kColumnThreads, 0, stream, a, blocks);
    }
    if (e == cudaSuccess && a.dx != nullptr)
      e = launch(access == kPieces    ? norm_grad_kernel<E, W, VW, 4, false, false>
                 : access == kShifted ? norm_grad_kernel<E, W, VW, 4, false, true>
                                      : norm_grad_kernel<E, W, 1, 8, false, false>,
                 spaced(access, a.M, a.lddy * (int)sizeof(E), blocks_of(a.M, threads, sms, 512)), threads,
                 shared_of(access, a.N, VW, sizeof(W)), stream, a);
  }
  if (e == cudaSuccess && dw != nullptr) {
    const long long all = (a.N + 31ll) / 32;
    e = launch(sum_kernel<W>, all < sms * 8ll ? all : sms * 8ll, 32 * kSumLanes, 0, stream,
               static_cast<const float*>(partial), blocks, a.N, dw);
  }
  return e;
}

int elem_bytes(int type) { return type == SGEMM_TYPE_F32 ? 4 : 2; }
bool type_ok(int type) {
  return type == SGEMM_TYPE_F32 || type == SGEMM_TYPE_BF16 || type == SGEMM_TYPE_F16;
}
bool misaligned(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) != 0;
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

template <bool I8>
int run_forward(int type, int weight_type, const NormArgs& a, cudaStream_t stream) {
  int sms = 0;
  const int st = device(&sms);
  if (st != SGEMM_OK) return st;
  using B = __nv_bfloat16;
  if (type == SGEMM_TYPE_F32) return done(forward<float, float, I8>(a, sms, stream));
  if (type == SGEMM_TYPE_BF16)
    return done(weight_type == SGEMM_TYPE_F32 ? forward<B, float, I8>(a, sms, stream)
                                              : forward<B, B, I8>(a, sms, stream));
  return done(weight_type == SGEMM_TYPE_F32 ? forward<__half, float, I8>(a, sms, stream)
                                            : forward<__half, __half, I8>(a, sms, stream));
}

// Checks that the three calls share; `ld`s are of the matrices that are given.
int check(int M, int N, int type, int weight_type) {
  if (!type_ok(type) || (weight_type != type && weight_type != SGEMM_TYPE_F32))
    return SGEMM_ERR_INVALID_VALUE;
  return M < 0 || N < 0 ? SGEMM_ERR_INVALID_DIM : SGEMM_OK;
}
bool short_ld(const void* p, int ld, int N) { return p != nullptr && ld < (N > 1 ? N : 1); }
bool eps_ok(float eps) { return eps >= 1e-30f && eps <= 3e38f; }

}  // namespace
}  // namespace rows
}  // namespace sgemm_gb300

using namespace sgemm_gb300;

SGEMM_API int sgemm_rms_norm(int M, int N, int type, const void* X, int ldx, const void* R, int ldr,
                             const void* weight, int weight_type, float eps, void* H, int ldh,
                             void* Y, int ldy, float* rstd, void* stream) {
  int st = rows::check(M, N, type, weight_type);
  if (st != SGEMM_OK) return st;
  if (!rows::eps_ok(eps)) return SGEMM_ERR_INVALID_VALUE;
  const int least = N > 1 ? N : 1;
  if (ldx < least || ldy < least || rows::short_ld(R, ldr, N) || rows::short_ld(H, ldh, N))
    return SGEMM_ERR_INVALID_LD;
  if (M == 0 || N == 0) return SGEMM_OK;
  if (X == nullptr || weight == nullptr || Y == nullptr || (R != nullptr && H == nullptr))
    return SGEMM_ERR_NULL_PTR;
  const int eb = rows::elem_bytes(type);
  if (rows::misaligned(X, eb) || rows::misaligned(R, eb) || rows::misaligned(H, eb) ||
      rows::misaligned(Y, eb) || rows::misaligned(weight, rows::elem_bytes(weight_type)) ||
      rows::misaligned(rstd, 4))
    return SGEMM_ERR_MISALIGNED;
  rows::NormArgs a = {};
  a.M = M;
  a.N = N;
  a.x = X;
  a.ldx = ldx;
  a.r = R;
  a.ldr = ldr;
  a.w = weight;
  a.h = R != nullptr ? H : nullptr;
  a.ldh = ldh;
  a.y = Y;
  a.ldy = ldy;
  a.rstd = rstd;
  a.eps = eps;
  return rows::run_forward<false>(type, weight_type, a, static_cast<cudaStream_t>(stream));
}

SGEMM_API int sgemm_rms_norm_i8(int M, int N, int type, const void* X, int ldx, const void* R,
                                int ldr, const void* weight, int weight_type, float eps, void* H,
                                int ldh, signed char* Q, int ldq, float* scale, void* stream) {
  int st = rows::check(M, N, type, weight_type);
  if (st != SGEMM_OK) return st;
  if (!rows::eps_ok(eps)) return SGEMM_ERR_INVALID_VALUE;
  const int least = N > 1 ? N : 1;
  if (ldx < least || ldq < least || rows::short_ld(R, ldr, N) || rows::short_ld(H, ldh, N))
    return SGEMM_ERR_INVALID_LD;
  if (M == 0 || N == 0) return SGEMM_OK;
  if (X == nullptr || weight == nullptr || Q == nullptr || scale == nullptr ||
      (R != nullptr && H == nullptr))
    return SGEMM_ERR_NULL_PTR;
  const int eb = rows::elem_bytes(type);
  if (rows::misaligned(X, eb) || rows::misaligned(R, eb) || rows::misaligned(H, eb) ||
      rows::misaligned(weight, rows::elem_bytes(weight_type)) || rows::misaligned(scale, 4))
    return SGEMM_ERR_MISALIGNED;
  rows::NormArgs a = {};
  a.M = M;
  a.N = N;
  a.x = X;
  a.ldx = ldx;
  a.r = R;
  a.ldr = ldr;
  a.w = weight;
  a.h = R != nullptr ? H : nullptr;
  a.ldh = ldh;
  a.y = Q;
  a.ldy = ldq;
  a.scale = scale;
  a.eps = eps;
  return rows::run_forward<true>(type, weight_type, a, static_cast<cudaStream_t>(stream));
}

SGEMM_API int sgemm_rms_norm_grad(int M, int N, int type, const void* dY, int lddy, const void* H,
                                  int ldh, const void* weight, int weight_type, const float* rstd,
                                  const void* dH, int lddh, void* dX, int lddx, void* dweight,
                                  void* stream_) {
  int st = rows::check(M, N, type, weight_type);
  if (st != SGEMM_OK) return st;
  const int least = N > 1 ? N : 1;
  if (lddy < least || ldh < least || rows::short_ld(dH, lddh, N) || rows::short_ld(dX, lddx, N))
    return SGEMM_ERR_INVALID_LD;
  if (N == 0 || (dX == nullptr && dweight == nullptr)) return SGEMM_OK;
  if (M > 0 && (dY == nullptr || H == nullptr || weight == nullptr || rstd == nullptr))
    return SGEMM_ERR_NULL_PTR;
  const int eb = rows::elem_bytes(type), wb = rows::elem_bytes(weight_type);
  if (rows::misaligned(dY, eb) || rows::misaligned(H, eb) || rows::misaligned(dH, eb) ||
      rows::misaligned(dX, eb) || rows::misaligned(weight, wb) || rows::misaligned(dweight, wb) ||
      rows::misaligned(rstd, 4))
    return SGEMM_ERR_MISALIGNED;
  int sms = 0, dev = 0;
  st = rows::device(&sms);
  if (st != SGEMM_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (M == 0) {   // no rows: dweight is zero
    if (dweight == nullptr) return SGEMM_OK;
    return rows::done(cudaMemsetAsync(dweight, 0, (size_t)N * wb, stream));
  }
  rows::GradArgs a = {};
  a.M = M;
  a.N = N;
  a.dy = dY;
  a.lddy = lddy;
  a.h = H;
  a.ldh = ldh;
  a.w = weight;
  a.rstd = rstd;
  a.dh = dX != nullptr ? dH : nullptr;
  a.lddh = lddh;
  a.dx = dX;
  a.lddx = lddx;
  const int vw = 16 / eb;
  const bool whole = rows::aligned(dY, lddy, eb, 16) && rows::aligned(H, ldh, eb, 16) &&
                     rows::aligned(a.dh, lddh, eb, 16) && rows::aligned(dX, lddx, eb, 16) &&
                     rows::aligned(weight, 0, wb, 16) && N % vw == 0;
  const bool shifted = rows::alike(H, ldh, dY, lddy, eb) && rows::alike(a.dh, lddh, dY, lddy, eb) &&
                       rows::alike(dX, lddx, dY, lddy, eb) && rows::shift(M, N, vw, wb, sms) &&
                       !rows::one_warp(N, vw, 65, 256);
  const rows::Access access = whole ? rows::kPieces : shifted ? rows::kShifted : rows::kSingle;
  const bool vec = access != rows::kSingle;
  const long long pieces = rows::pieces_of(access, N, vw);
  const int held = pieces > rows::held_of(vec ? vw : 1) * rows::kMaxThreads ? 0
                   : vec ? (pieces <= 32 ? 1 : (pieces <= 512 ? 2 : 4)) : 8;
  const int threads = held == 1   ? rows::small_lanes(pieces)
                      : held == 2 ? rows::threads_of(pieces, 2, false)
                                  : rows::threads_of(pieces, rows::held_of(vec ? vw : 1), M < 2 * sms);
  int blocks = 0;
  if (held == 1) {
    blocks = rows::small_blocks(M, threads, sms);
  } else if (held != 0) {
    blocks = rows::spaced(access, M, (long long)lddy * eb, rows::blocks_of(M, threads, sms, 512));
  } else {
    const int fill = sms * 8 / (int)((N + rows::kColumnThreads - 1ll) / rows::kColumnThreads) + 1;
    blocks = M < fill ? M : fill;
  }
  std::unique_lock<std::mutex> lock;
  float* partial = nullptr;
  if (dweight != nullptr) {
    if (cudaGetDevice(&dev) != cudaSuccess) return rows::done(cudaErrorInvalidDevice);
    lock = library_lock();   // to the last launch
    int* status = nullptr;
    st = library_workspace(dev, stream, (size_t)blocks * N, 0, &partial, &status, nullptr, nullptr,
                           nullptr);
    if (st != SGEMM_OK) return st;
  }
  using B = __nv_bfloat16;
  auto go = [&](auto e, auto w) {
    using E = decltype(e);
    using W = decltype(w);
    return rows::done(rows::backward<E, W>(a, static_cast<W*>(dweight), partial, blocks, sms, stream,
                                           threads, access, held));
  };
  if (type == SGEMM_TYPE_F32) return go(0.f, 0.f);
  if (type == SGEMM_TYPE_BF16) return weight_type == SGEMM_TYPE_F32 ? go(B{}, 0.f) : go(B{}, B{});
  return weight_type == SGEMM_TYPE_F32 ? go(__half{}, 0.f) : go(__half{}, __half{});
}
