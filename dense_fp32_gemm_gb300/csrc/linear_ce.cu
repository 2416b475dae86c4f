// linear_ce.cu -- sgemm_linear_ce and sgemm_linear_ce_grad: softmax cross
// entropy of the logits X W^T over a vocabulary, and its gradients, without
// keeping the logits.
//
// Mathematics, for token t with target word a and upstream gradient d:
//   z_v = x_t . w_v,  lse = log sum_v exp z_v,  loss = lse - z_a
//   g_v = (exp(z_v - lse) - [v == a]) d;   dX = G W,  dW = G^T X.
// The vocabulary is taken in pieces. 16-bit operands: the product's epilogue
// holds a token's logits in registers (ragged_kernel, kLse and kGrad), from
// which the loss takes the largest and the sum of exponentials of each tile,
// and the gradient pass, which forms the logits once more, writes a piece of G
// in the operands' type. FP32 operands: a piece of the logits is written in
// FP32, reduced or transformed in place by the kernels below.
//
// G in 16 bits: each of its values is off by at most 2^-8 (BF16) or 2^-11 of it, as
// the other operand of the two products is; in dX and dW these errors add up as
// random ones do. 300 tokens x 5000 words x 512: dX is off by 1.73e-3 (BF16) or 2.23e-4 of
// itself in the 2-norm, of which the rounding of dX alone makes 1.66e-3 and 2.07e-4. (In
// two parts of 16 bits G would leave that alone, for 4 T V H operations more.) So that small
// gradients keep their bits, rows are scaled by d / max|d|, times 2^14 in F16 (values
// up to 2^14; a probability of 10^-5 is a normal number), and the products by the
// inverse.
//
// Operations: 2 T V H forward; 6 T V H for the gradients, 2 of which form the
// logits again (in exchange a piece of G is all that is ever stored). Bound by the
// tensor cores under the power limit: 4096 tokens x 100003 words x 4096 BF16, loss
// and gradients in 8.5 to 8.7 ms, 1580 TFLOP/s of all 8 T V H (93 % of a library
// product's sustained 1706); 2048 x 65536 x 2048, the loss in 361 us, 1523. Small
// ones by latency: 65 x 1000 x 256 F16 in 32 us, six launches of 3 to 7 us. FP32 by
// the conversions of its products (1000 x 8191 x 777 in 355 us, 317 in products).
#include <cuda_runtime.h>
#include <algorithm>
#include <cmath>
#include <mutex>

#include "../../include/sgemm_gb300.h"
#include "elements.cuh"
#include "ragged_launch.cuh"

#define SGEMM_API extern "C" __attribute__((visibility("default")))

namespace sgemm_gb300 {
namespace loss {
namespace {

using ragged::Operand;
using ragged::Params;

// A piece of the vocabulary: as many words as keep what is stored of it (G, or
// FP32 logits) within this, at least kLeastWords. Each piece costs some 10 us of
// launches and ragged last waves, and dX's sums a way through memory; 4096 tokens
// have 65536 words a piece. (With 1 GB 100003 words in one piece 8.34 ms instead of
// 8.41, with 256 MB 8.72, with 128 MB 9.18.)
constexpr size_t kPieceBytes = 512u << 20;
constexpr int kLeastWords = 2048;
// Statistics of a piece (16 bits): 8 bytes for each token and half tile.
constexpr size_t kStatsBytes = 256u << 20;

// Values of h per tensor-core accumulation (which truncates) of the logits that the
// loss, a 32-bit result, is made of: off by 2.7e-7 of itself at 2048 values, 1024
// at a time 5.6e-7, 256 at a time 1.3e-7 (2048 x 65536 x 2048 361, 348 and 412 us). Those
// of G, which is rounded to 16 bits, take what 16-bit results take.
constexpr int kLossChunk = 512;

constexpr float kLeast = -3.402823466e38f;
constexpr uint32_t kAll = 0xffffffffu;

// (most, sum) of two disjoint sets of logits.
__device__ __forceinline__ float2 merge(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  return make_float2(m, a.y * expf(a.x - m) + b.y * expf(b.x - m));
}

// The parts of a piece and what the pieces before gave, token by token: 32
// tokens a block, kGroups threads a token.
constexpr int kGroups = 32;
struct Join {
  int T, V, parts;
  const float2* stats;        // [part][token]
  float2* state;              // [token]: of the pieces so far
  int first, last;
  const long long* target;
  long long ignore;
  const float* at_target;
  float *loss, *lse;
};
__global__ void __launch_bounds__(32 * kGroups) join_kernel(const Join a) {
  __shared__ float2 part[kGroups][32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
  for (long long t0 = blockIdx.x * 32ll; t0 < a.T; t0 += gridDim.x * 32ll) {
    const long long t = t0 + lane;
    float2 s = make_float2(kLeast, 0.f);
    if (t < a.T) {
      // (most first, then the sums: one exponential a part, loads that do not wait)
      float most = kLeast;
#pragma unroll 8
      for (int p = group; p < a.parts; p += kGroups)
        most = fmaxf(most, __ldg(&a.stats[(long long)p * a.T + t].x));
      float sum = 0.f;
#pragma unroll 8
      for (int p = group; p < a.parts; p += kGroups) {
        const float2 v = __ldg(&a.stats[(long long)p * a.T + t]);
        sum += v.y * expf(v.x - most);
      }
      s = make_float2(most, sum);
    }
    part[group][lane] = s;
    __syncthreads();
    if (group == 0 && t < a.T) {
      for (int g = 1; g < kGroups; ++g) s = merge(s, part[g][lane]);
      if (!a.first) s = merge(a.state[t], s);
      if (!a.last) {
        a.state[t] = s;
      } else {
        const float lse = s.x + logf(s.y);
        const long long word = a.target[t];
        if (a.lse != nullptr) a.lse[t] = lse;
        // a word that is none has no loss: NaN says so
        a.loss[t] = word == a.ignore ? 0.f
                    : word < 0 || word >= a.V ? __uint_as_float(0x7fc00000u)
                                              : lse - a.at_target[t];
      }
    }
    __syncthreads();
  }
}

// Factors of the tokens' gradients: d / c * unit, c the largest |d| among the
// numbers (an infinity leaves the other rows their range; 1 where there is none
// above 0, and in FP32), and c / unit, the factor of the products. 0 for a token
// that is not counted, NaN for one whose target is no word. One block.
constexpr int kScaleThreads = 1024;
__global__ void __launch_bounds__(kScaleThreads)
    scale_kernel(int T, int V, const long long* target, long long ignore, const float* d,
                 int scaled, float unit, float* row_scale, float* alpha) {
  __shared__ float part[kScaleThreads / 32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  float most = 0.f;
  for (long long t = threadIdx.x; t < T; t += kScaleThreads)
    if (target[t] != ignore && fabsf(d[t]) <= -kLeast) most = fmaxf(most, fabsf(d[t]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(kAll, most, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = most;
  __syncthreads();
  most = 0.f;
  for (int i = 0; i < kScaleThreads / 32; ++i) most = fmaxf(most, part[i]);
  const float c = scaled && most > 0.f ? most : 1.f;
  for (long long t = threadIdx.x; t < T; t += kScaleThreads) {
    const long long word = target[t];
    row_scale[t] = word == ignore              ? 0.f
                   : word < 0 || word >= V ? __uint_as_float(0x7fc00000u)
                                           : d[t] / c * unit;
  }
  if (threadIdx.x == 0) *alpha = c / unit;
}

// FP32: statistics of a piece of logits, a row per block.
constexpr int kRowThreads = 256;
__global__ void __launch_bounds__(kRowThreads)
    stats_kernel(int T, int n, const float* z, long long ldz, const long long* target, int col0,
                 float2* stats, float* at_target) {
  __shared__ float2 part[kRowThreads / 32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  for (long long t = blockIdx.x; t < T; t += gridDim.x) {
    const float* row = z + t * ldz;
    float2 s = make_float2(kLeast, 0.f);
    for (int c0 = threadIdx.x; c0 < n; c0 += 8 * kRowThreads) {
      float v[8], m = s.x;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = c0 + i * kRowThreads < n ? __ldcg(row + c0 + i * kRowThreads) : -INFINITY;
        m = fmaxf(m, v[i]);
      }
      float sum = s.y * expf(s.x - m);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += expf(v[i] - m);
      s = make_float2(m, sum);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      s = merge(s, make_float2(__shfl_xor_sync(kAll, s.x, o), __shfl_xor_sync(kAll, s.y, o)));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
      for (int w = 1; w < kRowThreads / 32; ++w) s = merge(s, part[w]);
      stats[t] = s;
      const long long rel = target[t] - col0;
      if (rel >= 0 && rel < n) at_target[t] = row[rel];
    }
    __syncthreads();
  }
}

// FP32: a piece of logits into G, in place. Rows start on 16 bytes; what is
// between a row's end and the next multiple of 4 is not used.
constexpr int kAhead = 2;                  // pieces of 16 bytes a thread
__global__ void __launch_bounds__(kRowThreads)
    gradient_kernel(int T, int n, float* z, long long ldz, const long long* target, int col0,
                    const float* lse, const float* row_scale) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  constexpr int kBlock = 4 * kAhead * kRowThreads;
  const long long blocks = (n + (long long)kBlock - 1) / kBlock;   // of a row
  for (long long b = blockIdx.x; b < blocks * T; b += gridDim.x) {
    const long long t = b / blocks;
    const long long c0 = (b - t * blocks) * kBlock + threadIdx.x * 4;
    float* row = z + t * ldz;
    float4 v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (c0 + i * (4 * kRowThreads) < n)
        v[i] = __ldcg(reinterpret_cast<const float4*>(row + c0 + i * (4 * kRowThreads)));
    const float l = lse[t], s = row_scale[t];
    const long long a = target[t] - col0;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const long long c = c0 + i * (4 * kRowThreads);
      if (c >= n) break;
      float g[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = expf(g[j] - l);
        g[j] = s == 0.f ? 0.f : (c + j == a ? e - 1.f : e) * s;
      }
      *reinterpret_cast<float4*>(row + c) = make_float4(g[0], g[1], g[2], g[3]);
    }
  }
}

// Rows of FP32 sums to the gradient's type.
template <typename E>
__global__ void __launch_bounds__(kRowThreads)
    round_kernel(int T, int H, const float* sums, E* out, long long ldo) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const long long blocks = (H + 4ll * kRowThreads - 1) / (4 * kRowThreads);
  for (long long b = blockIdx.x; b < blocks * T; b += gridDim.x) {
    const long long t = b / blocks;
    const long long c0 = (b - t * blocks) * (4 * kRowThreads) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long c = c0 + i * kRowThreads;
      if (c < H) out[t * ldo + c] = rows::from_f32<E>(__ldcg(sums + t * H + c));
    }
  }
}

template <typename... A>
cudaError_t start(void (*kernel)(A...), long long blocks, int threads, cudaStream_t stream,
                  std::common_type_t<A>... args) {
  cudaLaunchConfig_t lc = {};
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
int done(cudaError_t e) {
  if (e == cudaSuccess) return SGEMM_OK;
  cudaGetLastError();
  return SGEMM_ERR_LAUNCH;
}
long long at_most(long long a, long long b) { return a < b ? a : b; }
size_t padded(size_t bytes) { return (bytes + 255) / 256 * 256; }

// What both calls are given (checked), and the products they are made of.
struct Problem {
  int type, T, V, H;
  const void *X, *W;
  int ldx, ldw;
  const long long* target;
  long long ignore;

  int elem() const { return type == SGEMM_TYPE_F32 ? 4 : 2; }
  bool f32() const { return type == SGEMM_TYPE_F32; }
  Operand x() const { return Operand{X, elem(), T, H, ldx, 0, 1}; }
  Operand words(int v0, int n) const {
    return Operand{static_cast<const char*>(W) + (size_t)v0 * ldw * elem(), elem(), n, H, ldw, 0, 1};
  }
  // words of a piece: equal pieces of whole tiles
  int piece(size_t bytes_per_word, size_t most) const {
    if (V == 0) return 1;
    size_t n = bytes_per_word == 0 ? (size_t)V : most / bytes_per_word;
    if (n < (size_t)kLeastWords) n = kLeastWords;
    if (n >= (size_t)V) return V;
    const long long pieces = (V + (long long)n - 1) / (long long)n;
    return (int)at_most(V, ((V + pieces - 1) / pieces + 255) / 256 * 256);
  }
  // Tiles of P that are taken side by side: P's rows of them stay in L2 while the
  // other operand, which may be larger, is read once. (`bytes`: of 256 rows.) With
  // the words' tiles fastest W was read for each 256 tokens: 2048 tokens x 65536
  // words x 2048 BF16, loss 417 us, so 349 (both in sums of 1024).
  static int block(size_t bytes) { return std::max(1, (int)((32u << 20) / (bytes + 1))); }
  // Few tokens: words on the lanes, so that W streams through full tiles (10
  // tokens x 8344 words x 2912 F16: the loss in 16 us, with tokens on the lanes 37).
  bool few() const { return !f32() && T <= 64; }
  int lse_source() const { return few() ? ragged::kLseFew : ragged::kLse; }
  int grad_source() const { return few() ? ragged::kGradFew : ragged::kGrad; }
  // statistics of n words at most, and by the form that was chosen
  int most_parts(int n) const { return std::max(4 * ragged::cdiv(n, 128), 2 * ragged::cdiv(n, 64)); }
  int parts(int n, const ragged::Plan& plan) const {
    return few() ? 4 * ragged::cdiv(n, 128) : 2 * ragged::cdiv(n, plan.form->form.bq);
  }
  // logits of n words: 16 bits, reduced or transformed in the epilogue ...
  Params per_token(int n, int v0, int chunk) const {
    Params p = {};
    p.E = 1;
    p.T = few() ? T : n;
    p.P = few() ? n : T;
    p.K = H;
    p.bf16 = type == SGEMM_TYPE_BF16;
    p.alpha = 1.f;
    p.chunk = chunk;
    p.target = target;
    p.col0 = v0;
    if (!few()) p.p_block = block(512ull * H);
    return p;
  }
  // ... FP32, written as they are
  Params plain(int n, float* z, long long ldz) const {
    Params p = {};
    p.E = 1;
    p.T = T;
    p.P = n;
    p.K = H;
    p.out = z;
    p.ldo = ldz;
    p.out_type = SGEMM_TYPE_F32;
    p.alpha = 1.f;
    p.chunk = ragged::accumulation_chunk(ragged::kF32, SGEMM_TYPE_F32);
    return p;
  }
};

// Bytes of the workspace, handed out one after another.
struct Carve {
  size_t used = 0;
  size_t take(size_t bytes) {
    const size_t at = used;
    used += padded(bytes);
    return at;
  }
};

int check(int type, int T, int V, int H, const void* X, int ldx, const void* W, int ldw,
          const long long* target) {
  if (type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16 && type != SGEMM_TYPE_F16)
    return SGEMM_ERR_INVALID_VALUE;
  if (T < 0 || V < 0 || H < 0) return SGEMM_ERR_INVALID_DIM;
  const int least = H > 1 ? H : 1;
  if (ldx < least || ldw < least) return SGEMM_ERR_INVALID_LD;
  if (T > 0 && target == nullptr) return SGEMM_ERR_NULL_PTR;
  if (T > 0 && V > 0 && H > 0 && (X == nullptr || W == nullptr)) return SGEMM_ERR_NULL_PTR;
  const uintptr_t mask = type == SGEMM_TYPE_F32 ? 3u : 1u;
  if (((reinterpret_cast<uintptr_t>(X) | reinterpret_cast<uintptr_t>(W)) & mask) ||
      (reinterpret_cast<uintptr_t>(target) & 7u))
    return SGEMM_ERR_MISALIGNED;
  return SGEMM_OK;
}
bool odd(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

int forward(const Problem& q, float* loss, float* lse, cudaStream_t stream) {
  const int T = q.T, V = q.V;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return done(cudaErrorInvalidDevice);
  int st = library_device_sms(dev, &sms);
  if (st != SGEMM_OK) return st;
  // statistics of a piece: one part for a piece of FP32 logits, else two for
  // each tile of at least 64 words
  const int n = q.f32() ? q.piece((size_t)T * 4, kPieceBytes) : q.piece((size_t)T / 4 + 1, kStatsBytes);
  const int most_parts = q.f32() ? 1 : q.most_parts(n);
  const long long ldz = (n + 3) / 4 * 4;
  Carve ws;
  const size_t at_state = ws.take((size_t)T * 8), at_z = ws.take((size_t)T * 4);
  const size_t at_stats = ws.take((size_t)T * 8 * most_parts);
  const size_t at_logits = ws.take(q.f32() ? (size_t)T * ldz * 4 : 0);

  // (the first piece is the largest; the others run by its plan)
  ragged::Plan first = {};
  const Operand x = q.x();
  const int n0 = n < V ? n : V;
  if (V > 0) {
    const Operand w = q.words(0, n0);
    st = q.f32()   ? ragged::plan(ragged::kF32, q.type, q.plain(n0, nullptr, ldz), w, x, &first)
         : q.few() ? ragged::plan(q.lse_source(), q.type, q.per_token(n0, 0, kLossChunk), w, x, &first)
                   : ragged::plan(q.lse_source(), q.type, q.per_token(n0, 0, kLossChunk), x, w, &first);
    if (st != SGEMM_OK) return st;
  }
  float* base = nullptr;
  int* status = nullptr;
  uint32_t* counters = nullptr;
  const std::unique_lock<std::mutex> lock = library_lock();   // to the last launch
  st = library_workspace(dev, stream, (ws.used + (V > 0 ? first.bytes() : 0)) / 4,
                         V > 0 ? first.counters() : 1, &base, &status, nullptr, nullptr, &counters);
  if (st != SGEMM_OK) return st;
  char* at = reinterpret_cast<char*>(base);
  float2* stats = reinterpret_cast<float2*>(at + at_stats);
  float* at_target = reinterpret_cast<float*>(at + at_z);
  float* z = reinterpret_cast<float*>(at + at_logits);

  Join join = {};
  join.T = T;
  join.V = V;
  join.stats = stats;
  join.state = reinterpret_cast<float2*>(at + at_state);
  join.target = q.target;
  join.ignore = q.ignore;
  join.at_target = at_target;
  join.loss = loss;
  join.lse = lse;
  const long long join_blocks = at_most((T + 31ll) / 32, sms * 8ll);
  int v0 = 0;
  do {
    const int m = (int)at_most(n, V - v0);
    if (m > 0) {
      Params p = q.f32() ? q.plain(m, z, ldz) : q.per_token(m, v0, kLossChunk);
      p.status = status;
      p.counters = counters;
      p.stats = stats;
      p.at_target = at_target;
      const Operand w = q.words(v0, m);
      if (q.f32()) {
        st = ragged::launch(first, p, w, x, at + ws.used, stream, "linear_ce");
        if (st != SGEMM_OK) return st;
        st = done(start(stats_kernel, at_most(T, sms * 8ll), kRowThreads, stream, T, m,
                        static_cast<const float*>(z), ldz, q.target, v0, stats, at_target));
        join.parts = 1;
      } else {
        st = q.few() ? ragged::launch(first, p, w, x, at + ws.used, stream, "linear_ce")
                     : ragged::launch(first, p, x, w, at + ws.used, stream, "linear_ce");
        join.parts = q.parts(m, first);
      }
      if (st != SGEMM_OK) return st;
    }
    join.first = v0 == 0;
    v0 += m;
    join.last = v0 >= V;
    st = done(start(join_kernel, join_blocks, 32 * kGroups, stream, join));
    if (st != SGEMM_OK) return st;
  } while (v0 < V);
  return SGEMM_OK;
}

int backward(const Problem& q, const float* lse, const float* dloss, void* dX, int lddx, void* dW,
             int lddw, cudaStream_t stream) {
  const int T = q.T, V = q.V, H = q.H, elem = q.elem();
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return done(cudaErrorInvalidDevice);
  int st = library_device_sms(dev, &sms);
  if (st != SGEMM_OK) return st;
  const int n = q.piece((size_t)T * elem, kPieceBytes);
  const int n0 = n < V ? n : V;
  const bool sums = dX != nullptr && !q.f32() && n < V;   // dX is added up in FP32
  const int per16 = 16 / elem;
  const long long ldg = (n + per16 - 1) / per16 * per16;
  Carve ws;
  const size_t at_scale = ws.take((size_t)T * 4), at_alpha = ws.take(4);
  const size_t at_g = ws.take((size_t)T * ldg * elem);
  const size_t at_sums = ws.take(sums ? (size_t)T * H * 4 : 0);

  // X, and each piece of W, serve two products: where TMA cannot read them in
  // place they are copied once
  Operand x = q.x();
  Operand w0 = q.words(0, n0);
  const bool copy_x = !x.direct(), copy_w = !w0.direct();
  const size_t at_x = ws.take(copy_x ? x.packed_bytes(false) : 0);
  const size_t at_w = ws.take(copy_w ? w0.packed_bytes(false) : 0);

  const int src = q.f32() ? ragged::kF32 : ragged::kDense;
  auto copied = [&](Operand* a) {          // as pack_operands() will describe it
    a->ptr = reinterpret_cast<void*>(256);
    a->ld = a->packed_pitch(false) / a->elem;
  };
  if (copy_x) copied(&x);
  if (copy_w) copied(&w0);
  auto gradient = [&](int m, int v0, void* g) {
    Params p = q.f32() ? q.plain(m, static_cast<float*>(g), ldg) : q.per_token(m, v0, ragged::accumulation_chunk(ragged::k16, q.type));
    p.out = g;
    p.ldo = ldg;
    return p;
  };
  // dX = G W: W stored with the words, the contraction, as its rows
  auto input = [&](int m, int v0, float* acc) {
    Params p = {};
    p.E = 1;
    p.T = T;
    p.P = H;
    p.K = m;
    p.p_mn = 1;
    p.bf16 = q.type == SGEMM_TYPE_BF16;
    p.out = acc != nullptr ? acc : dX;
    p.ldo = acc != nullptr ? H : lddx;
    p.out_type = acc != nullptr ? SGEMM_TYPE_F32 : q.type;
    p.alpha = 1.f;
    p.beta = v0 > 0 ? 1.f : 0.f;
    // (sums over all words of a piece, through operands larger than L2: workers on
    // whole tiles read the same words at the same time, those on parts of tiles do
    // not. With two waves' tiles cut 6.3 GB came from DRAM instead of 3.0, and loss
    // and gradients of 4096 tokens x 100003 words x 4096 BF16 took 8.84 ms, not 8.41)
    p.cut_rest = 1;
    // (FP32 sums over pieces are rounded to 16 bits in the end, so their products are
    // accumulated as those of 16-bit results: off by 9e-7 of themselves, beside the
    // 2^-8 or 2^-11 of that rounding)
    p.chunk = ragged::accumulation_chunk(src, q.type);
    return p;
  };
  // dW = G^T X
  auto weight = [&](int m, int v0) {
    Params p = {};
    p.wgrad = 1;
    p.E = 1;
    p.T = T;
    p.P = H;
    p.Q = m;
    p.K = T;
    p.p_mn = p.q_mn = 1;
    p.bf16 = q.type == SGEMM_TYPE_BF16;
    p.p_block = Problem::block(256ull * elem * T);
    p.out = static_cast<char*>(dW) + (size_t)v0 * lddw * elem;
    p.ldo = lddw;
    p.out_type = q.type;
    p.alpha = 1.f;
    p.chunk = ragged::accumulation_chunk(src, q.type);
    return p;
  };
  auto g_of = [&](void* g, int m) { return Operand{g, elem, T, m, ldg, 0, 1}; };

  // (the first piece is the largest; the others run by its plans. Of where G will
  // lie only the alignment counts, which any multiple of 256 has)
  void* somewhere = reinterpret_cast<void*>(256);
  ragged::Plan plans[3] = {};
  size_t most = 0, most_counters = 1;
  for (int i = 0; V > 0 && i < 3; ++i) {
    if ((i == 1 && dX == nullptr) || (i == 2 && dW == nullptr)) continue;
    if (i == 0)
      st = q.f32()   ? ragged::plan(src, q.type, gradient(n0, 0, somewhere), w0, x, &plans[i])
           : q.few() ? ragged::plan(q.grad_source(), q.type, gradient(n0, 0, somewhere), w0, x, &plans[i])
                     : ragged::plan(q.grad_source(), q.type, gradient(n0, 0, somewhere), x, w0, &plans[i]);
    else if (i == 1)
      st = ragged::plan(src, q.type, input(n0, 0, nullptr), w0, g_of(somewhere, n0), &plans[i]);
    else
      st = ragged::plan(src, q.type, weight(n0, 0), x, g_of(somewhere, n0), &plans[i]);
    if (st != SGEMM_OK) return st;
    most = std::max(most, plans[i].bytes());
    most_counters = std::max(most_counters, plans[i].counters());
  }
  float* base = nullptr;
  int* status = nullptr;
  uint32_t* counters = nullptr;
  const std::unique_lock<std::mutex> lock = library_lock();   // to the last launch
  st = library_workspace(dev, stream, (ws.used + most) / 4, most_counters, &base, &status, nullptr,
                         nullptr, &counters);
  if (st != SGEMM_OK) return st;
  char* at = reinterpret_cast<char*>(base);
  float* row_scale = reinterpret_cast<float*>(at + at_scale);
  float* alpha = reinterpret_cast<float*>(at + at_alpha);
  void* g = at + at_g;
  float* acc = sums ? reinterpret_cast<float*>(at + at_sums) : nullptr;
  char* rest = at + ws.used;

  st = done(start(scale_kernel, 1, kScaleThreads, stream, T, V, q.target, q.ignore, dloss,
                  (int)!q.f32(), q.type == SGEMM_TYPE_F16 ? 16384.f : 1.f, row_scale, alpha));
  if (st != SGEMM_OK) return st;
  for (long long at_word = 0; at_word < V; at_word += n) {   // (steps past 2^31 at the end)
    const int v0 = (int)at_word, m = (int)at_most(n, V - at_word);
    auto with = [&](Params p) {
      p.status = status;
      p.counters = counters;
      return p;
    };
    Params p = with(gradient(m, v0, g));
    Operand w = q.words(v0, m);
    if (copy_w || (copy_x && v0 == 0)) {
      Operand first = q.x();
      const bool of_x = copy_x && v0 == 0;
      st = done(ragged::pack_operands(&first, of_x ? at + at_x : nullptr, &w,
                                      copy_w ? at + at_w : nullptr, false, sms, stream));
      if (st != SGEMM_OK) return st;
      if (of_x) x = first;
    }
    if (q.f32()) {
      st = ragged::launch(plans[0], p, w, x, rest, stream, "linear_ce_grad");
      if (st != SGEMM_OK) return st;
      const long long block = 4 * kAhead * kRowThreads, blocks = (m + block - 1) / block * T;
      st = done(start(gradient_kernel, at_most(blocks, sms * 8ll), kRowThreads, stream, T, m,
                      static_cast<float*>(g), ldg, q.target, v0, lse,
                      static_cast<const float*>(row_scale)));
    } else {
      p.lse = lse;
      p.row_scale = row_scale;
      st = q.few() ? ragged::launch(plans[0], p, w, x, rest, stream, "linear_ce_grad")
                   : ragged::launch(plans[0], p, x, w, rest, stream, "linear_ce_grad");
    }
    if (st != SGEMM_OK) return st;
    if (dX != nullptr) {
      p = with(input(m, v0, acc));
      p.alpha_dev = q.f32() ? nullptr : alpha;
      st = ragged::launch(plans[1], p, w, g_of(g, m), rest, stream, "linear_ce_dx");
      if (st != SGEMM_OK) return st;
    }
    if (dW != nullptr) {
      p = with(weight(m, v0));
      p.alpha_dev = q.f32() ? nullptr : alpha;
      st = ragged::launch(plans[2], p, x, g_of(g, m), rest, stream, "linear_ce_dw");
      if (st != SGEMM_OK) return st;
    }
  }
  if (sums) {
    const long long blocks = at_most((H + 4ll * kRowThreads - 1) / (4 * kRowThreads) * T, sms * 8ll);
    const float* s = acc;
    st = q.type == SGEMM_TYPE_BF16
             ? done(start(round_kernel<__nv_bfloat16>, blocks, kRowThreads, stream, T, H, s,
                          static_cast<__nv_bfloat16*>(dX), (long long)lddx))
             : done(start(round_kernel<__half>, blocks, kRowThreads, stream, T, H, s,
                          static_cast<__half*>(dX), (long long)lddx));
  }
  return st;
}

// Rows of zeros.
int clear(void* p, int rows, int cols, int ld, int elem, cudaStream_t stream) {
  if (p == nullptr || rows == 0 || cols == 0) return SGEMM_OK;
  return done(cudaMemset2DAsync(p, (size_t)ld * elem, 0, (size_t)cols * elem, rows, stream));
}

}  // namespace
}  // namespace loss
}  // namespace sgemm_gb300

using namespace sgemm_gb300;

SGEMM_API int sgemm_linear_ce(int type, int T, int V, int H, const void* X, int ldx, const void* W,
                              int ldw, const long long* target, long long ignore_index, float* loss,
                              float* lse, void* stream) {
  const int st = loss::check(type, T, V, H, X, ldx, W, ldw, target);
  if (st != SGEMM_OK) return st;
  if (T == 0) return SGEMM_OK;
  if (loss == nullptr) return SGEMM_ERR_NULL_PTR;
  if (loss::odd(loss, 4) || loss::odd(lse, 4)) return SGEMM_ERR_MISALIGNED;
  const loss::Problem q{type, T, V, H, X, W, ldx, ldw, target, ignore_index};
  return loss::forward(q, loss, lse, static_cast<cudaStream_t>(stream));
}

SGEMM_API int sgemm_linear_ce_grad(int type, int T, int V, int H, const void* X, int ldx,
                                   const void* W, int ldw, const long long* target,
                                   long long ignore_index, const float* lse, const float* dloss,
                                   void* dX, int lddx, void* dW, int lddw, void* stream_) {
  const int st = loss::check(type, T, V, H, X, ldx, W, ldw, target);
  if (st != SGEMM_OK) return st;
  const int least = H > 1 ? H : 1;
  if ((dX != nullptr && lddx < least) || (dW != nullptr && lddw < least)) return SGEMM_ERR_INVALID_LD;
  const int elem = type == SGEMM_TYPE_F32 ? 4 : 2;
  if (loss::odd(dX, elem) || loss::odd(dW, elem) || loss::odd(lse, 4) || loss::odd(dloss, 4))
    return SGEMM_ERR_MISALIGNED;
  if (T > 0 && (lse == nullptr || dloss == nullptr)) return SGEMM_ERR_NULL_PTR;
  if (H == 0 || (dX == nullptr && dW == nullptr)) return SGEMM_OK;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (T == 0) return loss::clear(dW, V, H, lddw, elem, stream);
  if (V == 0) return loss::clear(dX, T, H, lddx, elem, stream);
  const loss::Problem q{type, T, V, H, X, W, ldx, ldw, target, ignore_index};
  return loss::backward(q, lse, dloss, dX, lddx, dW, lddw, stream);
}
