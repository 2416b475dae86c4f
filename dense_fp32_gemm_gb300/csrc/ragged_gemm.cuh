// ragged_gemm.cuh -- tensor-core products of ragged groups: one kernel behind
// sgemm_grouped, sgemm_grouped_wgrad and sgemm_i8.
//
// Mathematics. A group e owns the token rows [off_e, off_e + n_e). The kernel
// forms tiles of D[p, q] = sum_k P_e[p, k] Q_e[q, k], where p runs along the
// contiguous dimension of the output and q along its rows:
//   rows   p = output feature, q = token row, k = input feature:
//          out[off_e + q, p] = sum_k W_e[p, k] X[off_e + q, k];
//   wgrad  p = column and q = row of the weight gradient, k = token row:
//          out_e[q, p] = sum_k B[off_e + k, p] A[off_e + k, q].
// P is the 128-lane side of the tensor-core instruction (M = 128), Q its N
// side of BQ columns, so a group of few tokens costs a narrow tile and its
// weights still stream through full 128-row tiles.
//
// Sources (SRC) and how they become MMA operands:
//   k16   BF16 or F16 tiles, read by the MMAs as TMA wrote them;
//   kF32  FP32 tiles, cut by converter warps into three BF16 parts
//         x = h + m + l (8 significant bits each, rounded to nearest, so 24 in
//         all); per k-step the six products hh, hm, mh, mm, hl, lh are
//         accumulated, what is dropped is below 2^-24 |a b|;
//   kI8   8-bit integers, turned by converter warps into F16 (exact), since
//         sm_103a has no integer tensor instruction of this generation. A
//         product is at most 2^14, so the FP32 sums of 1024 products are
//         exact integers.
//
// Accumulation. The tensor core adds into FP32 with truncation, an error that
// grows with the number of instructions. For 32-bit results a tile's sum is
// therefore cut into chunks of `chunk` k-slices: each goes to one of two
// tensor-memory accumulators and is added in registers (round to nearest; for
// kI8 as 32-bit integers) while the other is filled.
//
// Roles: warp 0 issues the TMA loads, warp 1 the MMAs, warps 2-9 read the
// accumulators (two warps per lane quarter, each half of the columns) and
// write the output, warps 10-17 (kF32, kI8) convert. The work list is
// computed on the device from the offsets: every CTA scans them, then takes
// the units blockIdx.x, + gridDim.x, ... With fewer tiles than CTAs each
// tile's sum is cut into ranges along k; the CTA that arrives last adds the
// partial tiles in a fixed order (so results do not depend on the order of
// arrival) -- no CTA waits for another.
//
// Every wait is bounded; a CTA that gives up drains its copies and MMAs,
// frees its tensor memory and returns. Offsets are clamped to the row count,
// so no value in them reaches outside the matrices.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "ffma_sgemm.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace sgemm_gb300 {
namespace ragged {

enum Src : int { k16 = 0, kF32 = 1, kI8 = 2 };
enum OutType : int { kOutF32 = 0, kOutBf16 = 1, kOutF16 = 2 };

constexpr int BP = 128;            // tile height in p (MMA M)
constexpr int kMaxGroups = 1024;   // the scanned offsets live in shared memory
constexpr int kEpiWarp0 = 2, kEpiWarps = 8, kEpiThreads = kEpiWarps * 32;
constexpr int kConvWarp0 = kEpiWarp0 + kEpiWarps, kConvWarps = 8;

struct Params {
  int wgrad;              // 0: rows, 1: weight gradient
  int E, T;               // groups, token rows
  int P, Q;               // output columns; output rows per group (wgrad)
  int K;                  // contraction length (rows); 0 skips the products
  int p_mn, q_mn;         // operand stored with k as its slow dimension
  int bf16;               // k16: operand type (else F16)
  const int* offsets;     // E + 1 row bounds on the device; null: one group of T rows
  void* out;
  long long ldo, stride_o;  // row pitch; pitch between the groups' outputs (wgrad)
  int out_type;
  float alpha, beta;
  const float* scale_p;   // kI8: scales of p and q
  const float* scale_q;
  int chunk;              // k-slices per tensor-memory accumulation
  float* partials;        // gridDim.x tiles of BQ x 128 floats (when tiles are cut along k)
  uint32_t* counters;     // arrivals per cut tile, zero between launches
  int* status;
  long long timeout_ns;
};

// Stage geometry. Raw tiles as TMA writes them (kSlice elements of k), and
// the converted operand tiles (kF32, kI8).
template <int SRC, int BQ>
struct Geo {
  static constexpr int kSlice = SRC == kF32 ? 32 : 64;
  static constexpr int kElem = SRC == k16 ? 2 : (SRC == kF32 ? 4 : 1);
  static constexpr int kRawRow = kSlice * kElem;               // 128, 128, 64 bytes
  static constexpr int kRawP = BP * kRawRow, kRawQ = BQ * kRawRow;
  static constexpr int kRaw = kRawP + kRawQ;
  static constexpr int kParts = SRC == kF32 ? 3 : 1;
  static constexpr int kOpP = BP * kSlice * 2, kOpQ = BQ * kSlice * 2;  // one part
  static constexpr int kOp = SRC == k16 ? 0 : kParts * (kOpP + kOpQ);
  static constexpr bool kConv = SRC != k16;
  static constexpr int kRegion = 192 * 1024;
  // operand stages first (at most 4), then as many raw stages as fit
  static constexpr int kOpFit = kConv ? (kRegion - 2 * kRaw) / kOp : 0;
  static constexpr int kOpStages = kConv ? (kOpFit < 4 ? kOpFit : 4) : 0;
  static constexpr int kRawFit = (kRegion - kOpStages * kOp) / kRaw;
  static constexpr int kRawStages = kRawFit < 12 ? kRawFit : 12;
  static_assert(!kConv || kOpStages >= 2, "operand stages");
  static_assert(kRawStages >= 2, "raw stages");
  static constexpr int kThreads = (kConv ? kConvWarp0 + kConvWarps : kConvWarp0) * 32;
  static constexpr int kTmemCols = 2 * BQ;
  static_assert(kTmemCols >= 32 && kTmemCols <= 512, "tensor memory");
  // FP32 sums leave tensor memory at the latest after this many slices when
  // they have to be exact integers (kI8: 1024 products of at most 2^14)
  static constexpr int kExactChunk = 1024 / kSlice;
};

struct Shared {
  uint64_t raw_full[12], raw_empty[12];
  uint64_t op_full[4], op_empty[4];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain, epi_sync;
  uint32_t tmem;
  int abort;
  int last;                     // this CTA's unit is the last of its tile
  int tiles, splits;
  int row0[kMaxGroups], rows[kMaxGroups], first[kMaxGroups + 1];  // the scanned groups
};
constexpr int kSharedBytes = ((int)sizeof(Shared) + 15) / 16 * 16;
constexpr int kSmemBytes = 1024 + 192 * 1024 + kSharedBytes;
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");

__host__ __device__ constexpr int cdiv(int a, int b) { return a / b + (a % b != 0); }

struct Unit {
  int e, p0, q0;       // group, first p, first q within the group
  int row0, nq;        // first token row of the group; valid q in the tile
  int kb, ke, klen;    // slices of this unit, contraction length
  int tile, part;      // tile number, which k-range
};

// Unit u of the work list (see Shared::first): tiles of a group are
// consecutive, q fastest, so that CTAs running together share weight tiles.
template <int SLICE, int BQ>
__device__ __forceinline__ Unit get_unit(const Params& p, const Shared* sh, int u) {
  Unit w;
  const int S = sh->splits;
  w.tile = u / S;
  w.part = u - w.tile * S;
  int lo = 0, hi = p.E - 1;     // last group with first <= tile
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sh->first[mid] <= w.tile) lo = mid; else hi = mid - 1;
  }
  w.e = lo;
  const int j = w.tile - sh->first[lo];
  w.row0 = sh->row0[lo];
  const int n = sh->rows[lo];
  const int qdim = p.wgrad ? p.Q : n;
  const int qt = cdiv(qdim, BQ);
  const int tp = j / qt, tq = j - tp * qt;
  w.p0 = tp * BP;
  w.q0 = tq * BQ;
  w.nq = min(BQ, qdim - w.q0);
  w.klen = p.K == 0 ? 0 : (p.wgrad ? n : p.K);
  const int ks = cdiv(w.klen, SLICE);
  w.kb = (int)((long long)ks * w.part / S);
  w.ke = (int)((long long)ks * (w.part + 1) / S);
  return w;
}

// ---- conversions --------------------------------------------------------------
// Two FP32 values into packed BF16 parts h, m, l (x = h + m + l up to 2^-24 |x|).
__device__ __forceinline__ void split2(float x, float y, uint32_t& h, uint32_t& m, uint32_t& l) {
  auto pack = [](float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  };
  h = pack(x, y);
  const float rx = x - __uint_as_float(h << 16), ry = y - __uint_as_float(h & 0xFFFF0000u);
  m = pack(rx, ry);
  l = pack(rx - __uint_as_float(m << 16), ry - __uint_as_float(m & 0xFFFF0000u));
}

// Four 8-bit integers into four F16 values: with the sign bit flipped a byte
// is v + 128; as the low byte of 0x6400 it reads 1024 + v + 128 in F16.
__device__ __forceinline__ uint2 i8_to_f16(uint32_t v) {
  const uint32_t u = v ^ 0x80808080u;
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
  uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), bias);
  const __half2 y = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

// One operand side of a stage, kF32: raw rows of 128 bytes (128-byte swizzle).
// K-major: row r = element r of the side, its 32 values of k -> parts with
// rows of 64 bytes (64-byte swizzle). MN-major: boxes of 32 elements x 32 rows
// of k -> chunks of 64 elements x 32 rows (128-byte swizzle). Rows of k at or
// past `klim` are written as zeros.
template <int ROWS>
__device__ __forceinline__ void convert_f32(const unsigned char* raw, unsigned char* op, bool mn,
                                            int klim, int t, int nt) {
  constexpr int PART = ROWS * 64;
  for (int i = t; i < ROWS * 4; i += nt) {
    const int r = i >> 2, c = i & 3;   // MN-major: r = box * 32 + k
    float4 a = *reinterpret_cast<const float4*>(raw + r * 128 + (((2 * c) ^ (r & 7)) << 4));
    float4 b = *reinterpret_cast<const float4*>(raw + r * 128 + (((2 * c + 1) ^ (r & 7)) << 4));
    int at;
    if (mn) {
      const int k = r & 31, box = r >> 5;
      if (k >= klim) a = b = make_float4(0.f, 0.f, 0.f, 0.f);
      at = (box >> 1) * 4096 + k * 128 + ((((box & 1) * 4 + c) ^ (k & 7)) << 4);
    } else {
      at = r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    }
    uint4 h, m, l;
    split2(a.x, a.y, h.x, m.x, l.x);
    split2(a.z, a.w, h.y, m.y, l.y);
    split2(b.x, b.y, h.z, m.z, l.z);
    split2(b.z, b.w, h.w, m.w, l.w);
    *reinterpret_cast<uint4*>(op + at) = h;
    *reinterpret_cast<uint4*>(op + PART + at) = m;
    *reinterpret_cast<uint4*>(op + 2 * PART + at) = l;
  }
}

// kI8: raw rows of 64 bytes (64-byte swizzle) -> rows of 64 F16 values
// (128-byte swizzle).
template <int ROWS>
__device__ __forceinline__ void convert_i8(const unsigned char* raw, unsigned char* op, int t,
                                           int nt) {
  for (int i = t; i < ROWS * 4; i += nt) {
    const int r = i >> 2, c = i & 3;
    const uint4 v = *reinterpret_cast<const uint4*>(raw + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
    const uint2 a = i8_to_f16(v.x), b = i8_to_f16(v.y), d = i8_to_f16(v.z), e = i8_to_f16(v.w);
    unsigned char* row = op + r * 128;
    *reinterpret_cast<uint4*>(row + (((2 * c) ^ (r & 7)) << 4)) = make_uint4(a.x, a.y, b.x, b.y);
    *reinterpret_cast<uint4*>(row + (((2 * c + 1) ^ (r & 7)) << 4)) = make_uint4(d.x, d.y, e.x, e.y);
  }
}

__device__ __forceinline__ float load_out(const void* base, long long at, int type) {
  if (type == kOutF32) return static_cast<const float*>(base)[at];
  if (type == kOutBf16) return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at]);
  return __half2float(static_cast<const __half*>(base)[at]);
}
__device__ __forceinline__ void store_out(void* base, long long at, int type, float v) {
  if (type == kOutF32)
    static_cast<float*>(base)[at] = v;
  else if (type == kOutBf16)
    static_cast<__nv_bfloat16*>(base)[at] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(base)[at] = __float2half_rn(v);
}

template <int SRC, int BQ>
__global__ void __launch_bounds__(Geo<SRC, BQ>::kThreads, 1)
    ragged_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap mapP,
                  const __grid_constant__ CUtensorMap mapQ) {
  using G = Geo<SRC, BQ>;
  constexpr int SL = G::kSlice;
  constexpr int RS = G::kRawStages, OS = G::kOpStages;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw_addr = ptx::smem_addr(smem_raw);
  unsigned char* base = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const uint32_t base_addr = ptx::smem_addr(base);
  // operand stages (kConv) start on 1024-byte boundaries, then the raw ones
  unsigned char* raw_base = base + OS * G::kOp;
  const uint32_t raw_base_addr = base_addr + OS * G::kOp;
  Shared* sh = reinterpret_cast<Shared*>(base + G::kRegion);
  volatile int* abort_w = &sh->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr uint32_t kAll = 0xffffffffu;

  if (tid == 0) {
    for (int s = 0; s < RS; ++s) {
      ptx::mbar_init(ptx::smem_addr(&sh->raw_full[s]), 1);
      ptx::mbar_init(ptx::smem_addr(&sh->raw_empty[s]), G::kConv ? kConvWarps : 1);
    }
    for (int s = 0; s < OS; ++s) {
      ptx::mbar_init(ptx::smem_addr(&sh->op_full[s]), kConvWarps);
      ptx::mbar_init(ptx::smem_addr(&sh->op_empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(ptx::smem_addr(&sh->acc_full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&sh->acc_empty[i]), kEpiWarps);
    }
    ptx::mbar_init(ptx::smem_addr(&sh->drain), 1);
    ptx::mbar_init(ptx::smem_addr(&sh->epi_sync), kEpiThreads);
    sh->abort = 0;
    ptx::mbar_fence_init();
    ptx::tma_prefetch_desc(&mapP);
    ptx::tma_prefetch_desc(&mapQ);
  }
  if (warp == 1) {
    tc::tmem_alloc(ptx::smem_addr(&sh->tmem), G::kTmemCols);
    tc::tmem_relinquish();
  }
  // launched with programmatic stream serialization: the set-up above overlaps
  // the end of the kernel ahead; nothing below touches global memory before it
  // has completed
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  if (warp == 0) {
    // scan of the groups: rows, and the number of the first tile of each
    const int ptiles = cdiv(p.P, BP);
    int carry = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int lo = 0, n = 0, tiles = 0;
      if (e < p.E) {
        lo = p.offsets == nullptr ? 0 : min(max(p.offsets[e], 0), p.T);
        const int hi = p.offsets == nullptr ? p.T : min(max(p.offsets[e + 1], 0), p.T);
        n = max(hi - lo, 0);
        tiles = ptiles * cdiv(p.wgrad ? p.Q : n, BQ);
      }
      int incl = tiles;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kAll, incl, d);
        if (lane >= d) incl += o;
      }
      if (e < p.E) {
        sh->row0[e] = lo;
        sh->rows[e] = n;
        sh->first[e] = carry + incl - tiles;
      }
      carry += __shfl_sync(kAll, incl, 31);
    }
    if (lane == 0) {
      sh->first[p.E] = carry;
      sh->tiles = carry;
      // fewer tiles than CTAs: cut each along k, at least four slices a range
      const int mean = p.wgrad ? p.T / p.E : p.K;
      const int most = cdiv(mean, SL) / 4;
      int S = carry > 0 ? (int)gridDim.x / carry : 1;
      S = min(S, most);
      sh->splits = S > 1 && p.partials != nullptr ? S : 1;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh->tmem;
  const int units = sh->tiles * sh->splits;

  if (warp == 0) {
    // ---- TMA producer ---------------------------------------------------------
    if (lane == 0) {
      int it = 0;
      for (int u = blockIdx.x; u < units && !*abort_w; u += gridDim.x) {
        const Unit w = get_unit<SL, BQ>(p, sh, u);
        const int qrow = p.wgrad ? 0 : w.row0;
        bool ok = true;
        for (int ks = w.kb; ks < w.ke; ++ks, ++it) {
          const int s = it % RS;
          if (!bounded_wait(ptx::smem_addr(&sh->raw_empty[s]), (uint32_t)((it / RS) & 1) ^ 1u,
                            abort_w, p.status, kDevTimeoutEmpty, p.timeout_ns)) {
            ok = false;
            break;
          }
          const uint32_t fb = ptx::smem_addr(&sh->raw_full[s]);
          const uint32_t st = raw_base_addr + (uint32_t)(s * G::kRaw);
          ptx::mbar_arrive_expect_tx(fb, (uint32_t)G::kRaw);
          const int k = ks * SL + (p.wgrad ? w.row0 : 0);
          const int pe = p.wgrad ? 0 : w.e;
          constexpr int BOX = G::kRawRow / G::kElem;  // elements along the fast dimension of a box
          if (p.p_mn) {
            for (int i = 0; i < BP / BOX; ++i)
              ptx::tma_load_3d(st + (uint32_t)(i * SL * G::kRawRow), &mapP, w.p0 + i * BOX, k, pe, fb);
          } else {
            ptx::tma_load_3d(st, &mapP, k, w.p0, pe, fb);
          }
          if (p.q_mn) {
            for (int i = 0; i < BQ / BOX; ++i)
              ptx::tma_load_3d(st + (uint32_t)(G::kRawP + i * SL * G::kRawRow), &mapQ,
                               w.q0 + i * BOX, k, 0, fb);
          } else {
            ptx::tma_load_3d(st + G::kRawP, &mapQ, k, qrow + w.q0, 0, fb);
          }
        }
        if (!ok) break;
      }
      // nothing may land after the CTA is gone: wait (bounded) for the last
      // stages issued
      const uint64_t t0 = ptx::global_ns();
      for (int j = it - 1; j >= 0 && j >= it - RS; --j) {
        const uint32_t fb = ptx::smem_addr(&sh->raw_full[j % RS]);
        while (!ptx::mbar_try_wait(fb, (uint32_t)((j / RS) & 1)))
          if ((long long)(ptx::global_ns() - t0) > cleanup_bound_ns(p.timeout_ns)) break;
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer -------------------------------------------------------------
    // operand tiles: K-major rows of 128 bytes (64 for kF32) in 8-row groups;
    // MN-major chunks of 64 elements x SL rows of k, 128 bytes a row
    constexpr bool kNarrow = SRC == kF32;
    const bool a_mn = p.p_mn, b_mn = p.q_mn;
    const uint32_t idesc = tc::idesc_f16(BP, BQ, SRC == kF32 || (SRC == k16 && p.bf16), a_mn, b_mn);
    auto desc = [](uint32_t addr, bool mn) {
      return mn ? tc::smem_desc(addr, SL * 128, 1024, true)
                : tc::smem_desc(addr, 16, kNarrow ? 512 : 1024, !kNarrow);
    };
    const uint32_t a_step = a_mn ? 2048u : 32u, b_step = b_mn ? 2048u : 32u;
    int it = 0, acc = 0;
    bool issued_any = false, ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const Unit w = get_unit<SL, BQ>(p, sh, u);
      for (int k0 = w.kb; k0 < w.ke && ok; k0 += p.chunk, ++acc) {
        const int buf = acc & 1;
        const uint32_t d = tmem + (uint32_t)(buf * BQ);
        ok = bounded_wait(ptx::smem_addr(&sh->acc_empty[buf]), (uint32_t)((acc >> 1) & 1) ^ 1u,
                          abort_w, p.status, kDevTimeoutSync, p.timeout_ns);
        ok = __all_sync(kAll, ok);
        if (!ok) break;
        tc::fence_after_sync();
        const int k1 = min(w.ke, k0 + p.chunk);
        for (int ks = k0; ks < k1; ++ks, ++it) {
          const int s = G::kConv ? it % (OS > 0 ? OS : 1) : it % RS;
          const uint32_t par = (uint32_t)((G::kConv ? it / (OS > 0 ? OS : 1) : it / RS) & 1);
          ok = bounded_wait(ptx::smem_addr(G::kConv ? &sh->op_full[s] : &sh->raw_full[s]), par,
                            abort_w, p.status, kDevTimeoutFull, p.timeout_ns);
          ok = __all_sync(kAll, ok);
          if (!ok) break;
          const uint32_t st = base_addr + (uint32_t)(s * (G::kConv ? G::kOp : G::kRaw));
          const int rem = w.klen - ks * SL;   // > 0
          const int steps = min(SL / 16, cdiv(rem, 16));
          if (SRC == k16 && p.wgrad && (rem & 15) && rem < SL) {
            // rows of k past the group's end belong to the next group: clear
            // them in both operands up to the end of their 16-row step (the
            // steps beyond are not issued)
            unsigned char* stp = base + s * G::kRaw;
            const int z0 = rem, nz = steps * 16 - rem;
            constexpr int kBoxes = (BP + BQ) / 64;
            for (int i = lane; i < kBoxes * nz * 8; i += 32) {
              const int box = i / (nz * 8), r = i - box * nz * 8;
              *reinterpret_cast<uint4*>(stp + box * (SL * 128) + z0 * 128 + r * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
            }
            ptx::fence_proxy_async_shared();
            __syncwarp();
          }
          tc::fence_after_sync();
          if (lane == 0) {
            constexpr int OP_P = SRC == k16 ? G::kRawP : G::kOpP;   // one part
            constexpr int OP_Q = SRC == k16 ? G::kRawQ : G::kOpQ;
            const uint32_t pa = st, qa = st + (uint32_t)(G::kParts * OP_P);
            for (int kk = 0; kk < steps; ++kk) {
              const uint32_t first = (ks == k0 && kk == 0) ? 0u : 1u;
              const uint64_t a0 = desc(pa + kk * a_step, a_mn), b0 = desc(qa + kk * b_step, b_mn);
              if (SRC == kF32) {
                const uint64_t a1 = desc(pa + OP_P + kk * a_step, a_mn);
                const uint64_t a2 = desc(pa + 2 * OP_P + kk * a_step, a_mn);
                const uint64_t b1 = desc(qa + OP_Q + kk * b_step, b_mn);
                const uint64_t b2 = desc(qa + 2 * OP_Q + kk * b_step, b_mn);
                tc::mma_f16(d, a2, b0, idesc, first);
                tc::mma_f16(d, a0, b2, idesc, 1u);
                tc::mma_f16(d, a1, b1, idesc, 1u);
                tc::mma_f16(d, a1, b0, idesc, 1u);
                tc::mma_f16(d, a0, b1, idesc, 1u);
                tc::mma_f16(d, a0, b0, idesc, 1u);
              } else {
                tc::mma_f16(d, a0, b0, idesc, first);
              }
            }
            tc::commit(ptx::smem_addr(G::kConv ? &sh->op_empty[s] : &sh->raw_empty[s]));
          }
          issued_any = true;
        }
        if (!ok) break;
        if (lane == 0) tc::commit(ptx::smem_addr(&sh->acc_full[buf]));
      }
    }
    if (*abort_w && issued_any && lane == 0) {
      // wait (bounded) until every MMA issued has completed
      tc::commit(ptx::smem_addr(&sh->drain));
      const uint64_t t0 = ptx::global_ns();
      while (!ptx::mbar_try_wait(ptx::smem_addr(&sh->drain), 0u))
        if ((long long)(ptx::global_ns() - t0) > cleanup_bound_ns(p.timeout_ns)) break;
    }
    __syncwarp();
  } else if (G::kConv && warp >= kConvWarp0) {
    // ---- converters: raw tiles -> operand tiles ----------------------------------
    const int t = tid - kConvWarp0 * 32;
    constexpr int NT = kConvWarps * 32;
    int it = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const Unit w = get_unit<SL, BQ>(p, sh, u);
      for (int ks = w.kb; ks < w.ke; ++ks, ++it) {
        const int rs = it % RS, os = it % (OS > 0 ? OS : 1);
        ok = bounded_wait(ptx::smem_addr(&sh->raw_full[rs]), (uint32_t)((it / RS) & 1), abort_w,
                          p.status, kDevTimeoutFull, p.timeout_ns) &&
             bounded_wait(ptx::smem_addr(&sh->op_empty[os]),
                          (uint32_t)((it / (OS > 0 ? OS : 1)) & 1) ^ 1u, abort_w, p.status,
                          kDevTimeoutEmpty, p.timeout_ns);
        ok = __all_sync(kAll, ok);
        if (!ok) break;
        const unsigned char* raw = raw_base + rs * G::kRaw;
        unsigned char* op = base + os * G::kOp;
        if (SRC == kF32) {
          const int klim = p.wgrad ? w.klen - ks * SL : SL;
          convert_f32<BP>(raw, op, p.p_mn, klim, t, NT);
          convert_f32<BQ>(raw + G::kRawP, op + G::kParts * G::kOpP, p.q_mn, klim, t, NT);
        } else {
          convert_i8<BP>(raw, op, t, NT);
          convert_i8<BQ>(raw + G::kRawP, op + G::kOpP, t, NT);
        }
        // the MMAs read the operand tiles, and TMA refills the raw ones,
        // through the async proxy
        ptx::fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(ptx::smem_addr(&sh->op_full[os]));
          ptx::mbar_arrive(ptx::smem_addr(&sh->raw_empty[rs]));
        }
      }
    }
  } else if (warp >= kEpiWarp0 && warp < kConvWarp0) {
    // ---- epilogue: accumulators -> registers -> output or partial tile -------------
    constexpr int HC = BQ / 2;                         // columns of this warp
    constexpr int CH = HC < 32 ? HC : 32;              // columns per tensor-memory read
    const int quarter = warp & 3;                      // TMEM lanes 32*quarter ..
    const int half = (warp - kEpiWarp0) >> 2;
    const int pr = quarter * 32 + lane;                // this thread's p within the tile
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    uint32_t sync_phase = 0;
    auto epi_sync = [&]() -> bool {                    // bounded rendezvous of the epilogue
      ptx::mbar_arrive(ptx::smem_addr(&sh->epi_sync));
      const bool ok = bounded_wait(ptx::smem_addr(&sh->epi_sync), sync_phase, abort_w, p.status,
                                   kDevTimeoutSync, p.timeout_ns);
      sync_phase ^= 1u;
      return __all_sync(kAll, ok);
    };
    int acc = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const Unit w = get_unit<SL, BQ>(p, sh, u);
      // kI8: the sums as 32-bit integers, kept in the same registers
      float sum[HC];
#pragma unroll
      for (int c = 0; c < HC; ++c) sum[c] = 0.f;
      for (int k0 = w.kb; k0 < w.ke; k0 += p.chunk, ++acc) {
        const int buf = acc & 1;
        ok = bounded_wait(ptx::smem_addr(&sh->acc_full[buf]), (uint32_t)((acc >> 1) & 1), abort_w,
                          p.status, kDevTimeoutFull, p.timeout_ns);
        ok = __all_sync(kAll, ok);
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t src = tmem + lane_base + (uint32_t)(buf * BQ + half * HC);
#pragma unroll
        for (int c0 = 0; c0 < HC; c0 += CH) {
          uint32_t v[CH];
#pragma unroll
          for (int i = 0; i < CH; i += 16)
            tc::tmem_ld16(src + (uint32_t)(c0 + i), *reinterpret_cast<uint32_t(*)[16]>(&v[i]));
          tc::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            if (SRC == kI8)
              sum[c0 + i] = __int_as_float(__float_as_int(sum[c0 + i]) +
                                           __float2int_rn(__uint_as_float(v[i])));
            else
              sum[c0 + i] += __uint_as_float(v[i]);
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&sh->acc_empty[buf]));
      }
      if (!ok) break;
      const int nq = w.nq - half * HC;                 // valid columns of this warp (may be <= 0)
      if (sh->splits > 1) {
        // publish this range's partial tile; the last CTA to arrive adds all
        // of them in order
        const int S = sh->splits;
        float* part = p.partials + (long long)u * (BP * BQ) + half * HC * BP + pr;
#pragma unroll
        for (int c = 0; c < HC; ++c)
          if (c < nq) __stcg(part + c * BP, sum[c]);
        __threadfence();
        ok = epi_sync();
        if (!ok) break;
        if (warp == kEpiWarp0 && lane == 0) {
          const uint32_t before = atomicAdd(p.counters + w.tile, 1u);
          const int last = before == (uint32_t)(S - 1);
          if (last) p.counters[w.tile] = 0u;           // ready for the next launch
          __threadfence();
          sh->last = last;
        }
        ok = epi_sync();
        if (!ok) break;
        if (!*reinterpret_cast<volatile int*>(&sh->last)) continue;
        __threadfence();
        const float* all = p.partials + (long long)w.tile * S * (BP * BQ) + half * HC * BP + pr;
#pragma unroll
        for (int c = 0; c < HC; ++c) {
          if (c >= nq) continue;
          float v = 0.f;
          for (int s = 0; s < S; ++s) {
            const float x = __ldcg(all + (long long)s * (BP * BQ) + c * BP);
            if (SRC == kI8)
              v = __int_as_float(__float_as_int(v) + __float_as_int(x));
            else
              v += x;
          }
          sum[c] = v;
        }
      }
      const int pp = w.p0 + pr;
      if (pp < p.P && nq > 0) {
        const float sp = SRC == kI8 ? p.scale_p[pp] : 1.f;
        const long long row = (long long)(p.wgrad ? 0 : w.row0) + w.q0 + half * HC;
        const long long at0 = (p.wgrad ? (long long)w.e * p.stride_o : 0ll) + row * p.ldo + pp;
#pragma unroll
        for (int c = 0; c < HC; ++c) {
          if (c >= nq) continue;
          const long long at = at0 + c * p.ldo;
          float v;
          if (SRC == kI8)
            v = (float)__float_as_int(sum[c]) * p.scale_q[row + c] * sp;
          else
            v = p.alpha * sum[c];
          if (p.beta != 0.f) v = fmaf(p.beta, load_out(p.out, at, p.out_type), v);
          store_out(p.out, at, p.out_type, v);
        }
      }
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, G::kTmemCols);
  }
}

}  // namespace ragged
}  // namespace sgemm_gb300
