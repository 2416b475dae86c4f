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
//         x = h + m + l (8 significant bits each, 24 in all); per k-step the
//         six products hh, hm, mh, mm, hl, lh are accumulated, what is dropped
//         is below 2^-23 |a b|;
//   kI8   8-bit integers, turned by converter warps into F16 (exact), since
//         sm_103a has no integer tensor instruction of this generation. A
//         product is at most 2^14, so the FP32 sums of 1024 products are
//         exact integers;
//   kI8Wide  the same integers, already as F16 in the workspace.
//
// Accumulation. The tensor core adds into FP32 with truncation, an error that
// grows with the number of instructions. A tile's sum is therefore cut into
// chunks of `chunk` values of k: each goes to one of two tensor-memory
// accumulators and is added in registers (round to nearest; for kI8 as 32-bit
// integers) while the other is filled.
//
// Kernel forms (CL): single CTAs, or clusters of two on vertically adjacent
// tiles whose even CTA issues M = 256 MMAs over both (cta_group::2): each CTA
// holds its 128 rows of P and half of the Q tile in shared memory and its 128
// lanes of the accumulator in tensor memory, so a slice moves two thirds of
// the bytes per multiply-add of a single 128 x 256 tile. Each CTA loads only
// its own tiles.
//
// Schedule. The work list is computed on the device from the offsets: every
// CTA scans them. Whole tiles are dealt out in waves of one per worker (a CTA
// or a pair) while at least two waves are left; the k-slices of the tiles that
// remain are dealt out evenly, each worker a contiguous range, so that it ends
// with (or, with few tiles, is) part of a tile. The worker that arrives last
// at a cut tile adds the partial tiles in the order of k, so results do not
// depend on the order of arrival -- no CTA waits for another. (Dealing out all
// tiles by slices would balance sums of different lengths exactly, but
// spreads the workers over all groups at once: the weight gradient of 8 groups
// of 1024 x (4096 + 1024) took 996 us that way against 141 in waves, at the
// same step of the work, its tiles no longer shared in L2.)
//
// Roles: warp 0 issues the TMA loads (both CTAs of a pair signal the even
// one's barriers), warp 1 the MMAs (in a pair only the even CTA's), warp 2 clears
// rows that belong to the next group (weight gradients), warps 4-11 read the
// accumulators (two warps per lane quarter, each half of the columns) and
// write the output, warps 12-19 (kF32, kI8) convert.
//
// Measured on GB300 (graphs of calls, operands larger than L2 but where noted;
// peaks: copy 6.78 TB/s, library BF16 product 1945 TFLOP/s):
//   256 x 2, BF16, 8192 rows in 8 groups, 4096 x 4096: 198 us, 1390 TFLOP/s under
//     sustained power, 179 in bursts of 2 ms (tensor pipe 68 % of active cycles).
//     The rest: ragged edges, the first wave's fill, the parts of the last tiles,
//     the accumulators' reads (2 %). Half the loads from L2 would gain 1-2 %.
//     The weight gradient of 8 groups of 1024 x (4096 + 1024) in FP32: 80 us, the
//     reads of the accumulators every 256 rows beside the MMAs 12 of them.
//   16 x 1, BF16: weights of 335 MB stream at 6.0 TB/s. The weights that 16 rows
//     choose of 32 of 1024 x 2048 (38 MB) take 13.8 us, DRAM's share 5.6: launch,
//     scan and first loads are some 3 us, the exchange of the parts of cut
//     tiles 2.5 us.
//   kF32 128: 2048 rows in 8 groups, 1024 x 2048: 63 us, tensor pipe 48 %: bound by
//     the hand-offs between converters, tensor memory and MMAs, not by DRAM.
//   kI8 16: a slice of 64 in 270 ns, bound by the converters' chain; kI8Wide: as
//     k16, plus 19 us to widen 2 x 4096 x 4096.
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

enum Src : int { k16 = 0, kF32 = 1, kI8 = 2, kI8Wide = 3 };
enum OutType : int { kOutF32 = 0, kOutBf16 = 1, kOutF16 = 2 };

constexpr int BP = 128;            // tile height in p (MMA M)
constexpr int kMaxGroups = 1024;   // the scanned offsets live in shared memory
// Slices by which one that has to be cleared is loaded early. Between a pair's
// CTAs the clearing takes longer than the loads are ahead of the MMAs (8 groups of
// 1000 x (4096 + 1024): 57.1 us with 0, 53.4 with 2, 52.8 with 3); a single CTA, with fewer
// stages, loses more by the one that is held (256 columns: 55.5 and 58.6 us). All
// with accumulations of 512 rows; of 256, as they are, the first takes 73 us.
__host__ __device__ constexpr int early_slices(int cl) { return cl == 2 ? 3 : 0; }
constexpr int kEpiWarp0 = 4, kEpiWarps = 8, kEpiThreads = kEpiWarps * 32;
constexpr int kConvWarp0 = kEpiWarp0 + kEpiWarps, kConvWarps = 8;

struct Params {
  int wgrad;              // 0: rows, 1: weight gradient
  int E, T;               // groups, token rows
  int P, Q;               // output columns; output rows per group (wgrad)
  int K;                  // contraction length (rows); 0 skips the products
  int p_mn, q_mn;         // operand stored with k as its slow dimension
  int p_shared;           // rows: one P matrix for all groups
  int bf16;               // k16: operand type (else F16; kI8Wide is F16)
  const int* offsets;     // E + 1 row bounds on the device; null: one group of T rows
  void* out;
  long long ldo, stride_o;  // row pitch; pitch between the groups' outputs (wgrad)
  int out_type;
  float alpha, beta;
  const float* scale_p;   // kI8: scales of p and q
  const float* scale_q;
  int chunk;              // values of k per tensor-memory accumulation (a multiple of the slice)
  // when tiles are cut along k: the slices a part has at least, and what a cut
  // costs, in 1/16 slices: once, and for each part of the tile
  int cut_least, cut_once, cut_part;
  float* partials;        // two tiles of BQ x 128 floats per CTA
  uint32_t* counters;     // arrivals at a cut tile, one per CTA, zero unless status is set
  int* status;
  long long timeout_ns;
};

// Stage geometry. Raw tiles as TMA writes them (kSlice elements of k), and
// the converted operand tiles (kF32, kI8).
template <int SRC, int BQ, int CL>
struct Geo {
  static constexpr bool kConv = SRC == kF32 || SRC == kI8;
  static constexpr bool kInt = SRC == kI8 || SRC == kI8Wide;
  // A slice is kSub tiles of kSubK values of k, each [P | Q] in rows of kRawRow
  // bytes. Narrow tiles take two: four MMAs of 16 columns last 160 cycles, the
  // waits and hand-offs of a stage some 270 more, which would bound the bytes
  // they stream.
  static constexpr int kSubK = SRC == kF32 ? 32 : 64;
  static constexpr int kSub = BQ <= 32 ? 2 : 1;
  static constexpr int kSlice = kSub * kSubK;
  static constexpr int kElem = SRC == kF32 ? 4 : (SRC == kI8 ? 1 : 2);
  static constexpr int kRows = BQ / CL;                         // rows of Q in one CTA
  static constexpr int kRawRow = kSubK * kElem;                 // 128, 128, 64 bytes
  static constexpr int kRawP = BP * kRawRow, kRawQ = kRows * kRawRow;
  static constexpr int kRawSub = kRawP + kRawQ, kRaw = kSub * kRawSub;
  static constexpr int kParts = SRC == kF32 ? 3 : 1;
  static constexpr int kOpQ = kRows * kSubK * 2;                // one converted part of Q's tile
  static constexpr int kOpSub = kParts * kOpQ, kOp = kConv ? kSub * kOpSub : 0;
  static constexpr int kRegion = 192 * 1024;
  // Converted stages: Q's parts in shared memory, P's in tensor memory behind
  // the two accumulators (a part is kSubK / 2 columns). The MMAs then read
  // only Q from shared memory: with both operands there, the six products of a
  // 128 x 128 FP32 tile moved 208 KB of it per slice, 1660 cycles against 770
  // of the MMAs. Up to 8 stages, as long as three raw ones fit beside them.
  static constexpr int kSubCols = kParts * kSubK / 2, kSlotCols = kSub * kSubCols;
  static constexpr int kSlotFit = (512 - 2 * BQ) / kSlotCols;
  static constexpr int kOpFit = kConv ? (kRegion - 3 * kRaw) / (kOp > 0 ? kOp : 1) : 0;
  static constexpr int kOpMin = kSlotFit < kOpFit ? kSlotFit : kOpFit;
  static constexpr int kOpStages = kConv ? (kOpMin < 8 ? kOpMin : 8) : 0;
  static constexpr int kRawFit = (kRegion - kOpStages * kOp) / kRaw;
  static constexpr int kRawStages = kRawFit < 12 ? kRawFit : 12;
  static_assert(kRawStages >= 2 && (!kConv || kOpStages >= 2), "stages");
  // Converter warps work in two groups (of four: each covers the 128 lanes of
  // tensor memory) that take the slices in turn, so that their chains of
  // latencies (wait, load, store, fence) overlap. Every raw barrier belongs to
  // one group: one that waited on a barrier whose phase before is another
  // group's, not yet complete, would take the phase before that for its own. So
  // the barriers form a ring of an even number, whatever the stages do.
  static constexpr int kConvGroups = 2, kGroupWarps = 4;
  static constexpr int kRawBars = kConv && kRawStages % 2 ? 2 * kRawStages : kRawStages;
  static constexpr int kThreads = (kConv ? kConvWarp0 + kConvWarps : kConvWarp0) * 32;
  // A thread of the epilogue holds BQ / 2 sums. For the widest tiles of a kind
  // they need more registers than the launch gives every thread, so the other
  // warpgroups give some up (what is raised is what is lowered).
  static constexpr bool kMoveRegs = BQ == (kConv ? 128 : 256);
  static constexpr int kRegs = kConv ? 96 : 168;      // at launch: 640 or 384 threads
  static constexpr int kRegsFew = kConv ? 48 : 72, kRegsMany = kConv ? 144 : 216;
  static constexpr int kRegsConv = 72;
  static_assert((kThreads == 640 || !kConv) && (kThreads == 384 || kConv) &&
                    128 * kRegsFew + 256 * kRegsMany + (kConv ? 256 * kRegsConv : 0) <=
                        kThreads * kRegs &&
                    kThreads * kRegs <= 65536,
                "register shares");
  static constexpr int kTmemCols = kConv ? 512 : 2 * BQ;
  static_assert(kTmemCols >= 32 && kTmemCols <= 512 &&
                    (!kConv || 2 * BQ + kOpStages * kSlotCols <= 512),
                "tensor memory");
  // (a K-major tile of 8-row groups, an MN-major one of 64-wide chunks)
  static_assert(kRows % 8 == 0 && BQ % 16 == 0 && BQ <= 256, "tile width");
};
// FP32 sums of integers leave tensor memory at the latest after this many
// values of k (products of at most 2^14 each).
constexpr int kExactK = 1024;

struct Shared {
  uint64_t raw_full[24], raw_empty[24];
  uint64_t op_full[8], op_empty[8];
  uint64_t tail_full[12];       // stages that end past their group: loaded, not yet cleared
  uint64_t peer_full[12];       // even CTA of a pair: the odd CTA's stage has been cleared
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain, epi_sync;
  uint32_t tmem;
  int abort;
  int last;                     // this CTA arrived last at its cut tile
  int dp;                       // tiles that are dealt out whole
  int base, len, cutters;       // slices dealt out: first position, number, workers
  // the scanned groups: first row, rows, number and slice position of the first tile
  int row0[kMaxGroups], rows[kMaxGroups], first[kMaxGroups], pos[kMaxGroups];
};
constexpr int kSharedBytes = ((int)sizeof(Shared) + 15) / 16 * 16;
constexpr int kSmemBytes = 1024 + 192 * 1024 + kSharedBytes;
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");

__host__ __device__ constexpr int cdiv(int a, int b) { return a / b + (a % b != 0); }

// Slices that a tile of a group counts for (one without a sum counts one, so
// that it has a place in the list).
template <int SLICE>
__device__ __forceinline__ int tile_slices(const Params& p, int rows) {
  return max(1, cdiv(p.K == 0 ? 0 : (p.wgrad ? rows : p.K), SLICE));
}

// Part of a worker's list: tile (p0, q0) of group e, its k-slices kb .. ke.
struct Unit {
  int e, p0, q0;       // group, first p, first q within the group
  int row0, nq;        // first token row of the group; valid q in the tile
  int nn;              // columns the MMAs compute: nq rounded up
  int kb, ke, klen;    // slices of this unit, contraction length
  // wgrad: the last slice (whose rows are partly the next group's, to be cleared)
  // is loaded as number `early` of the unit's, the MMAs read it last; else -1
  int early;
  int c0, parts;       // workers c0 .. c0 + parts - 1 share the tile
};

// Walks the list of worker w of `workers`; every role walks its own copy.
template <int SLICE, int BQ, int CL>
struct Walk {
  const Params& p;
  const Shared* sh;
  int w, workers, t, at, end;
  __device__ __forceinline__ Walk(const Params& p_, const Shared* sh_, int w_, int workers_)
      : p(p_), sh(sh_), w(w_), workers(workers_), t(w_), at(0), end(0) {
    if (w < sh->cutters) {
      at = sh->base + (int)((long long)sh->len * w / sh->cutters);
      end = sh->base + (int)((long long)sh->len * (w + 1) / sh->cutters);
    }
  }
  // last group whose entry is at most v (of equal entries the last, which has
  // the tiles)
  __device__ __forceinline__ int find(const int* a, int v) const {
    int lo = 0, hi = p.E - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a[mid] <= v) lo = mid; else hi = mid - 1;
    }
    return lo;
  }
  // the worker that has the slice at position v
  __device__ __forceinline__ int owner(int v) const {
    return (int)((((long long)(v - sh->base) + 1) * sh->cutters - 1) / sh->len);
  }
  __device__ __forceinline__ bool next(Unit& u) {
    int j, slices;
    u.parts = 1;
    if (t < sh->dp) {
      u.e = find(sh->first, t);
      j = t - sh->first[u.e];
      slices = tile_slices<SLICE>(p, sh->rows[u.e]);
      u.kb = 0;
      u.ke = slices;
      t += workers;
    } else if (at < end) {
      u.e = find(sh->pos, at);
      slices = tile_slices<SLICE>(p, sh->rows[u.e]);
      const int off = at - sh->pos[u.e];
      j = off / slices;
      u.kb = off - j * slices;
      u.ke = min(slices, u.kb + end - at);
      if (u.ke - u.kb < slices) {
        u.c0 = owner(at - u.kb);
        u.parts = owner(at - u.kb + slices - 1) - u.c0 + 1;
      }
      at += u.ke - u.kb;
    } else {
      return false;
    }
    u.row0 = sh->row0[u.e];
    const int n = sh->rows[u.e];
    const int qdim = p.wgrad ? p.Q : n;
    const int qt = cdiv(qdim, BQ);
    const int tp = j / qt;     // q fastest: workers running together share weight tiles
    u.p0 = tp * (BP * CL);
    u.q0 = (j - tp * qt) * BQ;
    u.nq = min(BQ, qdim - u.q0);
    u.nn = min(BQ, cdiv(u.nq, 16 * CL) * (16 * CL));
    u.klen = p.K == 0 ? 0 : (p.wgrad ? n : p.K);
    if (u.klen == 0) u.ke = u.kb;   // nothing to add
    // a sum that ends inside a 16-row step of its last slice
    constexpr int kEarly = early_slices(CL);
    const int n_k = u.ke - u.kb;
    u.early = p.wgrad && (u.klen & 15) && n_k > 0 && u.ke == slices ? max(0, n_k - 1 - kEarly) : -1;
    return true;
  }
};

// Waits for a barrier's phase, at most timeout_ns: then the abort word is set,
// the code recorded, and false returned. The clock is read only after some
// dozens of polls: a read takes longer than a k-slice.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort_w,
                                         int* status, int code, long long timeout_ns) {
  uint64_t t0 = 0;
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (ptx::mbar_try_wait(bar, parity)) return true;
    if (*abort_w) return false;
    const uint64_t t = ptx::global_ns();
    if (t0 == 0) {
      t0 = t;
    } else if ((long long)(t - t0) > timeout_ns) {
      *abort_w = 1;
      atomicCAS(status, 0, code);
      return false;
    }
  }
}

// The same for a barrier that threads of the peer CTA arrive on: once the phase
// is complete, one more test of it acquires at cluster scope (the phase cannot
// move on in between, its next completion needs work this thread has not
// issued yet).
__device__ __forceinline__ bool wait_for_pair(uint32_t bar, uint32_t parity, volatile int* abort_w,
                                              int* status, int code, long long timeout_ns) {
  if (!wait_for(bar, parity, abort_w, status, code, timeout_ns)) return false;
  return ptx::mbar_try_wait_cluster(bar, parity);
}

// ---- conversions --------------------------------------------------------------
// Two FP32 values into packed BF16 parts with x = h + m + l exactly (but for
// underflow): h is x rounded to nearest (and to BF16's largest value, not to
// infinity, where FP32 reaches beyond it), so at most 16 significant bits are
// left, of which m takes the first 8 and l the rest (both by truncation: two
// byte permutes instead of two conversions).
__device__ __forceinline__ void split2(float x, float y, uint32_t& h, uint32_t& m, uint32_t& l) {
  asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(y), "f"(x));
  const float rx = x - __uint_as_float(h << 16), ry = y - __uint_as_float(h & 0xFFFF0000u);
  m = __byte_perm(__float_as_uint(rx), __float_as_uint(ry), 0x7632);
  const float sx = rx - __uint_as_float(__float_as_uint(rx) & 0xFFFF0000u);
  const float sy = ry - __uint_as_float(__float_as_uint(ry) & 0xFFFF0000u);
  l = __byte_perm(__float_as_uint(sx), __float_as_uint(sy), 0x7632);
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

// The Q side of a stage, kF32: raw rows of 128 bytes (128-byte swizzle).
// K-major: row r = element r of the side, its 32 values of k -> parts with
// rows of 64 bytes (64-byte swizzle). MN-major: boxes of 32 elements x 32 rows
// of k -> chunks of 64 elements x 32 rows (128-byte swizzle). Rows of k at or
// past `klim` are written as zeros. NT threads, each 8 values at a time; U such
// pieces are loaded before the first is converted.
template <int ROWS, int NT, int U>
__device__ __forceinline__ void convert_f32(const unsigned char* raw, unsigned char* op, bool mn,
                                            int klim, int t) {
  constexpr int PART = ROWS * 64, N = ROWS * 4;
#pragma unroll 1
  for (int i0 = t; i0 < N; i0 += NT * U) {
    float4 a[U], b[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = i0 + j * NT, r = i >> 2, c = i & 3;   // MN-major: r = box * 32 + k
      if (N % (NT * U) && i >= N) continue;
      a[j] = *reinterpret_cast<const float4*>(raw + r * 128 + (((2 * c) ^ (r & 7)) << 4));
      b[j] = *reinterpret_cast<const float4*>(raw + r * 128 + (((2 * c + 1) ^ (r & 7)) << 4));
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = i0 + j * NT, r = i >> 2, c = i & 3;
      if (N % (NT * U) && i >= N) continue;
      int at;
      if (mn) {
        const int k = r & 31, box = r >> 5;
        if (k >= klim) a[j] = b[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        at = (box >> 1) * 4096 + k * 128 + ((((box & 1) * 4 + c) ^ (k & 7)) << 4);
      } else {
        at = r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
      }
      uint4 h, m, l;
      split2(a[j].x, a[j].y, h.x, m.x, l.x);
      split2(a[j].z, a[j].w, h.y, m.y, l.y);
      split2(b[j].x, b[j].y, h.z, m.z, l.z);
      split2(b[j].z, b[j].w, h.w, m.w, l.w);
      *reinterpret_cast<uint4*>(op + at) = h;
      *reinterpret_cast<uint4*>(op + PART + at) = m;
      *reinterpret_cast<uint4*>(op + 2 * PART + at) = l;
    }
  }
}

// The P side of a stage into tensor memory, a thread per element of the side
// (lane `r` of the tile, `taddr` its warp's lanes at the slot): 16 values of k
// at a time, part j at columns 16 * j .. (8 columns per 16 values).
__device__ __forceinline__ void convert_p_f32(const unsigned char* raw, uint32_t taddr, bool mn,
                                              int klim, int r) {
#pragma unroll
  for (int hk = 0; hk < 2; ++hk) {
    float v[16];
    if (mn) {
      // boxes of 32 elements x 32 rows of k: a warp reads 128 bytes a row
      const unsigned char* box = raw + (r >> 5) * 4096 + (r & 3) * 4;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int k = hk * 16 + j;
        const float x =
            *reinterpret_cast<const float*>(box + k * 128 + ((((r & 31) >> 2) ^ (k & 7)) << 4));
        v[j] = k < klim ? x : 0.f;
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<float4*>(&v[4 * c]) =
            *reinterpret_cast<const float4*>(raw + r * 128 + (((hk * 4 + c) ^ (r & 7)) << 4));
    }
    uint32_t h[8], m[8], l[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) split2(v[2 * j], v[2 * j + 1], h[j], m[j], l[j]);
    tc::tmem_st8(taddr + hk * 8, h);
    tc::tmem_st8(taddr + 16 + hk * 8, m);
    tc::tmem_st8(taddr + 32 + hk * 8, l);
  }
}
// kI8: 64 values, 32 columns.
__device__ __forceinline__ void convert_p_i8(const unsigned char* raw, uint32_t taddr, int r) {
  uint32_t o[32];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint4 v = *reinterpret_cast<const uint4*>(raw + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
    const uint2 a = i8_to_f16(v.x), b = i8_to_f16(v.y), d = i8_to_f16(v.z), e = i8_to_f16(v.w);
    o[8 * c] = a.x;
    o[8 * c + 1] = a.y;
    o[8 * c + 2] = b.x;
    o[8 * c + 3] = b.y;
    o[8 * c + 4] = d.x;
    o[8 * c + 5] = d.y;
    o[8 * c + 6] = e.x;
    o[8 * c + 7] = e.y;
  }
  tc::tmem_st32(taddr, o);
}

// The Q side, kI8: raw rows of 64 bytes (64-byte swizzle) -> rows of 64 F16
// values (128-byte swizzle).
template <int ROWS, int NT, int U>
__device__ __forceinline__ void convert_i8(const unsigned char* raw, unsigned char* op, int t) {
  constexpr int N = ROWS * 4;
#pragma unroll 1
  for (int i0 = t; i0 < N; i0 += NT * U) {
    uint4 v[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = i0 + j * NT, r = i >> 2, c = i & 3;
      if (N % (NT * U) && i >= N) continue;
      v[j] = *reinterpret_cast<const uint4*>(raw + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = i0 + j * NT, r = i >> 2, c = i & 3;
      if (N % (NT * U) && i >= N) continue;
      const uint2 a = i8_to_f16(v[j].x), b = i8_to_f16(v[j].y), d = i8_to_f16(v[j].z),
                  e = i8_to_f16(v[j].w);
      unsigned char* row = op + r * 128;
      *reinterpret_cast<uint4*>(row + (((2 * c) ^ (r & 7)) << 4)) = make_uint4(a.x, a.y, b.x, b.y);
      *reinterpret_cast<uint4*>(row + (((2 * c + 1) ^ (r & 7)) << 4)) = make_uint4(d.x, d.y, e.x, e.y);
    }
  }
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ void from_f32(float* d, float v) { *d = v; }
__device__ __forceinline__ void from_f32(__nv_bfloat16* d, float v) { *d = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(__half* d, float v) { *d = __float2half_rn(v); }

// Part of a thread's column of the tile: `n` valid values (of HC) at pitch ld,
// `live` when its p is inside the output. A warp writes 32 neighbours at a
// time. The element type, the full column and beta are decided once for all
// values: a branch per value made the unrolled loops outgrow the instruction
// cache (20 to 60 thousand cycles a tile, against one thousand). INT: scale_q
// holds the columns' scales.
template <bool INT, int HC, typename T>
__device__ __forceinline__ void write_column(T* out, long long ld, const float (&sum)[HC],
                                             float scale, const float* scale_q, float beta, int n,
                                             bool live) {
  auto value = [&](int c) {
    return INT ? (float)__float_as_int(sum[c]) * (c < n ? __ldg(scale_q + c) : 0.f) * scale
               : scale * sum[c];
  };
  if (beta == 0.f && n >= HC) {
#pragma unroll
    for (int c = 0; c < HC; ++c) {
      const float v = value(c);
      if (live) from_f32(out, v);
      out += ld;
    }
  } else {
#pragma unroll
    for (int c = 0; c < HC; ++c) {
      float v = value(c);
      if (live && c < n) {
        if (beta != 0.f) v = fmaf(beta, to_f32(*out), v);
        from_f32(out, v);
      }
      out += ld;
    }
  }
}

template <int SRC, int BQ, int CL>
__global__ void __launch_bounds__(Geo<SRC, BQ, CL>::kThreads, 1)
    ragged_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap mapP,
                  const __grid_constant__ CUtensorMap mapQ) {
  using G = Geo<SRC, BQ, CL>;
  using List = Walk<G::kSlice, BQ, CL>;
  constexpr int SL = G::kSlice;
  constexpr int RS = G::kRawStages, RB = G::kRawBars, OS = G::kConv ? G::kOpStages : RS;
  constexpr bool kPair = CL == 2;
  // weight gradients (Q stored with k as its slow dimension) take tiles of 64
  // and wider
  constexpr bool kQmn = BQ >= 64;
  static_assert(!kPair || !G::kConv, "pairs read their tiles as TMA wrote them");
  constexpr bool kReorder = kQmn && !G::kConv && early_slices(CL) > 0;
  static_assert(RS > early_slices(CL), "a slice loaded early keeps its stage");
  constexpr uint16_t kBoth = 0x3;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw_addr = ptx::smem_addr(smem_raw);
  unsigned char* base = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const uint32_t base_addr = ptx::smem_addr(base);
  // operand stages (kConv) start on 1024-byte boundaries, then the raw ones
  constexpr int kRawAt = G::kConv ? G::kOpStages * G::kOp : 0;
  unsigned char* raw_base = base + kRawAt;
  const uint32_t raw_base_addr = base_addr + kRawAt;
  Shared* sh = reinterpret_cast<Shared*>(base + G::kRegion);
  volatile int* abort_w = &sh->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = kPair ? (int)ptx::cluster_ctarank() : 0;
  const int worker = (int)blockIdx.x / CL, workers = (int)gridDim.x / CL;
  constexpr uint32_t kAll = 0xffffffffu;

  if (tid == 0) {
    // pair form: the even CTA's MMA warp waits on the stages of both CTAs, and
    // on the epilogue warps of both; its commits arrive in both
    for (int s = 0; s < RB; ++s) {
      ptx::mbar_init(ptx::smem_addr(&sh->raw_full[s]), 1);
      ptx::mbar_init(ptx::smem_addr(&sh->raw_empty[s]), G::kConv ? G::kGroupWarps : 1);
    }
    for (int s = 0; s < OS; ++s) {
      if (G::kConv) {
        ptx::mbar_init(ptx::smem_addr(&sh->op_full[s]), G::kGroupWarps);
        ptx::mbar_init(ptx::smem_addr(&sh->op_empty[s]), 1);
      }
      if (!G::kConv) {
        ptx::mbar_init(ptx::smem_addr(&sh->tail_full[s]), 1);
        ptx::mbar_init(ptx::smem_addr(&sh->peer_full[s]), 1);
      }
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(ptx::smem_addr(&sh->acc_full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&sh->acc_empty[i]), CL * kEpiWarps);
    }
    ptx::mbar_init(ptx::smem_addr(&sh->drain), 1);
    ptx::mbar_init(ptx::smem_addr(&sh->epi_sync), kEpiThreads);
    sh->abort = 0;
    ptx::mbar_fence_init();
    ptx::tma_prefetch_desc(&mapP);
    ptx::tma_prefetch_desc(&mapQ);
  }
  if (warp == 1) {
    tc::tmem_alloc<CL>(ptx::smem_addr(&sh->tmem), G::kTmemCols);
    tc::tmem_relinquish<CL>();
  }
  // launched with programmatic stream serialization: the set-up above overlaps
  // the end of the kernel ahead; nothing below touches global memory before it
  // has completed
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  if (warp == 0) {
    // scan of the groups: rows, number and slice position of each one's first
    // tile. A group starts at the end of those before it at the earliest, so the
    // groups together have at most T rows whatever the offsets hold.
    // A launch before this one that gave up may have left arrivals counted,
    // until its status is polled: then no tile is cut. (CTAs that read the word
    // on both sides of this launch's own giving up differ in their lists; the
    // launch has failed by then, and its waits end.)
    const int gave_up = *const_cast<const volatile int*>(p.status);
    const int ptiles = cdiv(p.P, BP * CL);
    int tiles_before = 0, pos_before = 0, end_before = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int lo = 0, hi = 0, n = 0, tiles = 0;
      if (e < p.E) {
        lo = p.offsets == nullptr ? 0 : min(max(p.offsets[e], 0), p.T);
        hi = p.offsets == nullptr ? p.T : min(max(p.offsets[e + 1], 0), p.T);
      }
      int ends = hi;                    // largest end up to this group
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kAll, ends, d);
        if (lane >= d) ends = max(ends, o);
      }
      const int before = __shfl_up_sync(kAll, ends, 1);
      lo = max(lo, max(end_before, lane > 0 ? before : 0));
      end_before = max(end_before, __shfl_sync(kAll, ends, 31));
      if (e < p.E) {
        n = max(hi - lo, 0);
        tiles = ptiles * cdiv(p.wgrad ? p.Q : n, BQ);
      }
      int incl = tiles, incl_pos = tiles * tile_slices<SL>(p, n);
      const int own_pos = incl_pos;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kAll, incl, d), q = __shfl_up_sync(kAll, incl_pos, d);
        if (lane >= d) {
          incl += o;
          incl_pos += q;
        }
      }
      if (e < p.E) {
        sh->row0[e] = lo;
        sh->rows[e] = n;
        sh->first[e] = tiles_before + incl - tiles;
        sh->pos[e] = pos_before + incl_pos - own_pos;
      }
      tiles_before += __shfl_sync(kAll, incl, 31);
      pos_before += __shfl_sync(kAll, incl_pos, 31);
    }
    __syncwarp();
    if (lane == 0) {
      const int tiles = tiles_before, total = pos_before;
      // whole waves first; what is left, one to two waves (or, with fewer tiles
      // than workers, all of them), by slices, unless that saves less time than
      // publishing and adding the parts takes
      const int over = tiles % workers;
      int dp = tiles, cutters = workers;
      if (over != 0 && gave_up == 0) {
        const int mean = total / tiles;
        int saved = mean * 16 / workers * (workers - over), parts = 2;
        if (tiles < workers) {
          cutters = min(workers, max(tiles, total / p.cut_least));
          parts = cutters / tiles + 1;
          saved = 16 * (mean - total / cutters);
        }
        if (saved >= p.cut_once + parts * p.cut_part) dp = max(0, tiles / workers - 1) * workers;
      }
      sh->dp = dp;
      int base_pos = total;
      if (dp == 0) {
        base_pos = 0;
      } else if (dp < tiles) {
        List l(p, sh, 0, 0);
        const int e = l.find(sh->first, dp);
        base_pos = sh->pos[e] + (dp - sh->first[e]) * tile_slices<SL>(p, sh->rows[e]);
      }
      sh->base = base_pos;
      sh->len = total - base_pos;
      sh->cutters = dp < tiles ? cutters : 0;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  // the peer's barriers must be initialised before the pair's first remote
  // arrival or commit reaches them
  if (kPair) ptx::cluster_sync();
  tc::fence_after_sync();
  const uint32_t tmem = sh->tmem;
  if (kPair) {
    if (tid == 0) {
      // the MMAs of the pair write the same tensor-memory address in both CTAs
      const uint32_t peer = ptx::ld_shared_cluster(
          ptx::mapa(ptx::smem_addr(&sh->tmem), (uint32_t)(rank ^ 1)));
      if (peer != tmem) {
        *abort_w = 1;
        atomicCAS(p.status, 0, (int)kDevTmemMismatch);
      }
    }
    __syncthreads();  // every role sees the abort word
  }

  bool issued_any = false;   // this thread has issued MMAs
  if (warp < kEpiWarp0) {
    if (G::kMoveRegs) ptx::regs_lower<G::kRegsFew>();
    // ---- warp 0: TMA producer, one thread of it -----------------------------------
    if (warp == 0 && ptx::elect_one()) {
      int it = 0, s = 0, bf = 0;            // stage and barrier to fill
      // the stage's last use: its barrier, and the parity to wait for (first
      // uses of a stage pass at once, on barriers that nothing has used)
      int be = RB == RS ? 0 : RS;
      uint32_t phase = 1;
      uint32_t tail_phase = 0;  // phases of the tail_full barriers (a bit each)
      bool ok = true;
      constexpr int BOX = G::kRawRow / G::kElem;  // elements along the fast dimension of a box
      const bool p_mn = p.p_mn, q_mn = p.q_mn, wgrad = p.wgrad;
      Unit w;
      for (List list(p, sh, worker, workers); ok && list.next(w);) {
        const int p0 = w.p0 + rank * BP, q0 = w.q0 + rank * (w.nn / CL);
        const int pe = wgrad || p.p_shared ? 0 : w.e, qrow = wgrad ? 0 : w.row0 + q0;
        const int n = w.ke - w.kb, early = kQmn && !G::kConv ? w.early : -1;
        const int first_k = w.kb * SL + (wgrad ? w.row0 : 0);
        for (int i = 0, next = 0; i < n; ++i, ++it) {
          const bool clear = i == early;
          const int k = first_k + (clear ? n - 1 : next++) * SL;
          ok = wait_for(ptx::smem_addr(&sh->raw_empty[be]), phase, abort_w, p.status,
                        kDevTimeoutEmpty, p.timeout_ns);
          if (!ok) break;
          // pair: the even CTA's barrier counts the bytes of both (the odd
          // CTA's loads may complete before it expects them), but for a stage
          // that is to be cleared. (A remote arrival for each of the odd CTA's
          // stages took its producer 1300 cycles.)
          const bool remote = kPair && rank != 0 && !clear;
          if (clear) tail_phase ^= 1u << s;
          uint32_t fb = ptx::smem_addr(clear ? &sh->tail_full[s] : &sh->raw_full[bf]);
          const uint32_t st = raw_base_addr + (uint32_t)(s * G::kRaw);
          if (remote)
            fb = ptx::mapa(fb, 0u);
          else
            ptx::mbar_arrive_expect_tx(
                fb, (uint32_t)(kPair && !clear ? 2 * G::kRaw : G::kRaw));
          auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y, int z) {
            if (kPair)
              ptx::tma_load_3d_pair(dst, map, x, y, z, fb);
            else
              ptx::tma_load_3d(dst, map, x, y, z, fb);
          };
#pragma unroll
          for (int sub = 0; sub < G::kSub; ++sub) {
            const int ksub = k + sub * G::kSubK;
            const uint32_t at = st + (uint32_t)(sub * G::kRawSub);
            if (p_mn) {
#pragma unroll
              for (int i = 0; i < BP / BOX; ++i)
                load(at + (uint32_t)(i * G::kSubK * G::kRawRow), &mapP, p0 + i * BOX, ksub, pe);
            } else {
              load(at, &mapP, ksub, p0, pe);
            }
            if (kQmn && q_mn) {
#pragma unroll
              for (int i = 0; i < G::kRows / BOX; ++i)
                load(at + (uint32_t)(G::kRawP + i * G::kSubK * G::kRawRow), &mapQ, q0 + i * BOX,
                     ksub, 0);
            } else {
              load(at + G::kRawP, &mapQ, ksub, qrow, 0);
            }
          }
          if (++s == RS) s = 0;
          if (++bf == RB) bf = 0;
          if (++be == RB) {
            be = 0;
            phase ^= 1u;
          }
        }
      }
      // nothing may land after the CTA is gone: wait (bounded) for the last
      // stages issued
      const uint64_t t0 = ptx::global_ns();
      for (int j = it - 1; j >= 0 && j >= it - RS; --j) {
        // (odd CTA: only stages that are cleared have a barrier here; the others
        // have landed once the even CTA's MMAs have read them)
        const uint32_t fb = ptx::smem_addr(kPair && rank != 0 ? &sh->tail_full[j % RS]
                                                              : &sh->raw_full[j % RB]);
        const uint32_t par = kPair && rank != 0 ? (tail_phase >> (j % RS) & 1u) ^ 1u
                                                : (uint32_t)((j / RB) & 1);
        while (!ptx::mbar_try_wait(fb, par))
          if ((long long)(ptx::global_ns() - t0) > cleanup_bound_ns(p.timeout_ns)) break;
      }
      if (kPair) {
        // the even CTA's commits arrive on this CTA's raw_empty barriers: wait
        // (bounded) for its arrivals on the last use of every stage
        for (int j = it; j < it + RS; ++j) {
          const uint32_t eb = ptx::smem_addr(&sh->raw_empty[j % RS]);
          while (!ptx::mbar_try_wait(eb, (uint32_t)((j / RS) & 1) ^ 1u))
            if ((long long)(ptx::global_ns() - t0) > cleanup_bound_ns(p.timeout_ns)) break;
        }
      }
    }
    __syncwarp();
    // ---- warp 2: clears the rows past a group's end (weight gradients) -------------
    // A slice that ends inside a 16-row step has rows of the next group in it, up
    // to that step's end (the steps beyond are not issued). They are set to zero
    // in both operands (what they hold may be no number) here, ahead of the MMAs:
    // in the MMA warp a tile's last slice cost 0.7 to 1.1 us (8 groups of 1009
    // x (4096 + 1024) 64.1 us, of 1008 56.9; here 52.9 and 50.5, with accumulations
    // of 512 rows; 73.5 and 71.6 with those of 256).
    if (!G::kConv && kQmn && warp == 2 && p.wgrad) {
      int it = 0;
      uint32_t tail_phase = 0;
      bool ok = true;
      Unit w;
      for (List list(p, sh, worker, workers); ok && list.next(w);) {
        const int s = (it + w.early) % RS, rem = w.klen - (w.ke - 1) * SL;
        it += w.ke - w.kb;
        if (w.early < 0) continue;
        const uint32_t par = tail_phase >> s & 1u;
        tail_phase ^= 1u << s;
        ok = wait_for(ptx::smem_addr(&sh->tail_full[s]), par, abort_w, p.status, kDevTimeoutFull,
                      p.timeout_ns);
        ok = __all_sync(kAll, ok);
        if (!ok) break;
        unsigned char* rows = base + s * G::kRaw + rem * 128;
        const int n = (cdiv(rem, 16) * 16 - rem) * 8;
        for (int i = lane; i < n; i += 32) {
#pragma unroll
          for (int box = 0; box < (BP + G::kRows) / 64; ++box)
            *reinterpret_cast<uint4*>(rows + box * (SL * 128) + i * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        ptx::fence_proxy_async_shared();
        __syncwarp();
        if (rank != 0) {
          if (lane == 0)
            ptx::mbar_arrive_remote(ptx::mapa(ptx::smem_addr(&sh->peer_full[s]), 0u));
        } else {
          if (kPair) {
            ok = wait_for_pair(ptx::smem_addr(&sh->peer_full[s]), par, abort_w, p.status,
                               kDevTimeoutFull, p.timeout_ns);
            ok = __all_sync(kAll, ok);
            if (!ok) break;
          }
          if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&sh->raw_full[s]));
        }
      }
    }
    // ---- warp 1: MMA issuer (even CTA of a pair), one thread of it ------------------
    if (warp == 1 && rank == 0 && ptx::elect_one()) {
    // operand tiles: K-major rows of 128 bytes (64 for kF32) in 8-row groups;
    // MN-major chunks of 64 elements x SL rows of k, 128 bytes a row. The
    // descriptors of stage 0 are made once; a stage, a part or a k-step moves
    // their address field. (Made anew for every MMA they cost more than a
    // slice's MMAs: the loop below took 540 cycles for a slice of any size.)
    constexpr bool kNarrow = SRC == kF32;
    constexpr int OP_Q = G::kConv ? G::kOpQ : G::kRawQ;   // one part
    constexpr uint32_t kStage16 = (G::kConv ? G::kOp : G::kRaw) >> 4;
    const bool a_mn = !G::kConv && p.p_mn, b_mn = kQmn && p.q_mn;   // (tensor memory: K-major)
    auto desc = [](uint32_t addr, bool mn) {
      return mn ? tc::smem_desc(addr, G::kSubK * 128, 1024, true)
                : tc::smem_desc(addr, 16, kNarrow ? 512 : 1024, !kNarrow);
    };
    const uint64_t a_desc = desc(base_addr, a_mn);
    const uint64_t b_desc = desc(base_addr + (uint32_t)(G::kConv ? 0 : G::kRawP), b_mn);
    const uint32_t a_step = a_mn ? 2048u >> 4 : 32u >> 4, b_step = b_mn ? 2048u >> 4 : 32u >> 4;
    const uint32_t a_slots = tmem + 2 * BQ;      // P's converted parts
    // the MMAs of k-step kk of stage s
    auto step = [&](uint32_t d, uint32_t idesc, int s, int kk, uint32_t add) {
      constexpr int kSteps = G::kSubK / 16;
      const int sub = kk / kSteps;
      kk -= sub * kSteps;
      const uint64_t b = b_desc + kk * b_step +
                         (uint64_t)(s * kStage16 + sub * ((G::kConv ? G::kOpSub : G::kRawSub) >> 4));
      if (G::kConv) {
        const uint32_t a = a_slots + (uint32_t)(s * G::kSlotCols + sub * G::kSubCols + kk * 8);
        if (SRC == kF32) {
          constexpr uint32_t P1 = G::kSubK / 2;
          constexpr uint64_t Q1 = OP_Q >> 4;
          tc::mma_f16_ts(d, a + 2 * P1, b, idesc, add);
          tc::mma_f16_ts(d, a, b + 2 * Q1, idesc, 1u);
          tc::mma_f16_ts(d, a + P1, b + Q1, idesc, 1u);
          tc::mma_f16_ts(d, a + P1, b, idesc, 1u);
          tc::mma_f16_ts(d, a, b + Q1, idesc, 1u);
          tc::mma_f16_ts(d, a, b, idesc, 1u);
        } else {
          tc::mma_f16_ts(d, a, b, idesc, add);
        }
      } else {
        const uint64_t a =
            a_desc + kk * a_step + (uint64_t)(s * kStage16 + sub * (G::kRawSub >> 4));
        if (kPair)
          tc::mma_f16_pair(d, a, b, idesc, add);
        else
          tc::mma_f16(d, a, b, idesc, add);
      }
    };
    auto commit = [&](uint64_t* bar) {
      if (kPair)
        tc::commit_pair_multicast(ptx::smem_addr(bar), kBoth);
      else
        tc::commit(ptx::smem_addr(bar));
    };
    int acc = 0, s = 0;
    uint32_t phase = 0;       // parity of the full barriers to wait for
    bool ok = true;
    const int chunk = p.chunk / SL;
    Unit w;
    for (List list(p, sh, worker, workers); ok && list.next(w);) {
      const int kb = w.kb, ke = w.ke, klen = w.klen, early = w.early;
      // A ragged tile's MMAs are as narrow as its rows (4096 rows over 16 groups,
      // 4096 x 2048, under sustained power 78 against 84.6 us). Where converters
      // set the pace that gains nothing.
      const uint32_t idesc = tc::idesc_f16(BP * CL, G::kConv ? BQ : w.nn,
                                           SRC == kF32 || (SRC == k16 && p.bf16), a_mn, b_mn);
      int early_s = 0, after_s = 0;
      uint32_t early_phase = 0, after_phase = 0;
      for (int k0 = kb; k0 < ke && ok; k0 += chunk, ++acc) {
        const int buf = acc & 1;
        const uint32_t d = tmem + (uint32_t)(buf * BQ);
        const uint32_t eb = ptx::smem_addr(&sh->acc_empty[buf]);
        const uint32_t par = (uint32_t)((acc >> 1) & 1) ^ 1u;
        ok = kPair ? wait_for_pair(eb, par, abort_w, p.status, kDevTimeoutSync, p.timeout_ns)
                   : wait_for(eb, par, abort_w, p.status, kDevTimeoutSync, p.timeout_ns);
        if (!ok) break;
        tc::fence_after_sync();
        const int k1 = min(ke, k0 + chunk);
        for (int ks = k0; ks < k1; ++ks) {
          const int rem = klen - ks * SL;   // > 0
          if (kReorder && early >= 0) {
            if (ks == kb + early) {         // step over the slice loaded early ...
              early_s = s;
              early_phase = phase;
              if (++s == OS) {
                s = 0;
                phase ^= 1u;
              }
            }
            if (ks == ke - 1) {             // ... and come back to it
              after_s = s;
              after_phase = phase;
              s = early_s;
              phase = early_phase;
            }
          }
          ok = wait_for(ptx::smem_addr(G::kConv ? &sh->op_full[s] : &sh->raw_full[s]), phase,
                        abort_w, p.status, kDevTimeoutFull, p.timeout_ns);
          if (!ok) break;
          tc::fence_after_sync();
          const uint32_t add = ks == k0 ? 0u : 1u;
          if (rem >= SL) {
#pragma unroll
            for (int kk = 0; kk < SL / 16; ++kk) step(d, idesc, s, kk, kk == 0 ? add : 1u);
          } else {
#pragma unroll 1
            for (int kk = 0; kk * 16 < rem; ++kk) step(d, idesc, s, kk, kk == 0 ? add : 1u);
          }
          commit(G::kConv ? &sh->op_empty[s] : &sh->raw_empty[s]);
          issued_any = true;
          if (kReorder && early >= 0 && ks == ke - 1) {
            s = after_s;
            phase = after_phase;
          } else if (++s == OS) {
            s = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        commit(&sh->acc_full[buf]);
      }
    }
    }
    __syncwarp();
  } else if (G::kConv && warp >= kConvWarp0) {
    // ---- converters: raw tiles -> operand tiles ----------------------------------
    if (G::kMoveRegs) ptx::regs_lower<G::kRegsConv>();
    const int group = (warp - kConvWarp0) / G::kGroupWarps;
    const int pr = (warp & 3) * 32 + lane;             // this thread's lane of the tile
    const int t = tid - (kConvWarp0 + group * G::kGroupWarps) * 32;
    constexpr int NT = G::kGroupWarps * 32;
    int it = 0;
    bool ok = true;
    Unit w;
    for (List list(p, sh, worker, workers); ok && list.next(w);) {
      for (int ks = w.kb; ks < w.ke; ++ks, ++it) {
        if (it % G::kConvGroups != group) continue;
        const int rs = it % RS, rb = it % RB, os = it % OS;
        ok = wait_for(ptx::smem_addr(&sh->raw_full[rb]), (uint32_t)((it / RB) & 1), abort_w,
                      p.status, kDevTimeoutFull, p.timeout_ns) &&
             wait_for(ptx::smem_addr(&sh->op_empty[os]), (uint32_t)((it / OS) & 1) ^ 1u, abort_w,
                      p.status, kDevTimeoutEmpty, p.timeout_ns);
        ok = __all_sync(kAll, ok);
        if (!ok) break;
        const unsigned char* raw = raw_base + rs * G::kRaw;
        unsigned char* op = base + os * G::kOp;
        // the MMAs that read this slot last have completed (they freed it)
        tc::fence_after_sync();
        const uint32_t slot = tmem + ((uint32_t)((warp & 3) * 32) << 16) +
                              (uint32_t)(2 * BQ + os * G::kSlotCols);
#pragma unroll 1
        for (int sub = 0; sub < G::kSub; ++sub) {
          const unsigned char* rw = raw + sub * G::kRawSub;
          const uint32_t cols = slot + (uint32_t)(sub * G::kSubCols);
          if (SRC == kF32) {
            const int klim = p.wgrad ? w.klen - ks * SL : SL;
            convert_p_f32(rw, cols, p.p_mn, klim, pr);
            convert_f32<BQ, NT, 2>(rw + G::kRawP, op + sub * G::kOpSub, kQmn && p.q_mn, klim, t);
          } else {
            convert_p_i8(rw, cols, pr);
            convert_i8<BQ, NT, BQ >= 64 ? 4 : 1>(rw + G::kRawP, op + sub * G::kOpSub, t);
          }
        }
        // the MMAs read the operand tiles, and TMA refills the raw ones,
        // through the async proxy
        ptx::fence_proxy_async_shared();
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(ptx::smem_addr(&sh->op_full[os]));
          ptx::mbar_arrive(ptx::smem_addr(&sh->raw_empty[rb]));
        }
      }
    }
  } else {
    // ---- epilogue: accumulators -> registers -> output or partial tile -------------
    if (G::kMoveRegs) ptx::regs_raise<G::kRegsMany>();
    constexpr int HC = BQ / 2;                         // columns of this warp
    constexpr int CH = HC < 32 ? HC : 32;              // columns per tensor-memory read
    const int quarter = warp & 3;                      // TMEM lanes 32*quarter ..
    const int half = (warp - kEpiWarp0) >> 2;
    const int pr = quarter * 32 + lane;                // this thread's p within the tile
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    uint32_t sync_phase = 0;
    auto epi_sync = [&]() -> bool {                    // bounded rendezvous of the epilogue
      ptx::mbar_arrive(ptx::smem_addr(&sh->epi_sync));
      const bool ok = wait_for(ptx::smem_addr(&sh->epi_sync), sync_phase, abort_w, p.status,
                                   kDevTimeoutSync, p.timeout_ns);
      sync_phase ^= 1u;
      return __all_sync(kAll, ok);
    };
    const int chunk = p.chunk / SL;
    int acc = 0;
    bool ok = true;
    Unit w;
    for (List list(p, sh, worker, workers); ok && list.next(w);) {
      const int nq = w.nq - half * HC;                 // valid columns of this warp (may be <= 0)
      const int pp = w.p0 + rank * BP + pr;
      const bool live = pp < p.P;
      const float sp = !G::kInt ? p.alpha : (live ? p.scale_p[pp] : 0.f);
      const long long row = (long long)(p.wgrad ? 0 : w.row0) + w.q0 + half * HC;
      const long long at = (p.wgrad ? (long long)w.e * p.stride_o : 0ll) + row * p.ldo + pp;
      // writes the sums of N columns from column c0 on
      auto write = [&](const auto& sums, int c0) {
        constexpr int N = sizeof(sums) / sizeof(float);
        const float* sq = G::kInt ? p.scale_q + row + c0 : nullptr;
        const long long a = at + c0 * p.ldo;
        if (p.out_type == kOutF32)
          write_column<G::kInt, N>(static_cast<float*>(p.out) + a, p.ldo, sums, sp, sq, p.beta,
                                   nq - c0, live);
        else if (p.out_type == kOutBf16)
          write_column<G::kInt, N>(static_cast<__nv_bfloat16*>(p.out) + a, p.ldo, sums, sp, sq,
                                   p.beta, nq - c0, live);
        else
          write_column<G::kInt, N>(static_cast<__half*>(p.out) + a, p.ldo, sums, sp, sq, p.beta,
                                   nq - c0, live);
      };
      // CH columns of the accumulator in use; integers as such, in the same registers
      auto load = [&](int c0, float (&v)[CH]) {
        uint32_t* r = reinterpret_cast<uint32_t*>(v);
        const uint32_t src = tmem + lane_base + (uint32_t)((acc & 1) * BQ + half * HC + c0);
        if constexpr (CH == 8) {
          tc::tmem_ld8(src, *reinterpret_cast<uint32_t(*)[8]>(r));
        } else {
#pragma unroll
          for (int i = 0; i < CH; i += 16)
            tc::tmem_ld16(src + (uint32_t)i, *reinterpret_cast<uint32_t(*)[16]>(r + i));
        }
        tc::tmem_wait_ld();
        if (G::kInt) {
#pragma unroll
          for (int i = 0; i < CH; ++i) v[i] = __int_as_float(__float2int_rn(v[i]));
        }
      };
      auto acquire = [&]() -> bool {                   // waits for the next accumulator
        const bool full =
            wait_for(ptx::smem_addr(&sh->acc_full[acc & 1]), (uint32_t)((acc >> 1) & 1), abort_w,
                     p.status, kDevTimeoutFull, p.timeout_ns);
        const bool all = __all_sync(kAll, full);
        tc::fence_after_sync();
        return all;
      };
      auto release = [&] {                             // all of its columns have been read
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          // the even CTA's MMA warp waits for the epilogues of both
          uint64_t* bar = &sh->acc_empty[acc & 1];
          if (kPair && rank != 0)
            ptx::mbar_arrive_remote(ptx::mapa(ptx::smem_addr(bar), 0u));
          else
            ptx::mbar_arrive(ptx::smem_addr(bar));
        }
        ++acc;
      };
      // this range's partial tile: slot 1 of this CTA for the range that starts
      // the tile, else slot 0
      auto slot = [&](int c, int which) -> float* {
        return p.partials + (((long long)c * 2 + which) * CL + rank) * (BP * BQ) + half * HC * BP + pr;
      };
      float* part = slot(worker, w.kb == 0 ? 1 : 0);

      // Sums that are all in one accumulation go straight from tensor memory to
      // their place, CH columns at a time in a rolled loop: a tile's first
      // pass through unrolled code waits for the instructions (3 us for 128
      // columns), which is most of a small call's epilogue. Others are added up
      // in registers, which only unrolled code can index.
      if (w.ke > w.kb && w.ke - w.kb <= chunk) {
        ok = acquire();
        if (!ok) break;
#pragma unroll 1
        for (int c0 = 0; c0 < HC && c0 < nq; c0 += CH) {
          float v[CH];
          load(c0, v);
          if (w.parts > 1) {
#pragma unroll
            for (int c = 0; c < CH; ++c)
              if (c0 + c < nq) __stcg(part + (c0 + c) * BP, v[c]);
          } else {
            write(v, c0);
          }
        }
        release();
      } else {
        float sum[HC];
#pragma unroll
        for (int c = 0; c < HC; ++c) sum[c] = 0.f;
        for (int k0 = w.kb; k0 < w.ke; k0 += chunk) {
          ok = acquire();
          if (!ok) break;
#pragma unroll
          for (int c0 = 0; c0 < HC; c0 += CH) {
            if (c0 >= nq) continue;                    // (the whole warp)
            float v[CH];
            load(c0, v);
#pragma unroll
            for (int i = 0; i < CH; ++i) {
              if (G::kInt)
                sum[c0 + i] = __int_as_float(__float_as_int(sum[c0 + i]) + __float_as_int(v[i]));
              else
                sum[c0 + i] += v[i];
            }
          }
          release();
        }
        if (!ok) break;
        if (w.parts > 1) {
#pragma unroll
          for (int c = 0; c < HC; ++c)
            if (c < nq) __stcg(part + c * BP, sum[c]);
        } else if (nq > 0) {
          write(sum, 0);
        }
      }
      if (w.parts > 1) {
        // all of the partial tile is written; the last worker to arrive adds
        // the parts in the order of k
        __threadfence();
        ok = epi_sync();
        if (!ok) break;
        if (warp == kEpiWarp0 && lane == 0) {
          uint32_t* counter = p.counters + w.c0 * CL + rank;
          const int last = atomicAdd(counter, 1u) == (uint32_t)(w.parts - 1);
          if (last) *counter = 0u;                     // ready for the next launch
          __threadfence();
          sh->last = last;
        }
        ok = epi_sync();
        if (!ok) break;
        if (!*reinterpret_cast<volatile int*>(&sh->last)) continue;
        __threadfence();
        // LP partials by CH columns are loaded at a time: one after another,
        // each would cost the latency of L2
        constexpr int LP = 32 / CH;
#pragma unroll 1
        for (int c0 = 0; c0 < HC && c0 < nq; c0 += CH) {
          float sum[CH];
#pragma unroll
          for (int c = 0; c < CH; ++c) sum[c] = 0.f;
#pragma unroll 1
          for (int i0 = 0; i0 < w.parts; i0 += LP) {
            float x[LP][CH];
#pragma unroll
            for (int i = 0; i < LP; ++i) {
              const float* src = slot(w.c0 + i0 + i, i0 + i == 0 ? 1 : 0) + c0 * BP;
#pragma unroll
              for (int c = 0; c < CH; ++c)
                x[i][c] = i0 + i < w.parts && c0 + c < nq ? __ldcg(src + c * BP) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < LP; ++i) {
#pragma unroll
              for (int c = 0; c < CH; ++c) {
                if (G::kInt)
                  sum[c] = __int_as_float(__float_as_int(sum[c]) + __float_as_int(x[i][c]));
                else
                  sum[c] += x[i][c];
              }
            }
          }
          write(sum, c0);
        }
      }
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  // A CTA that gives up waits (bounded) until every MMA it issued has completed:
  // here, since any role may be the one that gives up, with the last MMAs in
  // flight and their issuer done. (Where none has, the epilogue has waited for
  // all of them.)
  if (issued_any && *abort_w != 0) {
    if (kPair)
      tc::commit_pair(ptx::smem_addr(&sh->drain));
    else
      tc::commit(ptx::smem_addr(&sh->drain));
    const uint64_t t0 = ptx::global_ns();
    while (!ptx::mbar_try_wait(ptx::smem_addr(&sh->drain), 0u))
      if ((long long)(ptx::global_ns() - t0) > cleanup_bound_ns(p.timeout_ns)) break;
  }
  __syncwarp();
  // the even CTA's MMAs write the odd CTA's tensor memory and read its shared
  // memory: the pair frees its tensor memory together, once both are done
  if (kPair) ptx::cluster_sync();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc<CL>(tmem, G::kTmemCols);
  }
}

}  // namespace ragged
}  // namespace sgemm_gb300
