// mx4_gemm.cu -- sgemm_mx4: the product of two matrices of 4-bit floating point
// with a power of two for every 32 values of k, on the block-scaled tensor-core
// instruction (tcgen05.mma kind::mxf4).
//
// Mathematics: C[m, n] = sum_k A[m, k] B[n, k] 2^(sA[m, k / 32] + sB[n, k / 32] -
// 254). A product of two codes and its powers is exact; the tensor core adds them
// up in FP32.
//
// The 128 lanes of the instruction are output features (rows of B: P below), its
// columns are tokens (rows of A: Q), so a few tokens cost a narrow tile while the
// weights stream through full ones. A slice is 256 values of k, 128 bytes a row,
// four instructions. Its scales arrive by TMA beside the codes, as the 512-byte
// tiles of 128 rows x 4 blocks that they are stored in, and are copied to tensor
// memory by tcgen05.cp in the stream of the MMAs.
//
// Tensor memory. Each slice's scales have columns of their own until its MMAs are
// done: with two slices' worth the issuer waited for MMAs that had just been
// queued (8192 x 8192 x 8192 264 us, 172 without that wait). Beside them two
// 256-wide accumulators do not fit, so the second one's first half is the first
// one's second. The epilogue takes its columns into registers before it writes
// any, and the next tile's MMAs start once the shared half is read.
//
// Roles: warp 0 issues the loads, warp 1 the scales' copies and the MMAs, warps
// 4-11 read the accumulators (two warps a lane quarter, each half of the columns)
// and write. CL = 2: pairs of CTAs on vertically adjacent tiles, whose even CTA
// issues M = 256 MMAs over both; each holds its 128 rows of P, half of Q's rows
// and all of Q's scales.
//
// Schedule: whole tiles in turn. Where there are few tiles each is cut into 2, 4
// or 8 ranges of k, one for each CTA of a cluster (SPLIT). They leave their parts
// in their shared memory, and each adds some of the columns over all of them, in
// the order of k. (Through L2, by the last of them to arrive, the exchange of two
// 128 x 256 tiles took 9 us.)
//
// Measured on GB300: 8192 x 8192 x 4096 91 us, 6.0 PFLOP/s, x 8192 153 us, 7.2; 1 x
// 4096 x 4096 5.0 us, 512 x 4096 x 4096 8.1, 1000 x 300 x 4096 7.0. A slice of a
// pair's tile takes 300 ns: its MMAs 256 at the instruction's rate, its 35 KB at 64
// bytes a cycle into each SM 285. A tile costs 2.3 us beside its slices, of which the
// epilogue's half that the next tile waits for is 0.7. What did not help: the scales'
// copies issued by a warp of their own (97 us: a stage is held longer), blocks of
// tiles instead of rows of them (96: the divisions between tiles), all of an
// accumulator's columns read at once (92). The narrow tiles are bound by latency:
// launch and first loads 3 us, the exchange of parts 1.5.
//
// Every wait is bounded; a CTA that gives up drains its copies and MMAs, frees
// its tensor memory and returns.
#include <cuda.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdio>
#include <mutex>

#include "../../include/sgemm_gb300.h"
#include "elements.cuh"
#include "ragged_launch.cuh"

#define SGEMM_API extern "C" __attribute__((visibility("default")))

namespace sgemm_gb300 {
namespace mx4 {
namespace {

constexpr int BP = 128;                    // rows of P in a CTA
constexpr int kSliceK = 256, kRow = 128;   // values of k in a slice, their bytes
constexpr int kEpiWarp0 = 4, kEpiWarps = 8, kThreads = (kEpiWarp0 + kEpiWarps) * 32;
constexpr uint32_t kAll = 0xffffffffu;

struct Params {
  int P, Q, K;              // features, tokens, values of k
  int chunk;                // slices of one accumulation
  void* out;
  long long ldo;
  int out_type;
  // C's rows are at multiples of 16 bytes: 32 features at a time are written by TMA, the
  // last ones too (1), or by their threads (2)
  int tma_out;
  int* status;
  long long timeout_ns;
};

template <int BQ, int CL>
struct Geo {
  static constexpr int kRowsQ = BQ / CL;                       // rows of Q in a CTA
  static constexpr int kTilesQ = (BQ + 127) / 128;             // scale tiles of Q
  static constexpr int kP = BP * kRow, kQ = kRowsQ * kRow;
  static constexpr int kScaleP = 1024, kScaleQ = 1024 * kTilesQ;   // two blocks of 4 each
  static constexpr int kStage = kP + kQ + kScaleP + kScaleQ;
  // wide tiles: the epilogue's pieces of 32 x 32 on their way out, 4 KB a warp
  static constexpr bool kStaged = BQ >= 128;
  static constexpr int kRegion = (kStaged ? 176 : 208) * 1024;
  static constexpr int kFit = kRegion / kStage;
  static constexpr int kStages = kFit < 10 ? kFit : 10;
  static_assert(kStage % 1024 == 0 && kStages >= 3, "stages");
  // columns of a slice's scales, and where things lie in tensor memory
  static constexpr int kCols = 8 + 8 * kTilesQ;
  static constexpr bool kShare = BQ == 256;                    // accumulators share a half
  static constexpr int kSecond = kShare ? BQ / 2 : BQ;         // the second accumulator
  static constexpr int kScales = kSecond + BQ;
  // each stage's scales have columns of their own: the MMAs that read them last are done
  // once the stage has been loaded again
  static constexpr int kUsed = kScales + kStages * kCols;
  // A thread of a wide tile's epilogue holds 128 sums: it needs more registers
  // than the launch gives every thread, so the other warps give some up.
  static constexpr bool kMoveRegs = BQ == 256;
  static constexpr int kRegs = 168, kRegsFew = 72, kRegsMany = 216;
  static_assert(128 * kRegsFew + 256 * kRegsMany <= kThreads * kRegs && kThreads * kRegs <= 65536,
                "register shares");
  static constexpr int kTmem = kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
  static_assert(kUsed <= 512, "tensor memory");
};

struct Shared {
  uint64_t full[10], empty[10];
  uint64_t acc_full[2], acc_empty[2], acc_part[2];
  uint64_t drain;
  uint32_t tmem;
  int abort;
};
constexpr int kOut = 4096;                 // of a warp
constexpr int kSmem = 1024 + 208 * 1024 + 512;
static_assert(sizeof(Shared) <= 512 && kSmem <= 227 * 1024, "shared memory");

using ragged::cdiv;
using ragged::wait_for;
using ragged::wait_for_pair;

// Part of a worker's list: slices kb .. ke of the tile (p0, q0).
struct Unit {
  int p0, q0, nq, nn, kb, ke;
};

template <typename T>
__device__ __forceinline__ void put(T* out, long long at, int n, const float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) out[at + i] = rows::from_f32<T>(v[i]);
}

template <int BQ, int CL, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    mx4_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap map_p,
               const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_sp,
               const __grid_constant__ CUtensorMap map_sq,
               const __grid_constant__ CUtensorMap map_out) {
  using G = Geo<BQ, CL>;
  constexpr bool kPair = CL == 2;
  static_assert(!SPLIT || (!kPair && BQ <= 128 && BQ * BP * 4 <= G::kRegion), "cut tiles");
  constexpr int S = G::kStages;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw_addr = ptx::smem_addr(smem_raw);
  unsigned char* base = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const uint32_t base_addr = ptx::smem_addr(base);
  Shared* sh = reinterpret_cast<Shared*>(base + 208 * 1024);
  static_assert(!G::kStaged || G::kRegion + kEpiWarps * kOut <= 208 * 1024, "staged output");
  volatile int* abort_w = &sh->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = kPair ? (int)ptx::cluster_ctarank() : 0;
  const int split = SPLIT ? (int)ptx::cluster_nctarank() : 1;
  const int part = SPLIT ? (int)ptx::cluster_ctarank() : 0;
  const int worker = (int)blockIdx.x / (SPLIT ? split : CL), workers = (int)gridDim.x / (SPLIT ? split : CL);

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      ptx::mbar_init(ptx::smem_addr(&sh->full[s]), 1);
      ptx::mbar_init(ptx::smem_addr(&sh->empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(ptx::smem_addr(&sh->acc_full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&sh->acc_empty[i]), CL * kEpiWarps);
      ptx::mbar_init(ptx::smem_addr(&sh->acc_part[i]), CL * kEpiWarps / 2);
    }
    ptx::mbar_init(ptx::smem_addr(&sh->drain), 1);
    sh->abort = 0;
    ptx::mbar_fence_init();
    ptx::tma_prefetch_desc(&map_p);
    ptx::tma_prefetch_desc(&map_q);
    ptx::tma_prefetch_desc(&map_sp);
    ptx::tma_prefetch_desc(&map_sq);
    if (G::kStaged && p.tma_out) ptx::tma_prefetch_desc(&map_out);
  }
  if (warp == 1) {
    tc::tmem_alloc<CL>(ptx::smem_addr(&sh->tmem), G::kTmem);
    tc::tmem_relinquish<CL>();
  }
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  tc::fence_before_sync();
  __syncthreads();
  if (kPair) ptx::cluster_sync();
  tc::fence_after_sync();
  const uint32_t tmem = sh->tmem;
  if (kPair) {
    if (tid == 0) {
      const uint32_t peer =
          ptx::ld_shared_cluster(ptx::mapa(ptx::smem_addr(&sh->tmem), (uint32_t)(rank ^ 1)));
      if (peer != tmem) {
        *abort_w = 1;
        atomicCAS(p.status, 0, (int)kDevTmemMismatch);
      }
    }
    __syncthreads();  // every role sees the abort word
  }
  const int slices = cdiv(p.K, kSliceK), tiles_q = cdiv(p.Q, BQ);
  const int tiles_p = cdiv(p.P, BP * CL);
  // A worker's tiles, q fastest (workers running together share weight tiles), every
  // `workers`-th: a step is so many tiles of q, and of p, on (divisions between
  // two tiles of the load loop cost what a slice costs).
  const int step_p = workers / tiles_q, step_q = workers - step_p * tiles_q;
  struct At {
    int p, q;
  };
  auto start = [&] {
    At t;
    t.p = worker / tiles_q;
    t.q = worker - t.p * tiles_q;
    return t;
  };
  auto advance = [&](At& t) {
    t.p += step_p;
    t.q += step_q;
    if (t.q >= tiles_q) {
      t.q -= tiles_q;
      ++t.p;
    }
  };
  auto unit = [&](const At& t) {
    Unit u;
    u.p0 = t.p * (BP * CL);
    u.q0 = t.q * BQ;
    u.nq = min(BQ, p.Q - u.q0);
    u.nn = min(BQ, cdiv(u.nq, 16 * CL) * (16 * CL));
    u.kb = SPLIT ? (int)((long long)slices * part / split) : 0;
    u.ke = SPLIT ? (int)((long long)slices * (part + 1) / split) : slices;
    return u;
  };

  bool issued_any = false;
  if (G::kMoveRegs && warp < kEpiWarp0) ptx::regs_lower<G::kRegsFew>();
  if (warp == 0) {
    // ---- loads, one thread -------------------------------------------------------
    if (ptx::elect_one()) {
      int it = 0;
      bool ok = true;
      for (At t = start(); ok && t.p < tiles_p; advance(t)) {
        const Unit u = unit(t);
        const int p0 = u.p0 + rank * BP, q0 = u.q0 + rank * (u.nn / CL);
        for (int ks = u.kb; ks < u.ke; ++ks, ++it) {
          const int s = it % S;
          ok = wait_for(ptx::smem_addr(&sh->empty[s]), (uint32_t)((it / S) & 1) ^ 1u, abort_w,
                        p.status, kDevTimeoutEmpty, p.timeout_ns);
          if (!ok) break;
          // pair: the even CTA's barrier counts the bytes of both
          uint32_t fb = ptx::smem_addr(&sh->full[s]);
          const uint32_t st = base_addr + (uint32_t)(s * G::kStage);
          if (kPair && rank != 0)
            fb = ptx::mapa(fb, 0u);
          else
            ptx::mbar_arrive_expect_tx(fb, (uint32_t)(CL * G::kStage));
          auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y) {
            if (kPair)
              ptx::tma_load_3d_pair(dst, map, x, y, 0, fb);
            else
              ptx::tma_load_3d(dst, map, x, y, 0, fb);
          };
          load(st, &map_p, ks * kRow, p0);
          load(st + G::kP, &map_q, ks * kRow, q0);
          load(st + G::kP + G::kQ, &map_sp, ks * 256, p0 >> 7);
          load(st + G::kP + G::kQ + G::kScaleP, &map_sq, ks * 256, u.q0 >> 7);
        }
      }
      // nothing may land after the CTA is gone (the odd CTA's loads signal the
      // even one's barriers: they have landed once its MMAs have read them)
      const uint64_t t0 = ptx::global_ns();
      if (!kPair || rank == 0) {
        for (int j = it - 1; j >= 0 && j >= it - S; --j)
          while (!ptx::mbar_try_wait(ptx::smem_addr(&sh->full[j % S]), (uint32_t)((j / S) & 1)))
            if ((long long)(ptx::global_ns() - t0) > cleanup_bound_ns(p.timeout_ns)) break;
      }
      if (kPair) {
        for (int j = it; j < it + S; ++j)
          while (!ptx::mbar_try_wait(ptx::smem_addr(&sh->empty[j % S]), (uint32_t)((j / S) & 1) ^ 1u))
            if ((long long)(ptx::global_ns() - t0) > cleanup_bound_ns(p.timeout_ns)) break;
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- scales to tensor memory and MMAs, one thread of the even CTA ---------------
    if (rank == 0 && ptx::elect_one()) {
      auto commit = [&](uint64_t* bar) {
        if (kPair)
          tc::commit_pair_multicast(ptx::smem_addr(bar), (uint16_t)0x3);
        else
          tc::commit(ptx::smem_addr(bar));
      };
      auto wait_acc = [&](uint64_t* bar, uint32_t parity) {
        return kPair ? wait_for_pair(ptx::smem_addr(bar), parity, abort_w, p.status, kDevTimeoutSync,
                                     p.timeout_ns)
                     : wait_for(ptx::smem_addr(bar), parity, abort_w, p.status, kDevTimeoutSync,
                                p.timeout_ns);
      };
      const uint64_t a_desc = tc::smem_desc(base_addr, 16, 1024, true);
      const uint64_t b_desc = tc::smem_desc(base_addr + G::kP, 16, 1024, true);
      int it = 0, acc = 0;
      bool ok = true;
      for (At t = start(); ok && t.p < tiles_p; advance(t)) {
        const Unit u = unit(t);
        const uint32_t idesc[2] = {tc::idesc_mx4(BP * CL, u.nn, 0), tc::idesc_mx4(BP * CL, u.nn, 2)};
        for (int k0 = u.kb; k0 < u.ke && ok; k0 += p.chunk, ++acc) {
          const int buf = acc & 1;
          ok = wait_acc(&sh->acc_empty[buf], (uint32_t)((acc >> 1) & 1) ^ 1u);
          if (ok && G::kShare && acc > 0)
            ok = wait_acc(&sh->acc_part[buf ^ 1], (uint32_t)(((acc - 1) >> 1) & 1));
          if (!ok) break;
          tc::fence_after_sync();
          const uint32_t d = tmem + (uint32_t)(buf * G::kSecond);
          const int k1 = min(u.ke, k0 + p.chunk);
          for (int ks = k0; ks < k1; ++ks, ++it) {
            const int s = it % S;
            ok = wait_for(ptx::smem_addr(&sh->full[s]), (uint32_t)((it / S) & 1), abort_w, p.status,
                          kDevTimeoutFull, p.timeout_ns);
            if (!ok) break;
            tc::fence_after_sync();
            const uint32_t st = (uint32_t)(s * G::kStage);
            const uint32_t scales = base_addr + st + G::kP + G::kQ;
            const uint32_t sp = tmem + (uint32_t)(G::kScales + s * G::kCols), sq = sp + 8;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              tc::copy_scales<CL>(sp + h * 4, scales + h * 512);
#pragma unroll
              for (int t = 0; t < G::kTilesQ; ++t)
                tc::copy_scales<CL>(sq + (h * G::kTilesQ + t) * 4,
                                    scales + G::kScaleP + t * 1024 + h * 512);
            }
            const int steps = min(4, cdiv(p.K - ks * kSliceK, 64));
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              if (kk < steps)
                tc::mma_mx4<CL>(d, a_desc + (st >> 4) + kk * 2, b_desc + (st >> 4) + kk * 2,
                                idesc[kk & 1], sp + (kk >> 1) * 4, sq + (kk >> 1) * (G::kTilesQ * 4),
                                ks > k0 || kk > 0 ? 1u : 0u);
            commit(&sh->empty[s]);
            issued_any = true;
          }
          if (!ok) break;
          commit(&sh->acc_full[buf]);
        }
      }
    }
    __syncwarp();
  } else if (warp >= kEpiWarp0) {
    // ---- epilogue ------------------------------------------------------------------
    if (G::kMoveRegs) ptx::regs_raise<G::kRegsMany>();
    constexpr int HC = BQ / 2, CH = HC < 32 ? HC : 32;
    const int quarter = warp & 3, half = (warp - kEpiWarp0) >> 2;
    const int pr = quarter * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const int col0 = half * HC;                        // this warp's columns of the tile
    auto arrive = [&](uint64_t* bar) {
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (kPair && rank != 0)
          ptx::mbar_arrive_remote(ptx::mapa(ptx::smem_addr(bar), 0u));
        else
          ptx::mbar_arrive(ptx::smem_addr(bar));
      }
    };
    int acc = 0, boxes = 0;
    bool ok = true;
    for (At t = start(); ok && t.p < tiles_p; advance(t)) {
      const Unit u = unit(t);
      const int pp = u.p0 + rank * BP + pr;
      const bool live = pp < p.P;
      // v: this lane's feature of the tile's columns c .. c + CH - 1
      auto write = [&](const float (&v)[CH], int c) {
        const int n = u.nq - c;                        // valid columns from the tile's c-th on
        if constexpr (G::kStaged) {
          // token by token into the warp's buffer (16 bits: one of two, in turn),
          // then out as one box; lane by lane where C's rows do not allow that (every
          // box commits a group, an empty one then, as the waits count them)
          const bool f32 = p.out_type == SGEMM_TYPE_F32;
          unsigned char* buf = base + G::kRegion + (warp - kEpiWarp0) * kOut;
          if (f32) {
            ptx::bulk_wait_read<0>();
          } else {
            ptx::bulk_wait_read<1>();
            buf += (boxes & 1) * (kOut / 2);
          }
          __syncwarp();
          if (f32) {
            float* o = reinterpret_cast<float*>(buf) + lane;
#pragma unroll
            for (int j = 0; j < CH; ++j) o[j * 32] = v[j];
          } else if (p.out_type == SGEMM_TYPE_BF16) {
            __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(buf) + lane;
#pragma unroll
            for (int j = 0; j < CH; ++j) o[j * 32] = __float2bfloat16_rn(v[j]);
          } else {
            __half* o = reinterpret_cast<__half*>(buf) + lane;
#pragma unroll
            for (int j = 0; j < CH; ++j) o[j * 32] = __float2half_rn(v[j]);
          }
          if (p.tma_out == 1 || (p.tma_out == 2 && pp - lane + 32 <= p.P)) {
            ptx::fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
              if (pp < p.P)
                ptx::tma_store_3d(&map_out, ptx::smem_addr(buf), pp, u.q0 + c, 0);
              ptx::bulk_commit();
            }
          } else {
            if (lane == 0) ptx::bulk_commit();
            __syncwarp();
            const long long at = (long long)(u.q0 + c) * p.ldo + pp;
#pragma unroll 4
            for (int j = 0; j < min(n, CH); ++j) {
              if (!live) continue;
              if (f32)
                static_cast<float*>(p.out)[at + j * p.ldo] = reinterpret_cast<float*>(buf)[j * 32 + lane];
              else
                static_cast<uint16_t*>(p.out)[at + j * p.ldo] =
                    reinterpret_cast<uint16_t*>(buf)[j * 32 + lane];
            }
          }
          ++boxes;
        } else {
          const long long at = (long long)(u.q0 + c) * p.ldo + pp;
          if (p.out_type == SGEMM_TYPE_F32)
            ragged::write_column<false, CH>(static_cast<float*>(p.out) + at, p.ldo, v, 1.f, nullptr,
                                            0.f, n, live);
          else if (p.out_type == SGEMM_TYPE_BF16)
            ragged::write_column<false, CH>(static_cast<__nv_bfloat16*>(p.out) + at, p.ldo, v, 1.f,
                                            nullptr, 0.f, n, live);
          else
            ragged::write_column<false, CH>(static_cast<__half*>(p.out) + at, p.ldo, v, 1.f, nullptr,
                                            0.f, n, live);
        }
      };
      auto load = [&](int c, float (&v)[CH]) {
        uint32_t* r = reinterpret_cast<uint32_t*>(v);
        const uint32_t src = tmem + lane_base + (uint32_t)((acc & 1) * G::kSecond + col0 + c);
        if constexpr (CH == 8) {
          tc::tmem_ld8(src, *reinterpret_cast<uint32_t(*)[8]>(r));
        } else {
#pragma unroll
          for (int j = 0; j < CH; j += 16)
            tc::tmem_ld16(src + (uint32_t)j, *reinterpret_cast<uint32_t(*)[16]>(r + j));
        }
        tc::tmem_wait_ld();
      };
      auto acquire = [&]() -> bool {
        const bool full = wait_for(ptx::smem_addr(&sh->acc_full[acc & 1]), (uint32_t)((acc >> 1) & 1),
                                   abort_w, p.status, kDevTimeoutFull, p.timeout_ns);
        const bool all = __all_sync(kAll, full);
        tc::fence_after_sync();
        return all;
      };
      auto release = [&] {
        // the half that both accumulators have: the first one's second
        if (G::kShare && half == ((acc & 1) ^ 1)) arrive(&sh->acc_part[acc & 1]);
        arrive(&sh->acc_empty[acc & 1]);
        ++acc;
      };
      // a cut tile's part: column after column of 128 lanes, where the stages were
      auto keep = [&](const float (&v)[CH], int c) {
        float* o = reinterpret_cast<float*>(base) + c * BP + pr;
#pragma unroll
        for (int j = 0; j < CH; ++j) o[j * BP] = v[j];
      };
      if (!G::kShare && u.ke - u.kb <= p.chunk) {
        // one accumulation: from tensor memory to its place, in a rolled loop (a
        // tile's first pass through unrolled code waits for the instructions)
        ok = acquire();
        if (!ok) break;
#pragma unroll 1
        for (int c0 = 0; c0 < HC; c0 += CH) {
          const int c = col0 + c0;
          if (c >= u.nq) break;
          float v[CH];
          load(c0, v);
          if (SPLIT)
            keep(v, c);
          else
            write(v, c);
        }
        release();
      } else {
        float sum[HC];
#pragma unroll
        for (int c = 0; c < HC; ++c) sum[c] = 0.f;
        for (int k0 = u.kb; k0 < u.ke; k0 += p.chunk) {
          ok = acquire();
          if (!ok) break;
#pragma unroll
          for (int c0 = 0; c0 < HC; c0 += CH) {
            if (col0 + c0 < u.nq) {                    // (the whole warp)
              float v[CH];
              load(c0, v);
#pragma unroll
              for (int j = 0; j < CH; ++j) sum[c0 + j] += v[j];
            }
          }
          release();
        }
        if (!ok) break;
#pragma unroll
        for (int c0 = 0; c0 < HC; c0 += CH) {
          const int c = col0 + c0;
          if (c >= u.nq) continue;
          float v[CH];
#pragma unroll
          for (int j = 0; j < CH; ++j) v[j] = sum[c0 + j];
          if (SPLIT)
            keep(v, c);
          else
            write(v, c);
        }
      }
    }
    if (G::kStaged && !SPLIT) ptx::bulk_wait();                  // the buffers are read, C is written
  }

  tc::fence_before_sync();
  __syncthreads();
  // a CTA that gives up waits (bounded) for every MMA it issued
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
  if (kPair) ptx::cluster_sync();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc<CL>(tmem, G::kTmem);
  }
  if constexpr (SPLIT) {
    // every thread of every CTA of the cluster comes here, whoever gave up
    ptx::cluster_sync();
    const Unit u = unit(start());
    // a warp a column, four features a lane
    for (int c = part + split * warp; c < u.nq; c += split * (kThreads / 32)) {
      const uint32_t at = base_addr + (uint32_t)(c * BP + lane * 4) * 4u;
      float4 x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < split) x[i] = ptx::ld_shared_cluster_v4(ptx::mapa(at, (uint32_t)i));
      float4 s = x[0];
#pragma unroll
      for (int i = 1; i < 8; ++i)
        if (i < split) {
          s.x += x[i].x;
          s.y += x[i].y;
          s.z += x[i].z;
          s.w += x[i].w;
        }
      const float v[4] = {s.x, s.y, s.z, s.w};
      const int pp = u.p0 + lane * 4, n = min(4, p.P - pp);
      const long long o = (long long)(u.q0 + c) * p.ldo + pp;
      if (p.out_type == SGEMM_TYPE_F32)
        put(static_cast<float*>(p.out), o, n, v);
      else if (p.out_type == SGEMM_TYPE_BF16)
        put(static_cast<__nv_bfloat16*>(p.out), o, n, v);
      else
        put(static_cast<__half*>(p.out), o, n, v);
    }
    ptx::cluster_sync();      // the others have read this CTA's part
  }
}

// ---- host ---------------------------------------------------------------------------
// The built kernels, with what they take on GB300, in ns: a slice, and a tile
// beside its slices (8192 x 8192 x 4096 and x 8192; narrow ones 4864 x 16 .. 64).
struct Form {
  int bq, cl;
  bool split;
  int slice, tile;
  const void* kernel;
};
#define SGEMM_GB300_MX4(BQ, CL, SPLIT, SLICE, TILE) \
  {BQ, CL, SPLIT, SLICE, TILE, reinterpret_cast<const void*>(&mx4_kernel<BQ, CL, SPLIT>)}
const Form kForms[] = {
    SGEMM_GB300_MX4(16, 1, false, 170, 700),    SGEMM_GB300_MX4(16, 1, true, 170, 700),
    SGEMM_GB300_MX4(32, 1, false, 190, 800),    SGEMM_GB300_MX4(32, 1, true, 190, 800),
    SGEMM_GB300_MX4(64, 1, false, 220, 900),    SGEMM_GB300_MX4(64, 1, true, 220, 900),
    SGEMM_GB300_MX4(128, 1, false, 283, 1000),  SGEMM_GB300_MX4(128, 1, true, 283, 1000),
    SGEMM_GB300_MX4(256, 1, false, 383, 1900),  SGEMM_GB300_MX4(256, 2, false, 300, 2300)};
constexpr int kNumForms = sizeof(kForms) / sizeof(kForms[0]), kMaxDevices = 64;
constexpr int kSplitCost = 1500;           // what cutting a tile costs, ns
std::mutex g_mutex;
bool g_ready[kMaxDevices][kNumForms];
int g_resident[kMaxDevices][9];            // clusters of 2, 4, 8 CTAs resident at once

cudaLaunchConfig_t config(int ctas, int cluster, cudaLaunchAttribute (&la)[2], cudaStream_t stream) {
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  la[1].id = cudaLaunchAttributeClusterDimension;
  la[1].val.clusterDim.x = cluster;
  la[1].val.clusterDim.y = 1;
  la[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)ctas);
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = kSmem;
  lc.stream = stream;
  lc.attrs = la;
  lc.numAttrs = cluster > 1 ? 2 : 1;
  return lc;
}

// Makes the kernels ready on the device; false where that fails.
bool prepare(int dev, int sms) {
  if (dev < 0 || dev >= kMaxDevices) return false;
  std::lock_guard<std::mutex> lock(g_mutex);
  for (int i = 0; i < kNumForms; ++i) {
    if (g_ready[dev][i]) continue;
    const Form& f = kForms[i];
    if (cudaFuncSetAttribute(f.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) {
      cudaGetLastError();
      return false;
    }
    // (SMs form clusters within a GPC, so there can be fewer than sms / size; the
    // kernels' shared memory leaves one CTA an SM, so one kernel stands for all)
    for (int size = 2; size <= 8 && f.cl == 2; size *= 2) {
      cudaLaunchAttribute la[2];
      cudaLaunchConfig_t lc = config(sms / size * size, size, la, nullptr);
      lc.attrs = la + 1;
      lc.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&g_resident[dev][size], f.kernel, &lc) != cudaSuccess) {
        cudaGetLastError();
        g_resident[dev][size] = 0;
      }
    }
    g_ready[dev][i] = true;
  }
  return true;
}

bool encode(CUtensorMap* map, CUtensorMapDataType type, const void* ptr, long long cols,
            long long rows, long long pitch, int box_cols, int box_rows, CUtensorMapSwizzle swizzle) {
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, 1};
  cuuint64_t strides[2] = {(cuuint64_t)pitch, (cuuint64_t)(pitch * rows)};
  cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  auto call = [&] {
    return ragged::tensor_map_encode()(map, type, 3, const_cast<void*>(ptr), dims, strides, box, estr,
                                       CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (call()) return true;
  int dev = 0;   // (a host thread without a context: see ragged::encode_operand)
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && call();
}
// Codes as bytes, boxes of 128 bytes x `box_rows`.
bool encode_codes(CUtensorMap* map, const void* ptr, long long bytes, long long rows, int ld, int box_rows) {
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, ptr, bytes, rows, ld, kRow, box_rows,
                CU_TENSOR_MAP_SWIZZLE_128B);
}
// Scales as 32-bit words, a row of tiles a row, boxes of two tiles x `box_rows`.
bool encode_scales(CUtensorMap* map, const void* ptr, long long rows, long long tiles_k, int box_rows) {
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, ptr, tiles_k * 128, (rows + 127) / 128,
                tiles_k * 512, 256, box_rows, CU_TENSOR_MAP_SWIZZLE_NONE);
}
// The output, boxes of 32 features x 32 tokens.
bool encode_out(CUtensorMap* map, const void* ptr, int type, long long n, long long m, long long pitch) {
  return encode(map,
                type == SGEMM_TYPE_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                : type == SGEMM_TYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                          : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                ptr, n, m, pitch, 32, 32, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// The form and the parts of a tile that take least time by the table: waves of
// whole tiles, or one wave of tiles in parts. A tile narrower than 128 columns
// only where it holds all tokens (the scales of its rows start a tile of 128).
// `width`, `ctas`: a tile that is asked for (0: none).
struct Choice {
  const Form* form;
  int split;
};
Choice choose(int M, int N, int K, int sms, const int* resident, int width, int ctas) {
  Choice best{nullptr, 1};
  double least = 0;
  const int slices = cdiv(K, kSliceK);
  for (const Form& f : kForms) {
    if (f.bq < 128 && M > f.bq) continue;
    if (width > 0 && (f.bq != width || f.cl != ctas)) continue;
    const double tiles = (double)cdiv(N, BP * f.cl) * cdiv(M, f.bq);
    for (int split = f.split ? 2 : 1; split <= (f.split ? 8 : 1); split *= 2) {
      const int size = f.split ? split : f.cl, workers = size == 1 ? sms : resident[size];
      if (workers == 0 || (f.split && (tiles > workers || slices < 2 * split))) continue;
      const double waves = (double)(long long)((tiles + workers - 1) / workers);
      const double ns = waves * (f.tile + (double)cdiv(slices, split) * f.slice) +
                        (f.split ? kSplitCost : 0);
      if (best.form == nullptr || ns < least) {
        least = ns;
        best = Choice{&f, split};
      }
    }
  }
  return best;
}

int run(int M, int N, int K, const void* A, int lda, const void* SA, const void* B, int ldb,
        const void* SB, int out_type, void* C, int ldc, cudaStream_t stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return SGEMM_ERR_LAUNCH;
  }
  int st = library_device_sms(dev, &sms);
  if (st != SGEMM_OK) return st;
  if (ragged::tensor_map_encode() == nullptr) return SGEMM_ERR_LAUNCH;
  if (!prepare(dev, sms)) return SGEMM_ERR_LAUNCH;
  int width = 0, ctas = 0;
  ragged::forced_tile(&width, &ctas);
  Choice c{nullptr, 1};
  if (width > 0) c = choose(M, N, K, sms, g_resident[dev], width, ctas);
  if (c.form == nullptr) c = choose(M, N, K, sms, g_resident[dev], 0, 0);
  if (c.form == nullptr) return SGEMM_ERR_LAUNCH;
  const Form& f = *c.form;
  const int workers = f.cl == 2 ? g_resident[dev][2] : sms;
  const long long tiles = (long long)cdiv(N, BP * f.cl) * cdiv(M, f.bq);
  if (tiles > 0x7fffffffLL / 16) return SGEMM_ERR_INVALID_DIM;
  Params p = {};
  p.P = N;
  p.Q = M;
  p.K = K;
  // Slices of an accumulation, which truncates: 8, of 2048 values, are as exact as sums in
  // FP32 (blocks whose powers differ by up to 2^16, 512 x 2048 x 4096: 5.5e-7, a product
  // in FP32 5.1e-7; 4 slices 2.9e-7; without such differences the sums are exact). For 16
  // bits 32, 1.1e-6 at 8192 values. 8192 x 8192 x 8192, FP32 out: 4 slices 300 us, 8 226,
  // 32 173.
  p.chunk = out_type == SGEMM_TYPE_F32 ? 8 : 32;
  p.out = C;
  p.ldo = ldc;
  p.out_type = out_type;
  float* ws = nullptr;
  const std::unique_lock<std::mutex> lock = library_lock();   // to the launch
  st = library_workspace(dev, stream, 0, 0, &ws, &p.status, nullptr, nullptr, nullptr);
  if (st != SGEMM_OK) return st;
  p.timeout_ns = library_wait_timeout_ns();

  const long long blocks = (K + 31ll) / 32, tiles_k = (blocks + 3) / 4;
  CUtensorMap mp = {}, mq = {}, msp = {}, msq = {}, mo = {};
  if (!encode_codes(&mp, B, blocks * 16, N, ldb, BP) ||
      !encode_codes(&mq, A, blocks * 16, M, lda, f.bq / f.cl) ||
      !encode_scales(&msp, SB, N, tiles_k, 1) || !encode_scales(&msq, SA, M, tiles_k, (f.bq + 127) / 128))
    return SGEMM_ERR_LAUNCH;
  const int elem = out_type == SGEMM_TYPE_F32 ? 4 : 2;
  // (Narrow tiles and cut ones are written by their threads. A TMA store ends with the
  // 16 bytes that the row's last value is in: in rows that end inside those it would
  // write zeros behind them.)
  const bool tma_out = f.bq >= 128 && c.split == 1 && (reinterpret_cast<uintptr_t>(C) & 15u) == 0 &&
                       (long long)ldc * elem % 16 == 0;
  p.tma_out = !tma_out ? 0 : (long long)N * elem % 16 == 0 ? 1 : 2;
  if (p.tma_out && !encode_out(&mo, C, out_type, N, M, (long long)ldc * elem)) return SGEMM_ERR_LAUNCH;
  const int grid = c.split > 1 ? (int)tiles * c.split : (int)std::min<long long>(workers, tiles) * f.cl;
  cudaLaunchAttribute la[2];
  const cudaLaunchConfig_t lc = config(grid, c.split > 1 ? c.split : f.cl, la, stream);
  void* args[] = {&p, &mp, &mq, &msp, &msq, &mo};
  if (cudaLaunchKernelExC(&lc, f.kernel, args) != cudaSuccess) {
    cudaGetLastError();
    return SGEMM_ERR_LAUNCH;
  }
  char text[160];
  snprintf(text, sizeof(text), "mx4_%dx%dx%d cluster=%d grid=%d split=%d", BP * f.cl, f.bq, kSliceK,
           f.cl, grid, c.split);
  note_last_config(text);
  return SGEMM_OK;
}

// K == 0: zeros.
int clear(int M, int N, int out_type, void* C, int ldc, cudaStream_t stream) {
  const size_t e = out_type == SGEMM_TYPE_F32 ? 4 : 2;
  if (cudaMemset2DAsync(C, ldc * e, 0, N * e, M, stream) == cudaSuccess) return SGEMM_OK;
  cudaGetLastError();
  return SGEMM_ERR_LAUNCH;
}

}  // namespace
}  // namespace mx4
}  // namespace sgemm_gb300

using namespace sgemm_gb300;

SGEMM_API int sgemm_mx4(int M, int N, int K, const unsigned char* A, int lda,
                        const unsigned char* scaleA, const unsigned char* B, int ldb,
                        const unsigned char* scaleB, int out_type, void* C, int ldc, void* stream_) {
  if (out_type != SGEMM_TYPE_F32 && out_type != SGEMM_TYPE_BF16 && out_type != SGEMM_TYPE_F16)
    return SGEMM_ERR_INVALID_VALUE;
  if (M < 0 || N < 0 || K < 0) return SGEMM_ERR_INVALID_DIM;
  const long long bytes = (K + 31ll) / 32 * 16;
  if (lda < bytes || ldb < bytes || lda % 16 != 0 || ldb % 16 != 0 || ldc < (N > 1 ? N : 1))
    return SGEMM_ERR_INVALID_LD;
  if (M == 0 || N == 0) return SGEMM_OK;
  if (C == nullptr || (K > 0 && (A == nullptr || B == nullptr || scaleA == nullptr || scaleB == nullptr)))
    return SGEMM_ERR_NULL_PTR;
  const uintptr_t in = reinterpret_cast<uintptr_t>(A) | reinterpret_cast<uintptr_t>(B) |
                       reinterpret_cast<uintptr_t>(scaleA) | reinterpret_cast<uintptr_t>(scaleB);
  if ((K > 0 && (in & 15u)) ||
      (reinterpret_cast<uintptr_t>(C) & (out_type == SGEMM_TYPE_F32 ? 3u : 1u)))
    return SGEMM_ERR_MISALIGNED;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (K == 0) return mx4::clear(M, N, out_type, C, ldc, stream);
  return mx4::run(M, N, K, A, lda, scaleA, B, ldb, scaleB, out_type, C, ldc, stream);
}
