// grouped.cu -- sgemm_grouped and sgemm_grouped_wgrad (products grouped by
// expert with ragged row counts) and sgemm_i8 (8-bit integer product with
// token and channel scales): argument checks, tile width, operand maps and
// the launch of ragged_kernel.
#include <cstdio>

#include "ragged_launch.cuh"

#define SGEMM_API extern "C" __attribute__((visibility("default")))

namespace sgemm_gb300 {
namespace ragged {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encode() {
  static const PFN_cuTensorMapEncodeTiled_v12000 enc = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    cudaGetLastError();
    return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
  }();
  return enc;
}

namespace {

// Rows of `cols` elements from pitch ld (and matrix pitch stride) to one
// after another at pitch ldo.
template <typename E>
__global__ void pack_kernel(const E* __restrict__ src, long long ld, long long stride, int rows,
                            int cols, int batch, E* __restrict__ dst, long long ldo) {
  // may start before the kernel ahead on the stream has finished
  ptx::griddep_wait();
  const long long total = (long long)rows * batch;
  for (long long r = blockIdx.x; r < total; r += gridDim.x) {
    const E* s = src + (r / rows) * stride + (r % rows) * ld;
    E* d = dst + r * ldo;
    for (int c = threadIdx.x; c < cols; c += blockDim.x) d[c] = s[c];
  }
}

template <typename E>
cudaError_t pack(const Operand& op, void* dst, int sms, cudaStream_t stream) {
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  const long long rows = op.rows * op.batch;
  lc.gridDim = dim3((unsigned)(rows < sms * 8 ? rows : sms * 8));
  lc.blockDim = dim3(256);
  lc.stream = stream;
  lc.attrs = la;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, pack_kernel<E>, static_cast<const E*>(op.ptr), op.ld, op.stride,
                            (int)op.rows, (int)op.cols, op.batch, static_cast<E*>(dst),
                            op.packed_ld());
}

}  // namespace

cudaError_t pack_operand(Operand* op, void* dst, int sms, cudaStream_t stream) {
  const cudaError_t e = op->elem == 1   ? pack<uint8_t>(*op, dst, sms, stream)
                        : op->elem == 2 ? pack<uint16_t>(*op, dst, sms, stream)
                                        : pack<uint32_t>(*op, dst, sms, stream);
  op->ptr = dst;
  op->ld = op->packed_ld();
  op->stride = op->rows * op->ld;
  return e;
}

bool encode_operand(CUtensorMap* map, const Operand& op, CUtensorMapDataType type, int row_bytes,
                    int box_rows) {
  const long long pitch = op.ld * op.elem;
  const long long mat = op.batch > 1 ? op.stride * op.elem : pitch * op.rows;
  cuuint64_t dims[3] = {(cuuint64_t)op.cols, (cuuint64_t)op.rows, (cuuint64_t)op.batch};
  cuuint64_t strides[2] = {(cuuint64_t)pitch, (cuuint64_t)mat};
  cuuint32_t box[3] = {(cuuint32_t)(row_bytes / op.elem), (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return tensor_map_encode()(map, type, 3, const_cast<void*>(op.ptr), dims, strides, box, estr,
                             CU_TENSOR_MAP_INTERLEAVE_NONE,
                             row_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                              : CU_TENSOR_MAP_SWIZZLE_64B,
                             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

int elem_bytes(int type) { return type == SGEMM_TYPE_F32 ? 4 : 2; }
bool type_ok(int type) {
  return type == SGEMM_TYPE_F32 || type == SGEMM_TYPE_BF16 || type == SGEMM_TYPE_F16;
}
bool misaligned(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) != 0;
}

// Tile width in q. rows: wide enough that a typical group's rows fit one
// tile, at most 256 (128 for converted operands).
int rows_width(long long rows_per_group, int widest) {
  int bq = 32;
  while (bq < widest && bq < rows_per_group) bq *= 2;
  return bq;
}

// src: a Src; the operands as stored. Fills the maps (packing what TMA cannot
// read), the workspace fields of `p`, and launches.
int run(int src, int type, Params p, Operand op_p, Operand op_q, int bq, cudaStream_t stream,
        const char* what) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return SGEMM_ERR_LAUNCH;
  }
  int st = library_device_sms(dev, &sms);
  if (st != SGEMM_OK) return st;
  if (tensor_map_encode() == nullptr) return SGEMM_ERR_LAUNCH;

  // the most tiles the offsets can give
  const long long ptiles = cdiv(p.P, BP);
  const long long qtiles = p.wgrad ? (long long)p.E * cdiv(p.Q, bq)
                                   : (long long)p.T / bq + (p.T < p.E ? p.T : p.E);
  if (ptiles * qtiles > 0x7fffffffLL) return SGEMM_ERR_INVALID_DIM;
  const bool reads = p.K > 0;
  const int slice = src == kF32 ? 32 : 64;
  // tiles are cut along k only when there may be fewer of them than CTAs
  const long long least = p.wgrad ? ptiles * qtiles : ptiles * (p.T / bq > 0 ? p.T / bq : 1);
  const bool may_split = reads && 2 * least <= sms;
  const size_t pack_p = reads ? op_p.packed_bytes() : 0, pack_q = reads ? op_q.packed_bytes() : 0;
  const size_t partial = may_split ? (size_t)sms * BP * bq * 4 : 0;
  float* ws = nullptr;
  uint32_t epoch = 0;
  st = library_workspace(dev, stream, (pack_p + pack_q + partial) / 4, (size_t)sms, &ws, &p.status,
                         &p.counters, &epoch);
  if (st != SGEMM_OK) return st;
  char* at = reinterpret_cast<char*>(ws);
  if (pack_p && pack_operand(&op_p, at, sms, stream) != cudaSuccess) {
    cudaGetLastError();
    return SGEMM_ERR_LAUNCH;
  }
  if (pack_q && pack_operand(&op_q, at + pack_p, sms, stream) != cudaSuccess) {
    cudaGetLastError();
    return SGEMM_ERR_LAUNCH;
  }
  p.partials = may_split ? reinterpret_cast<float*>(at + pack_p + pack_q) : nullptr;
  p.timeout_ns = library_wait_timeout_ns();

  CUtensorMap mp = {}, mq = {};
  if (reads) {
    const CUtensorMapDataType dt =
        src == kI8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                   : (type == SGEMM_TYPE_F32
                          ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                          : (type == SGEMM_TYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                     : CU_TENSOR_MAP_DATA_TYPE_FLOAT16));
    const int row_bytes = src == kI8 ? 64 : 128;
    if (!encode_operand(&mp, op_p, dt, row_bytes, p.p_mn ? slice : BP) ||
        !encode_operand(&mq, op_q, dt, row_bytes, p.q_mn ? slice : bq))
      return SGEMM_ERR_LAUNCH;
  }
  const cudaError_t e = src == k16    ? launch_k16(dev, bq, sms, p, mp, mq, stream)
                        : src == kF32 ? launch_f32(dev, bq, sms, p, mp, mq, stream)
                                      : launch_i8(dev, bq, sms, p, mp, mq, stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return SGEMM_ERR_LAUNCH;
  }
  char text[160];
  snprintf(text, sizeof(text), "%s_%s_128x%dx%d grid=%d chunk=%d%s%s", what,
           src == k16 ? (type == SGEMM_TYPE_BF16 ? "bf16" : "f16") : (src == kF32 ? "f32" : "i8"),
           bq, slice, sms, p.chunk, pack_p ? " p=copied" : "", pack_q ? " q=copied" : "");
  note_last_config(text);
  return SGEMM_OK;
}

// k-slices per tensor-memory accumulation. 32-bit results leave it every 256
// values of k (64 for kF32: 24 instructions), 16-bit results once: the error of
// a truncating sum of 4096 values is far below their rounding.
int accumulation_chunk(int src, int out_type) {
  if (src == kF32) return 2;
  if (src == kI8) return Geo<kI8, 32>::kExactChunk;
  return out_type == kOutF32 ? 4 : 0x40000000;
}

}  // namespace
}  // namespace ragged
}  // namespace sgemm_gb300

using namespace sgemm_gb300;
using ragged::Operand;

SGEMM_API int sgemm_grouped(int op, int type, int out_type, int E, int T, int N, int K, float alpha,
                            const void* X, int ldx, const void* W, int ldw, long long strideW,
                            const int* offsets, float beta, void* Y, int ldy, void* stream) {
  if ((op != SGEMM_OP_N && op != SGEMM_OP_T) || !ragged::type_ok(type) ||
      !ragged::type_ok(out_type))
    return SGEMM_ERR_INVALID_VALUE;
  if (type == SGEMM_TYPE_F32 && out_type != SGEMM_TYPE_F32) return SGEMM_ERR_INVALID_VALUE;
  if (E < 0 || T < 0 || N < 0 || K < 0) return SGEMM_ERR_INVALID_DIM;
  if (E > ragged::kMaxGroups || strideW < 0) return SGEMM_ERR_INVALID_VALUE;
  const int ldw_min = op == SGEMM_OP_N ? N : K;
  if (ldx < (K > 1 ? K : 1) || ldw < (ldw_min > 1 ? ldw_min : 1) || ldy < (N > 1 ? N : 1))
    return SGEMM_ERR_INVALID_LD;
  if (E == 0 || T == 0 || N == 0) return SGEMM_OK;
  const bool reads = K > 0 && alpha != 0.f;
  if (Y == nullptr || offsets == nullptr || (reads && (X == nullptr || W == nullptr)))
    return SGEMM_ERR_NULL_PTR;
  const int eb = ragged::elem_bytes(type);
  if (ragged::misaligned(Y, ragged::elem_bytes(out_type)) || ragged::misaligned(offsets, 4) ||
      (reads && (ragged::misaligned(X, eb) || ragged::misaligned(W, eb))))
    return SGEMM_ERR_MISALIGNED;

  const int src = type == SGEMM_TYPE_F32 ? ragged::kF32 : ragged::k16;
  ragged::Params p = {};
  p.E = E;
  p.T = T;
  p.P = N;
  p.K = reads ? K : 0;
  p.p_mn = op == SGEMM_OP_N;
  p.bf16 = type == SGEMM_TYPE_BF16;
  p.offsets = offsets;
  p.out = Y;
  p.ldo = ldy;
  p.out_type = out_type;
  p.alpha = alpha;
  p.beta = beta;
  p.chunk = ragged::accumulation_chunk(src, out_type);
  const Operand w{W, eb, op == SGEMM_OP_N ? K : N, op == SGEMM_OP_N ? N : K, ldw, strideW, E};
  const Operand x{X, eb, T, K, ldx, 0, 1};
  const int bq = ragged::rows_width(((long long)T + E - 1) / E, src == ragged::k16 ? 256 : 128);
  return ragged::run(src, type, p, w, x, bq, static_cast<cudaStream_t>(stream), "grouped");
}

SGEMM_API int sgemm_grouped_wgrad(int type, int out_type, int E, int T, int M, int N, float alpha,
                                  const void* A, int lda, const void* B, int ldb,
                                  const int* offsets, float beta, void* C, int ldc,
                                  long long strideC, void* stream) {
  if (!ragged::type_ok(type) || !ragged::type_ok(out_type)) return SGEMM_ERR_INVALID_VALUE;
  if (type == SGEMM_TYPE_F32 && out_type != SGEMM_TYPE_F32) return SGEMM_ERR_INVALID_VALUE;
  if (E < 0 || T < 0 || M < 0 || N < 0) return SGEMM_ERR_INVALID_DIM;
  if (E > ragged::kMaxGroups || strideC < 0) return SGEMM_ERR_INVALID_VALUE;
  if (lda < (M > 1 ? M : 1) || ldb < (N > 1 ? N : 1) || ldc < (N > 1 ? N : 1))
    return SGEMM_ERR_INVALID_LD;
  if (E == 0 || M == 0 || N == 0) return SGEMM_OK;
  const bool reads = T > 0 && alpha != 0.f;
  if (C == nullptr || offsets == nullptr || (reads && (A == nullptr || B == nullptr)))
    return SGEMM_ERR_NULL_PTR;
  const int eb = ragged::elem_bytes(type);
  if (ragged::misaligned(C, ragged::elem_bytes(out_type)) || ragged::misaligned(offsets, 4) ||
      (reads && (ragged::misaligned(A, eb) || ragged::misaligned(B, eb))))
    return SGEMM_ERR_MISALIGNED;

  const int src = type == SGEMM_TYPE_F32 ? ragged::kF32 : ragged::k16;
  ragged::Params p = {};
  p.wgrad = 1;
  p.E = E;
  p.T = T;
  p.P = N;
  p.Q = M;
  p.K = reads ? T : 0;
  p.p_mn = p.q_mn = 1;
  p.bf16 = type == SGEMM_TYPE_BF16;
  p.offsets = offsets;
  p.out = C;
  p.ldo = ldc;
  p.stride_o = strideC;
  p.out_type = out_type;
  p.alpha = alpha;
  p.beta = beta;
  p.chunk = ragged::accumulation_chunk(src, out_type);
  const Operand pb{B, eb, T, N, ldb, 0, 1}, qa{A, eb, T, M, lda, 0, 1};
  int bq = src == ragged::k16 ? 256 : 128;
  while (bq > 64 && bq / 2 >= M) bq /= 2;
  return ragged::run(src, type, p, pb, qa, bq, static_cast<cudaStream_t>(stream), "wgrad");
}

SGEMM_API int sgemm_i8(int M, int N, int K, const signed char* A, int lda, const float* scaleA,
                       const signed char* B, int ldb, const float* scaleB, int out_type, void* C,
                       int ldc, void* stream) {
  if (!ragged::type_ok(out_type)) return SGEMM_ERR_INVALID_VALUE;
  if (M < 0 || N < 0 || K < 0) return SGEMM_ERR_INVALID_DIM;
  if (K > SGEMM_I8_MAX_K) return SGEMM_ERR_INVALID_DIM;
  if (lda < (K > 1 ? K : 1) || ldb < (K > 1 ? K : 1) || ldc < (N > 1 ? N : 1))
    return SGEMM_ERR_INVALID_LD;
  if (M == 0 || N == 0) return SGEMM_OK;
  if (C == nullptr || scaleA == nullptr || scaleB == nullptr ||
      (K > 0 && (A == nullptr || B == nullptr)))
    return SGEMM_ERR_NULL_PTR;
  if (ragged::misaligned(C, ragged::elem_bytes(out_type)) || ragged::misaligned(scaleA, 4) ||
      ragged::misaligned(scaleB, 4))
    return SGEMM_ERR_MISALIGNED;

  ragged::Params p = {};
  p.E = 1;
  p.T = M;
  p.P = N;
  p.K = K;
  p.out = C;
  p.ldo = ldc;
  p.out_type = out_type;
  p.alpha = 1.f;
  p.scale_p = scaleB;
  p.scale_q = scaleA;
  p.chunk = ragged::accumulation_chunk(ragged::kI8, out_type);
  const Operand w{B, 1, N, K, ldb, 0, 1}, x{A, 1, M, K, lda, 0, 1};
  return ragged::run(ragged::kI8, 0, p, w, x, ragged::rows_width(M, 128),
                     static_cast<cudaStream_t>(stream), "i8");
}
