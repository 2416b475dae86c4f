// grouped.cu -- sgemm_grouped and sgemm_grouped_wgrad (products grouped by
// expert with ragged row counts) and sgemm_i8 (8-bit integer product with
// token and channel scales): argument checks, tile width, operand maps and
// the launch of ragged_kernel.
#include <atomic>
#include <cmath>
#include <cstdio>
#include <mutex>

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

// One operand to copy: rows of `bytes` bytes at pitch ld (matrices at `stride`)
// from any address, to rows one after another at pitch ldo, a multiple of 16
// bytes. `lanes` threads copy a segment of a row at a time, each some 16-byte
// pieces of it.
struct Pack {
  const unsigned char* src;
  unsigned char* dst;
  long long ld, stride, ldo, total;   // total: segments of all rows
  const unsigned char* end;           // of the last row
  long long bytes;                    // of a row: beyond 32 bits from 2^29 FP32 values on
  int rows, segments;                 // segments: of a row
  int lanes;                          // 4 .. 32: as many as a short row needs
};
constexpr int kPackThreads = 256;
// Pieces of a thread, all loaded before the first is stored. Copies: 4 (25 MB in
// rows of 1554 bytes with their product 23.6 us, 24.6 with 2; the copy is some
// 9 us of it, 5.6 TB/s read and written). Widened ones write twice what they read
// and are best at 1 (2000 and 4096 rows of 1001 bytes with their product 35.3 us;
// 2: 36.0, 4: 37.6).
__host__ __device__ constexpr int pack_pieces(bool widen) { return widen ? 1 : 4; }

// Bytes a .. a + 15 of the 32 bytes x, y (W = a / 4).
template <int W>
__device__ __forceinline__ uint4 window(const uint4& x, const uint4& y, unsigned a) {
  const uint32_t in[9] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w, 0u};
  const unsigned sh = (a & 3u) * 8u;
  return make_uint4(
      __funnelshift_r(in[W], in[W + 1], sh), __funnelshift_r(in[W + 1], in[W + 2], sh),
      __funnelshift_r(in[W + 2], in[W + 3], sh), __funnelshift_r(in[W + 3], in[W + 4], sh));
}

// Copies a and then b (either may have no segments), WIDEN: 8-bit integers as
// F16 (two 16-byte words a piece). What lies between a row's end and the end of
// its last piece is set to zero, the rest of its pitch is not set. A piece at
// an odd address comes from the two aligned words it lies in, one shift for all
// of a segment.
template <bool WIDEN>
__global__ void __launch_bounds__(kPackThreads)
    pack_kernel(const __grid_constant__ Pack a, const __grid_constant__ Pack b) {
  // may start before the kernel ahead on the stream has finished
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  constexpr int kPieces = pack_pieces(WIDEN);
  // the threads of a first, then those of b
  const long long threads = gridDim.x * (long long)kPackThreads;
  const long long of_a = a.total * a.lanes, all = of_a + b.total * b.lanes;
  for (long long i = blockIdx.x * (long long)kPackThreads + threadIdx.x; i < all; i += threads) {
    const bool first = i < of_a;
    const Pack& p = first ? a : b;
    const int shift = __ffs(p.lanes) - 1;
    const long long unit = (first ? i : i - of_a) >> shift;
    const int lane = (int)(first ? i : i - of_a) & (p.lanes - 1);
    const int step = 16 * p.lanes;             // bytes between a thread's pieces
    long long r, mat;
    int seg;
    if (unit < 0x7fffffff) {                  // (a 64-bit division takes far longer)
      r = (int)unit / p.segments;
      seg = (int)unit - (int)r * p.segments;
      mat = p.stride == 0 ? 0 : (int)r / p.rows;
    } else {
      r = unit / p.segments;
      seg = (int)(unit - r * p.segments);
      mat = p.stride == 0 ? 0 : r / p.rows;
    }
    // the thread's first piece: byte of the row
    const long long c0 = (long long)seg * (kPieces * step) + lane * 16;
    const unsigned char* s = p.src + mat * p.stride + (r - mat * p.rows) * p.ld + c0;
    const unsigned at = (unsigned)reinterpret_cast<uintptr_t>(s) & 15u;   // (a segment's lanes agree)
    const unsigned char* base = s - at;
    uint4 x[kPieces], y[kPieces];
    bool inside[kPieces];                     // both words lie in the operand
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const unsigned char* w = base + step * j;
      inside[j] = c0 + step * j < p.bytes && w >= p.src && w + (at ? 32 : 16) <= p.end;
      if (inside[j]) {
        x[j] = __ldg(reinterpret_cast<const uint4*>(w));
        if (at) y[j] = __ldg(reinterpret_cast<const uint4*>(w) + 1);
      }
    }
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const long long c = c0 + step * j;
      if (c >= p.bytes) break;
      uint32_t w[4];
      if (inside[j]) {
        uint4 v = x[j];
        switch (at >> 2) {
          case 0: if (at) v = window<0>(x[j], y[j], at); break;
          case 1: v = window<1>(x[j], y[j], at); break;
          case 2: v = window<2>(x[j], y[j], at); break;
          default: v = window<3>(x[j], y[j], at); break;
        }
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        if (c + 16 > p.bytes) {               // the row's end
          const int left = (int)(p.bytes - c);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int n = left - 4 * k;       // valid bytes from this word on
            w[k] &= n >= 4 ? 0xffffffffu : (n <= 0 ? 0u : (1u << (8 * n)) - 1u);
          }
        }
      } else {                                // at the operand's ends: byte by byte
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = 0u;
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (c + k < p.bytes) w[k >> 2] |= (uint32_t)s[step * j + k] << (8 * (k & 3));
      }
      if (WIDEN) {
        const uint2 e = i8_to_f16(w[0]), f = i8_to_f16(w[1]), g = i8_to_f16(w[2]),
                    h = i8_to_f16(w[3]);
        uint4* o = reinterpret_cast<uint4*>(p.dst + r * p.ldo + 2 * c);
        o[0] = make_uint4(e.x, e.y, f.x, f.y);
        // (a row's pitch is a multiple of 8 F16 values, not always of 16)
        if (2 * c + 16 < p.ldo) o[1] = make_uint4(g.x, g.y, h.x, h.y);
      } else {
        *reinterpret_cast<uint4*>(p.dst + r * p.ldo + c) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

}  // namespace

cudaError_t pack_operands(Operand* a, void* dst_a, Operand* b, void* dst_b, bool widen, int sms,
                          cudaStream_t stream) {
  Pack p[2] = {};
  Operand* ops[2] = {a, b};
  void* dsts[2] = {dst_a, dst_b};
  long long total = 0;
  for (int i = 0; i < 2; ++i) {
    if (dsts[i] == nullptr) continue;
    Operand& op = *ops[i];
    const long long bytes = op.cols * op.elem;
    p[i].src = static_cast<const unsigned char*>(op.ptr);
    p[i].dst = static_cast<unsigned char*>(dsts[i]);
    p[i].ld = op.ld * op.elem;
    p[i].stride = op.batch > 1 ? op.stride * op.elem : 0;
    p[i].ldo = op.packed_pitch(widen);
    p[i].lanes = 4;
    const int per_lane = 16 * pack_pieces(widen);
    while (p[i].lanes < 32 && p[i].lanes * per_lane < bytes) p[i].lanes *= 2;
    const int segment = p[i].lanes * per_lane;
    p[i].segments = (int)((bytes + segment - 1) / segment);
    p[i].total = op.rows * op.batch * p[i].segments;
    p[i].end = p[i].src + (op.batch - 1) * p[i].stride + (op.rows - 1) * p[i].ld + bytes;
    p[i].rows = (int)op.rows;
    p[i].bytes = bytes;
    total += p[i].total * p[i].lanes;
    if (widen) op.elem = 2;
    op.ptr = dsts[i];
    op.ld = p[i].ldo / op.elem;
    op.stride = op.rows * op.ld;
  }
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  const long long blocks = (total + kPackThreads - 1) / kPackThreads;
  lc.gridDim = dim3((unsigned)(blocks < sms * 32ll ? blocks : sms * 32ll));
  lc.blockDim = dim3(kPackThreads);
  lc.stream = stream;
  lc.attrs = la;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, widen ? pack_kernel<true> : pack_kernel<false>, p[0], p[1]);
}

bool encode_operand(CUtensorMap* map, const Operand& op, CUtensorMapDataType type, int row_bytes,
                    int box_rows) {
  const long long pitch = op.ld * op.elem;
  const long long mat = op.batch > 1 ? op.stride * op.elem : pitch * op.rows;
  cuuint64_t dims[3] = {(cuuint64_t)op.cols, (cuuint64_t)op.rows, (cuuint64_t)op.batch};
  cuuint64_t strides[2] = {(cuuint64_t)pitch, (cuuint64_t)mat};
  cuuint32_t box[3] = {(cuuint32_t)(row_bytes / op.elem), (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  auto encode = [&] {
    return tensor_map_encode()(map, type, 3, const_cast<void*>(op.ptr), dims, strides, box, estr,
                               CU_TENSOR_MAP_INTERLEAVE_NONE,
                               row_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                                : CU_TENSOR_MAP_SWIZZLE_64B,
                               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (encode()) return true;
  // a host thread whose first CUDA work this is (autograd's, for one) has no
  // context yet, which the encoder needs: selecting the device gives it one
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && encode();
}

namespace {

int elem_bytes(int type) { return type == SGEMM_TYPE_F32 ? 4 : 2; }
bool type_ok(int type) {
  return type == SGEMM_TYPE_F32 || type == SGEMM_TYPE_BF16 || type == SGEMM_TYPE_F16;
}
bool misaligned(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) != 0;
}

// The built kernels, and per device what prepare() said of each.
constexpr int kMaxDevices = 64, kMaxForms = 24;
struct Built {
  bool ready;
  int workers;
};
std::mutex g_mutex;
Built g_built[kMaxDevices][kMaxForms];
// Tile width and CTAs per worker for later calls (tests, measurements); 0: by rule.
std::atomic<int> g_width{0}, g_ctas{0};

const FormEntry* form_entry(int i) {
  if (i < kNumForms16) return &kForms16[i];
  i -= kNumForms16;
  if (i < kNumFormsF32) return &kFormsF32[i];
  i -= kNumFormsF32;
  return i < kNumFormsI8 ? &kFormsI8[i] : nullptr;
}

// The entry of a form and its resident workers on `dev` (null: not built or,
// for pairs, not runnable).
const FormEntry* find_form(int dev, int sms, int src, int bq, int cl, int* workers) {
  if (dev < 0 || dev >= kMaxDevices) return nullptr;
  for (int i = 0; const FormEntry* f = form_entry(i); ++i) {
    if (f->form.src != src || f->form.bq != bq || f->form.cl != cl) continue;
    std::lock_guard<std::mutex> lock(g_mutex);
    Built& b = g_built[dev][i];
    if (!b.ready) {
      if (f->prepare(sms, &b.workers) != cudaSuccess) {
        cudaGetLastError();
        return nullptr;
      }
      b.ready = true;
    }
    *workers = b.workers;
    return b.workers > 0 ? f : nullptr;
  }
  return nullptr;
}

// What a tile of each width costs on a worker, in ns: a slice of 64 values of k
// (measured on GB300: 8192 x 4096 x 4096 over 8 groups for 16-bit operands, 8192
// x 2048 x 4096 for FP32, one wave of tiles for integers) and its epilogue.
struct TileCost {
  int src, bq, cl, slice, epilogue;
};
constexpr TileCost kTileCosts[] = {
    {k16, 16, 1, 181, 600},    {k16, 32, 1, 184, 700},   {k16, 64, 1, 280, 1100},
    {k16, 128, 1, 282, 1300},  {k16, 256, 1, 403, 2000}, {k16, 256, 2, 364, 2500},
    {kF32, 16, 1, 800, 600},   {kF32, 32, 1, 810, 700},  {kF32, 64, 1, 1080, 1100},
    {kF32, 128, 1, 1300, 1300},
    {kI8, 16, 1, 270, 600},    {kI8, 32, 1, 275, 700},   {kI8, 64, 1, 425, 1100},
    {kI8, 128, 1, 460, 1300},
    {kI8Wide, 256, 2, 364, 2500},
};
// The costs of a form: those of its own number of CTAs (integers that have been
// widened cost what F16 operands do).
TileCost tile_cost(int src, int bq, int cl) {
  const int as = src == kI8Wide ? k16 : src;
  for (const TileCost& c : kTileCosts)
    if (c.src == as && c.bq == bq && c.cl == cl) return c;
  return kTileCosts[0];   // (every built form has its entry)
}
// What cutting a tile along k costs, ns: publishing a part and the rendezvous,
// and reading one part back (a load of L2 for every 32 columns of a warp; four
// narrow parts go in one).
int cut_once(int bq) { return 1500 + 6 * bq; }
int cut_part(int bq) { return bq <= 32 ? 12 * bq : 100 + 12 * bq; }
// Slices (of `slice` ns) that a part of a tile of `sum` slices has at least: with
// p parts the sum takes sum / p slices and adding them p * cut_part, least at
// parts of this length.
int cut_least(double sum, int slice, int bq) {
  const int n = (int)std::sqrt(sum * cut_part(bq) / slice);
  return n < 3 ? 3 : n;
}

// The tile of a call: the one whose list takes least time on the workers it
// has, by the costs above. The host does not know the groups' sizes: they are
// taken to be equal but for half a tile of raggedness each. *ns: that time.
Form choose_tile(int src, const Params& p, int sms, double* ns) {
  Form best{src, 0, 1};
  double least = 0;
  for (const TileCost& c : kTileCosts) {
    if (c.src != src || (p.wgrad && c.bq < 64)) continue;
    const int workers = sms / c.cl;
    const double groups = p.E < p.T ? p.E : (p.T > 0 ? p.T : 1);
    const double q = p.wgrad ? (double)p.E * cdiv(p.Q, c.bq)
                             : (p.E == 1 ? (double)cdiv(p.T, c.bq)
                                         : (double)p.T / c.bq + groups / 2 > groups
                                               ? (double)p.T / c.bq + groups / 2
                                               : groups);
    const double tiles = q * cdiv(p.P, BP * c.cl);
    const double k = p.wgrad ? (double)p.T / p.E : p.K, slices = k / 64 < 1 ? 1 : k / 64;
    const double sum = slices * c.slice, tile = sum > c.epilogue ? sum : c.epilogue;
    const double whole = (double)(long long)((tiles + workers - 1) / workers) * tile;
    double parts = 2, cutters = workers;
    if (tiles < workers) {
      const double most = tiles * slices / cut_least(slices, c.slice, c.bq);
      cutters = most < tiles ? tiles : (most < workers ? most : workers);
      parts = cutters / tiles + 1;
    }
    const double cut = tiles / cutters * tile + cut_once(c.bq) + parts * cut_part(c.bq);
    const double time = (cut < whole ? cut : whole) + c.epilogue;
    if (best.bq == 0 || time < least) {
      least = time;
      best = Form{src, c.bq, c.cl};
    }
  }
  *ns = least;
  return best;
}

// Whether an 8-bit product widens its operands to F16 first, for the widest
// tiles, or converts them tile by tile: by the times above, the widening at 4 us
// and 0.65 ns for 1000 values, the copies that the other form may need at 3 us
// and 0.3. Measured on both sides, us (tile by tile / widened): 512 x 4096 x 4096
// 32 / 49, 768 47 / 39, 2048 102 / 63; 2048 x 1024 x 4096 32 / 44; 256 x 8191 x 1000
// (copied) 17 / 21, 384 24 / 22; 512 x 14336 x 4096 86 / 94, 768 131 / 107; 2048 x
// 512 x 512 9 / 15. Of 54 such sizes it takes the faster side of all.
bool widen_first(const Params& p, int sms, double tiles_ns, double copied, double values) {
  double ns = 0;
  choose_tile(kI8Wide, p, sms, &ns);
  if (copied > 0) tiles_ns += 3000 + 0.3e-3 * copied;
  return ns + 4000 + 0.65e-3 * values < tiles_ns;
}

// The operands as stored. Fills the maps (copying what TMA cannot read), the
// workspace fields of `p`, and launches.
int run(int src, int type, Params p, Operand op_p, Operand op_q, cudaStream_t stream,
        const char* what) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return SGEMM_ERR_LAUNCH;
  }
  int st = library_device_sms(dev, &sms);
  if (st != SGEMM_OK) return st;
  if (tensor_map_encode() == nullptr) return SGEMM_ERR_LAUNCH;

  const int width = g_width.load(), ctas = g_ctas.load();
  double ns = 0;
  Form t = choose_tile(src, p, sms, &ns);
  if (src == kI8) {
    const double vp = (double)op_p.rows * op_p.cols, vq = (double)op_q.rows * op_q.cols;
    const double copied = (op_p.direct() ? 0 : vp) + (op_q.direct() ? 0 : vq);
    // (256 columns are built for widened operands only)
    if (width > 0 ? width == 256 : widen_first(p, sms, ns, copied, vp + vq)) {
      src = kI8Wide;
      t = choose_tile(src, p, sms, &ns);
    }
  }
  int workers = 0;
  const FormEntry* form = nullptr;
  if (width > 0 && (!p.wgrad || width >= 64)) form = find_form(dev, sms, src, width, ctas, &workers);
  if (form == nullptr) form = find_form(dev, sms, t.src, t.bq, t.cl, &workers);
  if (form == nullptr && t.cl == 2) form = find_form(dev, sms, t.src, t.bq, 1, &workers);
  if (form == nullptr) return SGEMM_ERR_LAUNCH;
  const int bq = form->form.bq, cl = form->form.cl;

  // tiles and k-slices are numbered with 32-bit integers
  const int sub_k = src == kF32 ? 32 : 64, slice = bq <= 32 ? 2 * sub_k : sub_k;
  const long long tiles = (long long)cdiv(p.P, BP * cl) *
                          (p.wgrad ? (long long)p.E * cdiv(p.Q, bq)
                                   : (long long)p.T / bq + (p.T < p.E ? p.T : p.E));
  const long long slices =
      p.wgrad ? (long long)cdiv(p.P, BP * cl) * cdiv(p.Q, bq) * ((long long)p.T / slice + 2 * p.E)
              : tiles * (cdiv(p.K, slice) + 1);
  if (tiles > 0x7fffffffLL || slices > 0x7fffffffLL) return SGEMM_ERR_INVALID_DIM;

  const bool reads = p.K > 0;
  const bool widen = src == kI8Wide;
  const size_t pack_p = reads ? op_p.packed_bytes(widen) : 0;
  const size_t pack_q = reads ? op_q.packed_bytes(widen) : 0;
  const size_t partial = (size_t)workers * cl * 2 * BP * bq * 4;
  float* ws = nullptr;
  const std::unique_lock<std::mutex> lock = library_lock();   // to the last launch
  st = library_workspace(dev, stream, (pack_p + pack_q + partial) / 4, (size_t)workers * cl, &ws,
                         &p.status, nullptr, nullptr, &p.counters);
  if (st != SGEMM_OK) return st;
  char* at = reinterpret_cast<char*>(ws);
  if ((pack_p || pack_q) &&
      pack_operands(&op_p, pack_p ? at : nullptr, &op_q, pack_q ? at + pack_p : nullptr, widen, sms,
                    stream) != cudaSuccess) {
    cudaGetLastError();
    return SGEMM_ERR_LAUNCH;
  }
  p.partials = reinterpret_cast<float*>(at + pack_p + pack_q);
  {
    const double ns = (double)tile_cost(src, bq, cl).slice * slice / 64;
    const double sum = (double)(p.wgrad ? p.T / p.E : p.K) / slice;
    p.cut_least = cut_least(sum < 1 ? 1 : sum, (int)ns, bq);
    p.cut_once = (int)(16 * cut_once(bq) / ns) + 1;
    p.cut_part = (int)(16 * cut_part(bq) / ns) + 1;
  }
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
    if (!encode_operand(&mp, op_p, dt, row_bytes, p.p_mn ? sub_k : BP) ||
        !encode_operand(&mq, op_q, dt, row_bytes, p.q_mn ? sub_k : bq / cl))
      return SGEMM_ERR_LAUNCH;
  }
  if (form->launch(workers, p, mp, mq, stream) != cudaSuccess) {
    cudaGetLastError();
    return SGEMM_ERR_LAUNCH;
  }
  char text[160];
  snprintf(text, sizeof(text), "%s_%s_%dx%dx%d cluster=%d grid=%d%s%s", what,
           src == k16 ? (type == SGEMM_TYPE_BF16 ? "bf16" : "f16") : (src == kF32 ? "f32" : "i8"),
           BP * cl, bq, slice, cl, workers * cl, pack_p ? " p=copied" : "", pack_q ? " q=copied" : "");
  note_last_config(text);
  return SGEMM_OK;
}

// Values of k per tensor-memory accumulation. Each instruction truncates its
// sum: with n of them in one accumulation a 32-bit result is off by 1.4e-8 n
// (2-norm, relative). Measured: 16 (256 values) 2.3e-7 for 16-bit operands, where
// a sum in FP32 is off by 3.3e-7; the gradient of 8 groups of 1024 x (4096 + 1024)
// in 80 us (24: 3.3e-7 and 72 us, 32: 4.5e-7 and 68 us). For kF32, six a step, 36
// (96 values) 6e-7 (a sum in FP32 of 2048 products: 8e-7). 16-bit results take 64
// (1024 values): 1.1e-6, or 5e-6 where all products have one sign, 2 % of F16's own
// half unit whatever the length. In one accumulation that share grew with it
// (131072 rows: 1.5e-5, and 8e-5 of one sign); 8192 x 4096 x 4096 over 8 groups took
// 192 us so, 197 now.
int accumulation_chunk(int src, int out_type) {
  if (src == kF32) return 96;
  if (src == kI8 || src == kI8Wide) return kExactK;
  return out_type == kOutF32 ? 256 : 1024;
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
  p.p_shared = E > 1 && strideW == 0;   // one matrix for every group
  const Operand w{W, eb, op == SGEMM_OP_N ? K : N, op == SGEMM_OP_N ? N : K, ldw, strideW,
                  p.p_shared ? 1 : E};
  const Operand x{X, eb, T, K, ldx, 0, 1};
  return ragged::run(src, type, p, w, x, static_cast<cudaStream_t>(stream), "grouped");
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
  return ragged::run(src, type, p, pb, qa, static_cast<cudaStream_t>(stream), "wgrad");
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
  return ragged::run(ragged::kI8, SGEMM_TYPE_F16, p, w, x, static_cast<cudaStream_t>(stream), "i8");
}

SGEMM_API int sgemm_grouped_set_tile(int width, int ctas) {
  if (width != 0) {
    bool built = false;
    for (int i = 0; const ragged::FormEntry* f = ragged::form_entry(i); ++i)
      built = built || (f->form.bq == width && f->form.cl == ctas);
    if (!built) return SGEMM_ERR_INVALID_VALUE;
  }
  ragged::g_width.store(width);
  ragged::g_ctas.store(ctas);
  return SGEMM_OK;
}
