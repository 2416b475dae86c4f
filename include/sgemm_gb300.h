/*
 * sgemm_gb300.h -- C ABI of the GB300 (sm_103a) single-precision GEMM library.
 *
 * The operation is the one every kernel on the pages computes:
 *   C = alpha * A * B + beta * C
 * on row-major FP32 matrices ("Shared Memory Tiling", kernel listing, final
 * store alpha * acc + beta * C; "Warp Tiling: A Third Level of Tiling",
 * section "The Kernel", epilogue; "Vectorized Memory Access: 128-bit Loads and
 * Stores", section "The Kernel", epilogue). The pages' kernels take
 * (M, N, K, alpha, A, B, beta, C) with implicit leading dimensions lda = K,
 * ldb = ldc = N; this interface adds explicit leading dimensions and a stream.
 *
 * Layout (row-major): A(i,k) = A[i*lda + k] for i < M, k < K;
 *                     B(k,j) = B[k*ldb + j] for k < K, j < N;
 *                     C(i,j) = C[i*ldc + j] for i < M, j < N.
 * Elements outside those ranges (padding between rows) are never read or
 * written. (The norms and sgemm_mx4_quantize() at the end of this file may read
 * what lies between two rows of a matrix, 16 bytes at a time, and make no use of
 * it; it is never written.)
 *
 * Ownership: all matrix pointers are DEVICE pointers owned by the caller. The
 * library owns only a small per-(device, stream) workspace (split-K partial
 * tiles, their flags and a device status word), allocated on first use and
 * released by sgemm_shutdown(). No call here takes a torch type.
 *
 * Errors: every function returns an sgemm_status. Argument errors are found on
 * the host before anything is launched, and leave C untouched. Launch errors
 * are returned synchronously. A kernel that gives up on a bounded wait (a
 * copy, slot or partial that never arrived within the wait limit) records a
 * device status that sgemm_poll_device_status() reports.
 *
 * Threading: calls are asynchronous with respect to the host and ordered on
 * `stream`; the workspace is per (device, stream), so concurrent calls on
 * different streams do not share it. Host-side state is guarded by a mutex,
 * and the launches of one call are queued together: host threads may call on
 * one stream.
 *
 * CUDA graphs: sgemm, sgemm_ex, sgemm_strided_batched, sgemm_3xtf32,
 * sgemm_grouped, sgemm_grouped_wgrad, sgemm_i8, sgemm_grad_clip,
 * sgemm_rms_norm_grad, sgemm_linear_ce, sgemm_linear_ce_grad and sgemm_mx4 can be
 * captured into a graph and replayed, once a call of at least the same size
 * (for all but the first four and sgemm_grad_clip, whose workspace goes by the
 * form that their sizes choose: of the same sizes, leading dimensions and 16-byte
 * alignment of the matrices) has run on the capturing stream
 * outside the capture (it sets the device up and sizes the stream's workspace;
 * a call that would have to grow it during capture returns SGEMM_ERR_CAPTURE
 * and launches nothing). The graph keeps the stream's workspace: do not replay
 * it concurrently with other work on that stream's workspace. A later call
 * that needs a larger one gets a new block; the one that graphs hold stays
 * allocated until sgemm_shutdown(), after which they must not be replayed.
 * sgemm_noalloc, sgemm_rms_norm, sgemm_rms_norm_i8, sgemm_mx4_quantize and
 * sgemm_mx4_dequantize need no workspace at all.
 */
#ifndef SGEMM_GB300_H
#define SGEMM_GB300_H

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SGEMM_OK = 0,
  SGEMM_ERR_INVALID_DIM = -1,       /* M, N or K negative                        */
  SGEMM_ERR_INVALID_LD = -2,        /* lda < max(1,K), ldb < max(1,N), ldc < max(1,N) */
  SGEMM_ERR_NULL_PTR = -3,          /* a matrix that must be accessed is NULL     */
  SGEMM_ERR_UNSUPPORTED_DEVICE = -4,/* current device is not sm_103               */
  SGEMM_ERR_LAUNCH = -5,            /* CUDA runtime error while launching         */
  SGEMM_ERR_DEVICE_TIMEOUT = -6,    /* a kernel gave up on a bounded wait         */
  SGEMM_ERR_ALLOC = -7,             /* workspace allocation failed                */
  SGEMM_ERR_MISALIGNED = -8,        /* a pointer is not aligned to its element type (4 bytes for FP32) */
  SGEMM_ERR_INVALID_VALUE = -9,     /* other invalid argument (config id, buffer) */
  SGEMM_ERR_NOALLOC_CAPACITY = -10, /* sgemm_noalloc: problem needs more scratch
                                       than its fixed buffer holds             */
  SGEMM_ERR_CAPTURE = -11           /* the per-stream workspace would have to grow
                                       while `stream` is captured into a CUDA
                                       graph (nothing launched; call once on
                                       the stream before capturing)            */
} sgemm_status;

/* Operand forms of sgemm_ex / sgemm_strided_batched (row-major storage). */
typedef enum {
  SGEMM_OP_N = 0, /* the operand as stored                               */
  SGEMM_OP_T = 1  /* its transpose: A stored K x M, or B stored N x K     */
} sgemm_op;

/*
 * C = alpha * A * B + beta * C (FP32, FFMA path).
 *
 * M, N, K >= 0. lda >= max(1, K), ldb >= max(1, N), ldc >= max(1, N).
 * Quick returns: M == 0 or N == 0 does nothing. K == 0 or alpha == 0 scales
 * C by beta without reading A or B. beta == 0 never reads C, so C may hold
 * NaN or garbage. A and B may have any 4-byte alignment (the 128-bit and TMA
 * paths are used only when alignment allows). C must not overlap A or B.
 * stream: a cudaStream_t (NULL = legacy default stream). Problems with
 * M * N * K <= 2^25 run a latency-first kernel (one CTA per 32 x 32 tile, no
 * K-split) unless a tile configuration is forced; larger ones the persistent
 * kernel with the tuned configuration of their shape class.
 * Pages: the result is the one every kernel of "Shared Memory Tiling" (kernel
 * listing, final store), "Vectorized Memory Access: 128-bit Loads and Stores"
 * and "Warp Tiling: A Third Level of Tiling" (section "The Kernel",
 * epilogues) computes. The pages are silent on leading dimensions, shapes that
 * are not tile multiples, alignment, and the beta == 0 / alpha == 0 / K == 0
 * cases; the rules above are the plain BLAS reading of those points.
 */
int sgemm(int M, int N, int K, float alpha, const float* A, int lda, const float* B, int ldb,
          float beta, float* C, int ldc, void* stream);

/*
 * Opt-in tensor-core path: the same C = alpha * A * B + beta * C, with the
 * same arguments, checks and workspace, computed as three TF32 products per
 * FP32 product on the tcgen05 tensor cores (each operand split into a TF32
 * high part and a TF32 residual; the dropped residual product is below
 * 3 * 2^-20 of sum |a||b|, inside the library's FP32 tolerance, and integer
 * inputs up to 2^11 stay exact). The pages have no tensor-core kernel; this is
 * the split-operand method of Ootomo and Yokota (2022). It uses 4 * N * K
 * bytes of workspace for a transposed copy of B, plus 4 * M * K when the rows
 * of A are not 16-byte aligned (A is then copied). Reported separately from the
 * FFMA path.
 */
int sgemm_3xtf32(int M, int N, int K, float alpha, const float* A, int lda, const float* B,
                 int ldb, float beta, float* C, int ldc, void* stream);

/*
 * Kernel form of sgemm_3xtf32 for later calls (process-wide):
 *   SGEMM_X3_PAIR (the default): clusters of two CTAs on vertically adjacent
 *     128 x 256 tiles; the even CTA issues M = 256 MMAs over both
 *     (tcgen05 cta_group::2), each CTA holding its A tile and half of the B
 *     tile in shared memory and its 128 rows of the accumulator in TMEM;
 *   SGEMM_X3_SINGLE: single CTAs, each loading its own A and B tiles.
 * In both forms every CTA loads only its own tiles (no TMA load is shared
 * between CTAs). The pair form runs where the device can co-schedule CTA
 * pairs and the problem has at least two waves of whole tile pairs, else
 * single CTAs. Both give the same results within the tolerance (bit-identical
 * on integer inputs). Returns the previous setting, or
 * SGEMM_ERR_INVALID_VALUE (nothing changed) for another value. The pages are
 * silent (no tensor-core kernel).
 */
#define SGEMM_X3_SINGLE 1
#define SGEMM_X3_PAIR 2
int sgemm_3xtf32_set_kernel_form(int form);

/*
 * The plan sgemm_3xtf32 follows for an M x N x K problem (host arithmetic
 * only, no device needed): `form` is the requested kernel form, `pairs` how
 * many CTA pairs the device keeps resident (0: none), `sms` its SM count.
 * out (9 ints) = {form that runs, k-slice width, stages, CTAs, schedule
 * units (a CTA pair each in the pair forms), whole-tile units, K-split units,
 * k-slices, tile width in N}. The pair form falls back to single CTAs when
 * pairs == 0 or when every tile would be split along K. The tile width: 64
 * for N <= 64 and for problems of few 128-wide tiles ((sms / tiles)^2 >
 * ceil(K / 32) / 2), 128 for N <= 128 and for fewer than two waves of
 * 256-wide tiles with at most 48 slices of 32 of their work per SM, else 256;
 * the 64- and 128-wide tiles run on single CTAs with 32-wide slices.
 * Returns SGEMM_OK, SGEMM_ERR_INVALID_DIM unless
 * M, N, K >= 1 (only such problems launch the GEMM kernel), or
 * SGEMM_ERR_INVALID_VALUE for another form, pairs < 0, sms < 1 or a NULL out.
 * The pages are silent (no tensor-core kernel, one CTA per tile).
 */
int sgemm_3xtf32_plan(int M, int N, int K, int form, int pairs, int sms, int* out);

/*
 * C = alpha * op(A) * op(B) + beta * C, row-major, FFMA path. op(A) is M x K:
 * A itself (SGEMM_OP_N, stored M x K, lda >= max(1, K)) or the transpose of an
 * A stored K x M (SGEMM_OP_T, lda >= max(1, M)); op(B) is K x N: B (stored
 * K x N, ldb >= max(1, N)) or the transpose of a B stored N x K (ldb >=
 * max(1, K)). A stored transposed A arrives by TMA (no transposing copy); a
 * stored transposed B goes through the transposing copy the kernel uses for
 * row-major A. Column-major callers: a column-major M x N result is the
 * row-major N x M result of op(B)^T op(A)^T, i.e. call with the operands and
 * M, N swapped. Otherwise as sgemm(); SGEMM_ERR_INVALID_VALUE for another op.
 * The pages compute row-major A * B only; transposed operands are the BLAS
 * generalisation they never reach (silent).
 */
int sgemm_ex(int opA, int opB, int M, int N, int K, float alpha, const float* A, int lda,
             const float* B, int ldb, float beta, float* C, int ldc, void* stream);

/*
 * `batch` independent products C_i = alpha * op(A_i) * op(B_i) + beta * C_i
 * with A_i = A + i * strideA, B_i = B + i * strideB, C_i = C + i * strideC
 * (strides in elements, >= 0; a zero stride reuses one matrix for every i,
 * which is only valid for A and B). One launch covers every product: the
 * batch index is the outermost tile coordinate of the persistent schedule.
 * C_i must not overlap each other or any A_j, B_j. batch == 0 does nothing.
 * The pages are silent (one product per launch).
 */
int sgemm_strided_batched(int opA, int opB, int M, int N, int K, float alpha, const float* A,
                          int lda, long long strideA, const float* B, int ldb, long long strideB,
                          float beta, float* C, int ldc, long long strideC, int batch,
                          void* stream);

/*
 * The same C = alpha * A * B + beta * C with A, B and C in HOST memory (pinned
 * memory gives full copy bandwidth; pageable memory works but the copies may
 * block the calling thread). K is cut into chunks whose host -> device copies
 * overlap the multiplication of the previous chunk on the GPU (by default the
 * chunks grow geometrically, each as much wider as multiplying a column of K
 * takes longer than copying it); the incoming C (read only when beta != 0)
 * arrives in row panels and is added panel by panel at the end, and each
 * finished row panel is copied back while the next one is computed. All work is queued behind earlier work on
 * `stream`, and `stream` waits for the final copy: once the caller has
 * synchronised `stream`, C holds the result. The host buffers must stay
 * valid until then. Device buffers, two copy streams and their events are
 * owned by the library per (device, stream) and reused by later calls (freed
 * by sgemm_shutdown). Same argument checks and status codes as sgemm().
 * The pages are silent: they time device-resident operands only.
 */
int sgemm_host(int M, int N, int K, float alpha, const float* A, int lda, const float* B, int ldb,
               float beta, float* C, int ldc, void* stream);

/*
 * Copy/compute pipeline of later sgemm_host calls (process-wide). With
 * mid == 0 (the default) K is cut into geometrically growing chunks: a first
 * chunk of `first` columns (0: 128), each next one min(4, max(1.5,
 * M N / (M + N) / 755)) times wider, a remainder narrower than half the next
 * width joining the chunk before it, and, when last > 0, a last chunk of
 * `last` columns. With mid > 0: a first chunk of `first` columns (0: none;
 * taken only when K >= 2 * first + last), middle chunks of about `mid`
 * columns, and a last chunk of `last` columns (0: as wide as the middle
 * chunks). The last chunk is computed and copied back in `panels` row panels
 * (0: 4; at most 8; fewer when M < 512 * panels). Widths are rounded up to
 * multiples of 32; at most 9 chunks.
 * The result does not depend on the setting beyond the order of the sum
 * over k. Returns SGEMM_ERR_INVALID_VALUE (nothing changed) for a negative
 * value or more than 8 panels. The pages are silent.
 */
int sgemm_host_set_pipeline(int first, int mid, int last, int panels);

/* Human-readable text for a status code (static storage, never NULL). The
 * pages are silent: their kernels return no status. */
const char* sgemm_status_string(int status);

/*
 * Name of the tile configuration and schedule the calling thread's last
 * sgemm() used, copied into buf (at most len bytes, NUL-terminated).
 * Returns SGEMM_OK, or SGEMM_ERR_INVALID_VALUE if buf is NULL or len < 1.
 * The pages name the configuration beside every measurement ("Autotuning:
 * Searching the Tile-Shape Space", section "What The Sweep Found"); this is
 * that name for the library's own choice.
 */
int sgemm_last_config(char* buf, int len);

/*
 * Waits for `stream`, then reports and clears the device status word of this
 * (device, stream) workspace: SGEMM_OK, or SGEMM_ERR_DEVICE_TIMEOUT if a
 * kernel gave up on a bounded wait since the last poll. *detail (if not NULL)
 * receives the device-side code (1 = operand tile, 2 = slot release, 3 =
 * split partial, 4 = CTA rendezvous, 5 = the two CTAs of a two-SM pair of
 * sgemm_3xtf32 got different tensor-memory columns; none of them is a device
 * fault, and the context stays usable). SGEMM_ERR_LAUNCH if synchronising
 * fails. `detail` extends the one-argument form this call would otherwise have: the
 * status alone cannot say which wait gave up. The pages are silent (their
 * kernels have no bounded waits and report nothing).
 */
int sgemm_poll_device_status(void* stream, int* detail);

/* Frees every workspace, device buffer, stream and event the library
 * allocated (after synchronising the device). Later calls allocate again.
 * The pages are silent (their kernels allocate nothing). */
void sgemm_shutdown(void);

/*
 * Tile configurations compiled into the library. sgemm_config_count() gives
 * their number; sgemm_config_info() fills name (len bytes) and the tile
 * parameters of configuration `id` as
 * {BM, BN, BK, WM, WN, WNITER, TM, TN, NT, STAGES, MINB, KU, ORDER} in
 * params[13] (KU: k-steps per unrolled chunk; ORDER: 0 row-by-row FFMA, 1 zig-zag
 * FFMA, 2 paired FMA, 3 paired FMA column by column).
 * Pages: the tuple of "Autotuning: Searching the Tile-Shape Space", section
 * "Mechanics" (the kernel's template parameters), plus this kernel's own
 * pipeline depth, residency, unroll and FMA order.
 */
int sgemm_config_count(void);
int sgemm_config_info(int id, char* name, int len, int* params);

/*
 * Forces every later sgemm() on this process to use configuration `id`
 * (-1 restores the automatic per-shape choice). For tuning and tests; the
 * sweep of "Autotuning: Searching the Tile-Shape Space" ("Mechanics") times
 * one configuration at a time in the same way.
 */
int sgemm_force_config(int id);

/*
 * How row-major A reaches shared memory in later calls (process-wide).
 * The staged variant: where the configuration is built with it (32-wide
 * k-slices, at most 64 accumulators per lane), B arrives by TMA and A is
 * 16-byte aligned with lda (and, batched, the matrix stride) a multiple of 4,
 * one TMA box per k-slice copies A as it is stored into a staging slot and
 * one extra producer warp transposes it into the padded As[k][m], so the FMA
 * warps issue no copies. Otherwise every thread issues the transposing
 * 4-byte copy ("Vectorized Memory Access: 128-bit Loads and Stores", section
 * "Why As Has To Be Transposed"; the pages copy with the FMA threads).
 * on = 1 (the default): the staged variant where allowed and each CTA runs
 * at least 8 k-slices on average (below that its extra step of latency
 * costs more than it saves); 2: wherever allowed, whatever the size; 0:
 * never. Both fill the same As[k][m] and sum in the same order, so results
 * are bit-identical. Returns the previous setting, or
 * SGEMM_ERR_INVALID_VALUE (nothing changed) for another value.
 */
int sgemm_set_staged_a(int on);

/*
 * 1 when tile configuration `id` is built for every operand layout (op(A),
 * op(B) in {N, T}; sgemm_ex and sgemm_strided_batched can use it), 0 when
 * only for row-major A and B, SGEMM_ERR_INVALID_VALUE for an unknown id.
 * The pages are silent (row-major operands only).
 */
int sgemm_config_layouts(int id);

/*
 * The configuration sgemm() picks by itself for an M x N x K problem (the
 * tuned table's entry for the problem's shape class, ignoring
 * sgemm_force_config). *shape_class (if not NULL) receives the class:
 * 0 square-large (M * N >= 12 Mi), 1 square-small (M * N < 3 Mi),
 * 2 K-dominant (K >= 4 max(M, N)), 3 N <= 96, 4 M <= 96, 5 tiny (at most
 * 2^28 multiply-adds), 6 square-mid (3 Mi <= M * N < 12 Mi).
 * Returns the configuration id or SGEMM_ERR_INVALID_DIM. Host only.
 * Pages: "Autotuning: Searching the Tile-Shape Space" picks one configuration
 * by measurement for one shape ("What The Sweep Found") and notes that the
 * winner depends on the shape ("What Could Be Improved"); this repeats the
 * search per shape class.
 */
int sgemm_choose_config(int M, int N, int K, int* shape_class);

/*
 * The legality checker of the tile configurations, evaluated on the host:
 * 0 if the tuple is legal for the FFMA kernel, else the number of the first
 * rule it breaks. params = {BM, BN, BK, WM, WN, WNITER, TM, TN, NT, STAGES,
 * MINB, KU, ORDER}. derived (if not NULL) receives {WMITER, WSUBM, WSUBN, accumulators
 * per thread, shared bytes per CTA} when the tuple is legal.
 * Pages: "Autotuning: Searching the Tile-Shape Space", sections "Most
 * Configurations Are Not Wrong By A Little" (the kernel's unstated
 * assumptions) and "Mechanics" (a compile-time legality gate); the rules here
 * are this kernel's own assumptions.
 */
int sgemm_cfg_check(const int* params, int* derived);

/*
 * The persistent schedule sgemm() would use for an M x N x K problem with
 * configuration `id` on `capacity` resident CTAs (host arithmetic only, no
 * device needed), under the policy sgemm() would take (a forced one, else
 * the tuned policy of the problem's shape class). out = {tiles_m, tiles_n,
 * kiters, grid, dp_tiles, sk_q, sk_r, group_m}. Returns SGEMM_OK or an
 * argument error.
 * The pages launch one CTA per C tile ("Shared Memory Tiling", kernel launch
 * grid); the persistent schedule is this library's (silent on the pages).
 */
int sgemm_schedule_query(int M, int N, int K, int id, int capacity, int* out);

/*
 * Persistent-schedule policies (the values of policy[0]):
 *   SGEMM_SCHED_HYBRID      whole tiles, then the last one to two waves' worth
 *                           of tiles split into k-slice units (with fewer
 *                           tiles than CTA slots, every tile is split);
 *   SGEMM_SCHED_HYBRID_TAIL whole waves of whole tiles; only the ragged last
 *                           wave is split;
 *   SGEMM_SCHED_DATA_PARALLEL whole tiles only;
 *   SGEMM_SCHED_STREAM_K    every tile split, the k-slice units spread evenly;
 *   SGEMM_SCHED_SPLIT_K     every tile cut into policy[3] equal k-ranges.
 * A policy is int[4] = {mode, raster group height in tiles (>= 1), fewest
 * k-slices per CTA when splitting (>= 1), splits (>= 1)}. Every policy gives
 * a correct result; split partial sums are added in a fixed order, so a
 * policy always gives the same bits. The pages are silent (one CTA per tile).
 */
#define SGEMM_SCHED_HYBRID 0
#define SGEMM_SCHED_HYBRID_TAIL 1
#define SGEMM_SCHED_DATA_PARALLEL 2
#define SGEMM_SCHED_STREAM_K 3
#define SGEMM_SCHED_SPLIT_K 4

/*
 * The schedule of an M x N x K problem with BM x BN tiles and BK-wide
 * k-slices on `capacity` CTA slots under `policy` (host arithmetic only):
 * out as for sgemm_schedule_query. Returns SGEMM_OK, SGEMM_ERR_INVALID_DIM
 * (negative size, or more than 2^31 - 1 tiles) or SGEMM_ERR_INVALID_VALUE.
 */
int sgemm_schedule_plan(int M, int N, int K, int BM, int BN, int BK, int capacity,
                        const int* policy, int* out);

/*
 * Forces `policy` on every later sgemm(), sgemm_ex() and
 * sgemm_strided_batched() call of this process (the tuner and tests); NULL or
 * policy[0] < 0 restores the tuned policy of each problem's shape class.
 * Returns SGEMM_OK or SGEMM_ERR_INVALID_VALUE (nothing changed).
 */
int sgemm_force_schedule(const int* policy);

/*
 * The tuned policy sgemm() uses by itself for an M x N x K problem (that of
 * its shape class), written to policy[4]. Returns SGEMM_OK or an argument
 * error. Host only.
 */
int sgemm_choose_policy(int M, int N, int K, int* policy);

/*
 * Piece `i` of CTA `b` under the schedule {tiles_m, tiles_n, kiters, grid,
 * dp_tiles, sk_q, sk_r, group_m} (as returned above): out = {tile, kb, ke,
 * tile_m, tile_n, contributors, is_partial}. Returns the number of pieces of
 * CTA b, or a negative status. Host arithmetic only. Pages: silent (see
 * sgemm_schedule_query).
 */
int sgemm_schedule_piece(const int* sched, int b, int i, int* out);

/*
 * Diagnostic: launches one CTA that waits on a shared-memory barrier nothing
 * ever arrives on, with a limit of timeout_ns, through the same bounded wait
 * the GEMM kernels use. The wait must run out and record device code 1; read
 * it with sgemm_poll_device_status(). Nothing faults and nothing hangs. It
 * also leaves the workspace's flags and counters as launches that gave up can
 * leave them: later calls have to be right all the same, polled or not.
 * The pages are silent.
 */
int sgemm_diag_wait_timeout(long long timeout_ns, void* stream);

/* Upper bound, in nanoseconds, of every wait inside the kernels (default
 * 4e9). Values < 1000 are rejected. Returns the previous value or a negative
 * status. The pages are silent. */
long long sgemm_set_wait_timeout_ns(long long ns);

/*
 * Diagnostic: the TF32 tensor-core throughput of the current device, in
 * TFLOP/s, measured. One CTA per SM issues `iters` x 4 back-to-back
 * tcgen05.mma.kind::tf32 of M 128, N 256, K 8 from shared memory into tensor
 * memory, with no loads in the loop; the launch is timed with CUDA events
 * (about 6 ms at iters = 20000 on GB300). Synchronous. The 3xTF32 path's
 * roofline divides this by three. Returns SGEMM_ERR_INVALID_VALUE for iters
 * < 1 or a NULL result pointer, SGEMM_ERR_DEVICE_TIMEOUT if the MMAs did not
 * complete within 4 s. The pages are silent (no tensor-core kernel).
 */
int sgemm_diag_tf32_mma_rate(int iters, double* tflops);

/*
 * Diagnostic: the same measurement for the pair form the 3xTF32 path runs by
 * default. Clusters of two CTAs (as many as are resident at once); the even
 * CTA issues `iters` x 4 tcgen05.mma.cta_group::2.kind::tf32 of M 256 (128
 * rows per CTA), N 256 (half of B in each CTA), K 8. The rate counts the
 * multiply-adds of all SMs taking part. Same arguments, errors and duration
 * as sgemm_diag_tf32_mma_rate. The pages are silent.
 */
int sgemm_diag_tf32_pair_mma_rate(int iters, double* tflops);

/*
 * The same C = alpha * A * B + beta * C as sgemm(), with the same arguments,
 * checks and results, for callers that must not allocate device memory: code
 * running while a stream is captured into a graph, applications whose memory
 * pool owns every free byte and forbids hidden allocations, and latency-bound
 * loops that cannot absorb an allocation. The pages have no counterpart; this
 * is a packaging of the same kernel.
 *
 * The kernel's scratch (status word, one flag per persistent CTA, split-K
 * partial tiles) lives in one fixed 24 MiB device array inside the library,
 * which every GPU that loads the library holds until the process exits; no
 * call allocates. The first call on a device does the set-up (the array's
 * device address, the kernels' attributes): make it before any stream
 * capture. A problem whose schedule needs more scratch than the array holds
 * returns SGEMM_ERR_NOALLOC_CAPACITY and launches nothing (on a 152-SM GB300
 * every problem fits). All calls share the array: calls that overlap on the
 * GPU (other streams, other host threads) race and must not be issued. Every
 * wait inside the kernel is bounded by the library's wait limit
 * (sgemm_set_wait_timeout_ns). A kernel that gives up records its code in the
 * array, where it stays until sgemm_noalloc_poll_status() reads it
 * (sgemm_poll_device_status() reports only the per-stream workspaces). The
 * tile configuration is always the automatic choice (sgemm_force_config()
 * does not apply), and problems with M * N * K <= 2^25 run the same
 * tiny-problem kernel as sgemm().
 */
int sgemm_noalloc(int M, int N, int K, float alpha, const float* A, int lda, const float* B,
                  int ldb, float beta, float* C, int ldc, void* stream);

/*
 * Waits for `stream`, then reports and clears the device status that
 * sgemm_noalloc calls on the current device recorded in the library's fixed
 * array: SGEMM_OK, or SGEMM_ERR_DEVICE_TIMEOUT with *detail (if not NULL)
 * set to the code (the same codes as sgemm_poll_device_status). After a
 * timeout it also clears the array's split-K flags, which an aborted call can
 * leave published. Allocates nothing. SGEMM_OK when sgemm_noalloc has not
 * run on this device; SGEMM_ERR_LAUNCH if synchronising or a copy fails.
 * The pages have no counterpart (they report no device-side errors).
 */
int sgemm_noalloc_poll_status(void* stream, int* detail);

/*
 * Three kernels of the pages' series, rebuilt for this GPU to measure what
 * each technique buys; sgemm() never uses them:
 *   kernel 3 -- shared-memory tiling ("Shared Memory Tiling"): 32 x 32 C tile
 *               per CTA of 1024 threads, one output per thread;
 *   kernel 7 -- vectorized 2-D block tiling ("Vectorized Memory Access:
 *               128-bit Loads and Stores"): 128 x 128 C tile, BK = 8, 8 x 8
 *               outputs per thread, 128-bit loads, A transposed in shared
 *               memory;
 *   kernel 8 -- warp tiling ("Warp Tiling: A Third Level of Tiling"):
 *               128 x 64 C tile, BK = 16, 64 x 32 warp tiles of 2 x 2
 *               sub-tiles, 4 x 4 outputs per thread and sub-tile.
 * Arguments after `kernel`, their checks, the quick returns and the result
 * are those of sgemm(): any shape, leading dimension and 4-byte alignment
 * (128-bit accesses are used only when A, B and C are 16-byte aligned and
 * lda, ldb, ldc are multiples of 4). One CTA per C tile on `stream`; no
 * workspace and no device status. kernel other than 3, 7 or 8 returns
 * SGEMM_ERR_INVALID_VALUE; more than 2^31 - 1 tiles SGEMM_ERR_INVALID_DIM.
 */
int sgemm_ladder(int kernel, int M, int N, int K, float alpha, const float* A, int lda,
                 const float* B, int ldb, float beta, float* C, int ldc, void* stream);

/*
 * The linear layers of a language model's experts: products grouped by expert
 * with ragged row counts, their weight gradients, the 8-bit integer product
 * that serves such a layer, and the clipping of many gradients. The pages
 * have none of these.
 */

/* Element types of the calls below. */
typedef enum {
  SGEMM_TYPE_F32 = 0,  /* IEEE single precision */
  SGEMM_TYPE_BF16 = 1, /* bfloat16              */
  SGEMM_TYPE_F16 = 2   /* IEEE half precision   */
} sgemm_type;

/*
 * Y[r, :] = alpha * X[r, :] * op(W_e) + beta * Y[r, :] for every row r of group
 * e, e = 0 .. E - 1. X is T x K and Y is T x N, row-major; group e is the rows
 * [offsets[e], offsets[e + 1]), offsets being E + 1 ints on the DEVICE (they
 * may come from a kernel queued before; the host never reads them). op(W_e) is
 * K x N: W_e = W + e * strideW (in elements) as stored K x N (SGEMM_OP_N, ldw >=
 * max(1, N)) or the transpose of a W_e stored N x K (SGEMM_OP_T, ldw >= max(1,
 * K)). The gradient of X is the same call on dY with the other op.
 *
 * type is that of X and W, out_type that of Y: FP32 operands give FP32; BF16
 * and F16 operands give any type. Products are accumulated in FP32 and rounded
 * once (16-bit results of 16-bit operands leave the tensor cores, which
 * truncate, every 1024 products); FP32 operands are cut into three BF16 parts each (an error below
 * 2^-23 of |x||w| per product). An FP32 operand that is infinite or NaN makes
 * every output it takes part in NaN; BF16 and F16 follow IEEE arithmetic.
 * beta == 0 never reads Y; alpha == 0 or K == 0 never reads X or W.
 *
 * Rows outside every group are not touched. Groups may be empty. Offsets are
 * clamped to 0 .. T; a group whose end lies before its start is empty, and rows
 * that an earlier group has are left out of a later one. strideW == 0 reads one
 * matrix for every group. E <= 1024. Any element-aligned pointers and leading
 * dimensions work; operands whose rows (or strideW) are not multiples of 16
 * bytes are first copied into the per-stream workspace. Y must not overlap X or
 * W. Workspace, capture and device status as for sgemm().
 * Returns SGEMM_ERR_INVALID_VALUE for another op or type, E > 1024, strideW <
 * 0 or 16-bit results of FP32 operands; SGEMM_ERR_INVALID_DIM, _INVALID_LD,
 * _NULL_PTR and _MISALIGNED as sgemm().
 */
int sgemm_grouped(int op, int type, int out_type, int E, int T, int N, int K, float alpha,
                  const void* X, int ldx, const void* W, int ldw, long long strideW,
                  const int* offsets, float beta, void* Y, int ldy, void* stream);

/*
 * C_e = alpha * A_e^T * B_e + beta * C_e, e = 0 .. E - 1: A is T x M, B is T x
 * N, row-major, A_e and B_e their rows [offsets[e], offsets[e + 1]), and C_e =
 * C + e * strideC (in elements) is M x N. With A = dY and B = X it is the
 * gradient of weights stored N x K (op T above), with A = X and B = dY of
 * weights stored K x N. An empty group gives beta * C_e (zeros for beta == 0,
 * without reading C). Types, offsets, accuracy and errors as sgemm_grouped();
 * FP32 results of 16-bit operands leave the tensor cores every 256 rows and
 * are added in FP32 with rounding to nearest. The C_e must not overlap.
 */
int sgemm_grouped_wgrad(int type, int out_type, int E, int T, int M, int N, float alpha,
                        const void* A, int lda, const void* B, int ldb, const int* offsets,
                        float beta, void* C, int ldc, long long strideC, void* stream);

/*
 * Rows of X (M x K, of `type`) to 8-bit integers with one scale a row:
 * scale[m] = max_k |X[m, k]| / 127, Q[m, k] = X[m, k] / scale[m] rounded to the
 * nearest integer (ties to even) within +-127; both quotients are rounded to
 * FP32. A row of zeros has scale 0 and zeros. A row with an infinity or a NaN
 * gets it as its scale (NaN where both occur), and its products are NaN.
 */
int sgemm_i8_quantize(int M, int K, int type, const void* X, int ldx, signed char* Q, int ldq,
                      float* scale, void* stream);

/*
 * C[m, n] = (sum_k A[m, k] * B[n, k]) * scaleA[m] * scaleB[n]: A is M x K and B
 * N x K (a channel per row), 8-bit integers; scaleA has M, scaleB N FP32
 * values. The sum is an exact 32-bit integer for every input; its product with
 * the scales is formed in FP32 and rounded once to out_type. K <=
 * SGEMM_I8_MAX_K (SGEMM_ERR_INVALID_DIM beyond). K == 0 gives zeros times the
 * scales. Any leading dimensions (>= max(1, K), ldc >= max(1, N)) and byte
 * alignment; rows of A or B that are not multiples of 16 bytes are first copied
 * into the workspace. Errors, workspace and capture as sgemm().
 */
#define SGEMM_I8_MAX_K 131071
int sgemm_i8(int M, int N, int K, const signed char* A, int lda, const float* scaleA,
             const signed char* B, int ldb, const float* scaleB, int out_type, void* C, int ldc,
             void* stream);

/*
 * Tile of later sgemm_grouped, sgemm_grouped_wgrad, sgemm_i8, sgemm_linear_ce and
 * sgemm_mx4 calls
 * (process-wide; for measurements and tests): `width` token rows (wgrad: rows
 * of C) by 128 output columns on one CTA (ctas = 1), or by 256 on a pair of CTAs
 * that share their MMAs (ctas = 2). width 0 restores the choice by size. A call
 * whose types have no kernel of that tile keeps its own choice. Results differ
 * only in the order of sums. Returns SGEMM_ERR_INVALID_VALUE (nothing changed)
 * for a tile that no kernel is built for.
 */
int sgemm_grouped_set_tile(int width, int ctas);

/*
 * The 2-norm of n tensors taken together, and their clipping:
 *   norm = sqrt(sum of all g^2), coef = min(1, max_norm / (norm + 1e-6)),
 *   out_i = grads_i * coef.
 * grads, out, sizes and types are HOST arrays of n: device pointers, element
 * counts and element types (out_i has the type of grads_i, and is grads_i or
 * does not overlap any grads_j). *norm (device memory; may be NULL) receives
 * the norm before clipping. out == NULL computes the norm only. Tensors that
 * are their own out are not written when coef is 1. Squares are summed in FP32
 * over at most 32 values and in FP64 beyond, in an order that does not depend
 * on timing. A NaN among the gradients makes the norm and every output NaN; an
 * infinity makes the norm infinite and coef 0, as the formula says. The host
 * arrays are read before the call returns (a captured graph keeps them).
 * Returns SGEMM_ERR_INVALID_DIM for n < 0 or a size < 0 or above 2^40,
 * SGEMM_ERR_INVALID_VALUE for max_norm < 0 or NaN or an unknown type,
 * SGEMM_ERR_NULL_PTR, SGEMM_ERR_MISALIGNED (pointers need element alignment).
 */
int sgemm_grad_clip(int n, const void* const* grads, void* const* out, const long long* sizes,
                    const int* types, float max_norm, float* norm, void* stream);

/*
 * The output end of a language model: the residual's addition with the norm of
 * its rows, what follows it in training (the loss over the vocabulary) and in
 * serving (8-bit and 4-bit products). The pages have none of these.
 */

/*
 * H = X + R rounded to `type` (R == NULL: H is X, and the argument H is not
 * used), and row by row
 *   rstd = 1 / sqrt(mean(H^2) + eps),   Y = H * rstd * weight.
 * X, R, H and Y are M x N of `type`, weight has N values of weight_type (`type`
 * or FP32), rstd (may be NULL) M FP32 values. Sums and products are FP32, Y is
 * rounded once. eps is at least 1e-30. A row with an infinity or a NaN gives
 * what the formula gives. Y and H may be X or R themselves (the same address and
 * pitch); otherwise they must not overlap what is read, nor each other. N == 0
 * or M == 0 does nothing. Any leading dimensions (>= max(1, N)) and element
 * alignment; rows that start on 16 bytes are faster. Capturable without any
 * call before.
 * Returns SGEMM_ERR_INVALID_VALUE (type, eps), _INVALID_DIM, _INVALID_LD,
 * _NULL_PTR, _MISALIGNED as sgemm().
 */
int sgemm_rms_norm(int M, int N, int type, const void* X, int ldx, const void* R, int ldr,
                   const void* weight, int weight_type, float eps, void* H, int ldh, void* Y,
                   int ldy, float* rstd, void* stream);

/*
 * The same norm as 8-bit integers with one scale a row, as sgemm_i8 takes them:
 * with u = H * weight in FP32,
 *   step = max_n |u[m, n]| / 127,  Q = u / step rounded to the nearest integer
 *   (ties to even) within +-127,  scale[m] = step * rstd[m];
 * both quotients are rounded to FP32. A row of zeros has scale 0 and zeros. A row
 * with an infinity or a NaN has a NaN for its scale (an infinity where only a
 * product u overflows), so its products are no numbers. H may be X or R
 * themselves. Errors as sgemm_rms_norm().
 */
int sgemm_rms_norm_i8(int M, int N, int type, const void* X, int ldx, const void* R, int ldr,
                      const void* weight, int weight_type, float eps, void* H, int ldh,
                      signed char* Q, int ldq, float* scale, void* stream);

/*
 * Gradients of sgemm_rms_norm, with n = H * rstd and d = dY * weight:
 *   dX = rstd * (d - n * mean(d * n)) + dH,   dweight = sum over rows of dY * n.
 * dX is the gradient of X and of R alike. dH (may be NULL) is the gradient that
 * reaches H itself. dX or dweight (of weight_type) may be NULL: not formed. dX
 * may be dY, H or dH itself. dweight is summed in FP32 in an order that depends
 * on the sizes, the leading dimensions, where the matrices start within 16 bytes
 * and the GPU's number of SMs, not on timing, and rounded once; M == 0 sets it to
 * zeros. Workspace and capture as said above; errors as sgemm_rms_norm().
 */
int sgemm_rms_norm_grad(int M, int N, int type, const void* dY, int lddy, const void* H, int ldh,
                        const void* weight, int weight_type, const float* rstd, const void* dH,
                        int lddh, void* dX, int lddx, void* dweight, void* stream);

/*
 * Softmax cross entropy over a vocabulary without keeping the logits. With z[t,
 * v] = X[t] . W[v], X being T x H and W V x H of `type`, row-major:
 *   lse[t] = log(sum_v exp(z[t, v])),   loss[t] = lse[t] - z[t, target[t]];
 * target has T 64-bit integers on the device. loss[t] is 0 where target[t] is
 * ignore_index, and NaN where it is neither that nor in 0 .. V - 1. lse (may be
 * NULL) is written for every row. Both are FP32, and so are the logits and the
 * sums: 16-bit operands are multiplied exactly and leave the tensor cores every
 * 512 products, FP32 ones as in sgemm_grouped(). Logits of -infinity have no
 * share; a NaN or +infinity among a row's makes its loss NaN. (FP32 operands
 * have no infinite logits: an infinity among them makes every logit that it takes
 * part in NaN, as in sgemm_grouped(), and with it the row's loss.)
 * The vocabulary is taken in pieces, so that the workspace stays below 256 MB
 * beside the products' own (FP32: 512 MB), or the statistics (logits) of 2048
 * words at a time. Any leading dimensions (>= max(1, H)) and element
 * alignment; operands whose rows are not multiples of 16 bytes are copied piece
 * by piece. Workspace, capture, device status and errors as sgemm().
 */
int sgemm_linear_ce(int type, int T, int V, int H, const void* X, int ldx, const void* W, int ldw,
                    const long long* target, long long ignore_index, float* loss, float* lse,
                    void* stream);

/*
 * Gradients of sgemm_linear_ce: with dloss[t] the gradient of loss[t] and
 *   G[t, v] = (exp(z[t, v] - lse[t]) - (v == target[t])) * dloss[t]
 * (0 where target[t] is ignore_index, NaN where it is no word),
 *   dX = G W (T x H),   dW = G^T X (V x H), of `type`; either may be NULL.
 * The logits are formed once more; a piece of G at a time is held in `type`,
 * scaled by a power of two and max|dloss| so that F16 keeps small ones. Sums are
 * FP32, rounded once. X must hold finite numbers in rows that are not counted,
 * too, and W in words that have no share (0 times an infinity or a NaN is NaN). dX and dW must not overlap X, W or each other. Workspace:
 * 512 MB (or 2048 words of G) beside the products' own, and T x H FP32 sums
 * where G takes several pieces. Errors as sgemm_linear_ce().
 */
int sgemm_linear_ce_grad(int type, int T, int V, int H, const void* X, int ldx, const void* W,
                         int ldw, const long long* target, long long ignore_index, const float* lse,
                         const float* dloss, void* dX, int lddx, void* dW, int lddw, void* stream);

/*
 * Rows of X (M x K, of `type`) to 4-bit floating point (E2M1: 0, 0.5, 1, 1.5, 2,
 * 3, 4, 6 and their negatives) in blocks of 32 values with a power of two each:
 * the power is floor(log2(max|x|)) - 2, at least -127, and x / 2^power is rounded
 * to the nearest of those values, ties to the even code, beyond 6 to 6. All of
 * this is exact, whatever the order of the work.
 *
 * Q has M rows of 16 bytes for each block, ldq bytes apart (a multiple of 16, at
 * least 16 * ceil(K / 32)): value 2i of a block in the low half of byte i, its
 * sign in the half's highest bit. Values past the row's end are zeros.
 *
 * scale holds power + 127 as a byte for each block, in the order in which the
 * tensor cores read them: tiles of 128 rows x 4 blocks, 512 bytes each, all of
 * the first 128 rows' tiles first; in a tile row r and block b stand at (r % 32)
 * * 16 + (r / 32) * 4 + b. It has 512 * ceil(M / 128) * ceil(ceil(K / 32) / 4)
 * bytes; places that belong to no block are set to 0. A block of zeros has 0. A
 * block with an infinity or a NaN has 255, which stands for NaN.
 *
 * Q and scale start on 16 bytes; X at any element, with any ldx >= max(1, K).
 * M == 0 or K == 0 does nothing. Capturable without any call before. Errors as
 * sgemm().
 */
int sgemm_mx4_quantize(int M, int K, int type, const void* X, int ldx, unsigned char* Q, int ldq,
                       unsigned char* scale, void* stream);

/* The values that Q and scale stand for, rounded to `type`: M x K. Errors as
 * sgemm_mx4_quantize(). */
int sgemm_mx4_dequantize(int M, int K, const unsigned char* Q, int ldq, const unsigned char* scale,
                         int type, void* X, int ldx, void* stream);

/*
 * C[m, n] = sum_k A[m, k] * B[n, k]: A is M x K and B N x K (a channel per row),
 * codes and scales as sgemm_mx4_quantize() writes them; C is M x N of out_type.
 * Products are exact and added up in FP32 on the tensor cores (which truncate;
 * sums leave them every 8192 values of k, FP32 results every 2048), rounded
 * once. A scale of 255 makes every sum that its block takes part in NaN. The
 * scales' places that belong to no block must not be 255. K == 0 gives zeros.
 * lda and ldb are in bytes (multiples of 16); A, B and the scales start on 16
 * bytes; C at any element with any ldc >= max(1, N). C must not overlap the
 * operands. Workspace, capture, device status and errors as sgemm().
 */
int sgemm_mx4(int M, int N, int K, const unsigned char* A, int lda, const unsigned char* scaleA,
              const unsigned char* B, int ldb, const unsigned char* scaleB, int out_type, void* C,
              int ldc, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_GB300_H */
