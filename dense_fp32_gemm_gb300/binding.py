"""ctypes binding of libsgemm_gb300.so: the C ABI of include/sgemm_gb300.h
under the same names, plus a torch convenience that only marshals arguments
(device tensors -> pointers and leading dimensions, the current stream).

There is no fallback: if the CUDA library is not built, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.machinery
import importlib.util
import os
import threading

from . import build as _build

_lock = threading.Lock()
_lib = None

SGEMM_OK = 0
SGEMM_ERR_INVALID_DIM = -1
SGEMM_ERR_INVALID_LD = -2
SGEMM_ERR_NULL_PTR = -3
SGEMM_ERR_UNSUPPORTED_DEVICE = -4
SGEMM_ERR_LAUNCH = -5
SGEMM_ERR_DEVICE_TIMEOUT = -6
SGEMM_ERR_ALLOC = -7
SGEMM_ERR_MISALIGNED = -8
SGEMM_ERR_INVALID_VALUE = -9
SGEMM_ERR_NOALLOC_CAPACITY = -10
SGEMM_ERR_CAPTURE = -11

SGEMM_OP_N = 0
SGEMM_OP_T = 1

SGEMM_TYPE_F32 = 0
SGEMM_TYPE_BF16 = 1
SGEMM_TYPE_F16 = 2
SGEMM_I8_MAX_K = 131071

PARAM_NAMES = ("BM", "BN", "BK", "WM", "WN", "WNITER", "TM", "TN", "NT", "STAGES", "MINB", "KU", "ORDER")


class SgemmError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {sgemm_status_string(status)} (status {status})")
        self.status = status


def library_path() -> str:
    """The library to load: SGEMM_GB300_LIB if set (the tuner's candidate
    build), else the in-tree product library."""
    return os.environ.get("SGEMM_GB300_LIB") or _build.LIB_PATH


def lib() -> ctypes.CDLL:
    """The loaded CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is missing: build the CUDA library first "
                    "(python -c 'import __graft_entry__ as g; g.build()')")
            L = ctypes.CDLL(path)
            I, F, P, LL = ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_longlong
            IP = ctypes.POINTER(ctypes.c_int)
            sig = {
                "sgemm": (I, [I, I, I, F, P, I, P, I, F, P, I, P]),
                "sgemm_status_string": (ctypes.c_char_p, [I]),
                "sgemm_last_config": (I, [ctypes.c_char_p, I]),
                "sgemm_poll_device_status": (I, [P, IP]),
                "sgemm_shutdown": (None, []),
                "sgemm_config_count": (I, []),
                "sgemm_config_info": (I, [I, ctypes.c_char_p, I, IP]),
                "sgemm_force_config": (I, [I]),
                "sgemm_set_staged_a": (I, [I]),
                "sgemm_cfg_check": (I, [IP, IP]),
                "sgemm_schedule_query": (I, [I, I, I, I, I, IP]),
                "sgemm_schedule_piece": (I, [IP, I, I, IP]),
                "sgemm_schedule_plan": (I, [I, I, I, I, I, I, I, IP, IP]),
                "sgemm_force_schedule": (I, [IP]),
                "sgemm_choose_policy": (I, [I, I, I, IP]),
                "sgemm_diag_wait_timeout": (I, [LL, P]),
                "sgemm_set_wait_timeout_ns": (LL, [LL]),
                "sgemm_noalloc": (I, [I, I, I, F, P, I, P, I, F, P, I, P]),
                "sgemm_noalloc_poll_status": (I, [P, IP]),
                "sgemm_choose_config": (I, [I, I, I, IP]),
                "sgemm_3xtf32": (I, [I, I, I, F, P, I, P, I, F, P, I, P]),
                "sgemm_ex": (I, [I, I, I, I, I, F, P, I, P, I, F, P, I, P]),
                "sgemm_host": (I, [I, I, I, F, P, I, P, I, F, P, I, P]),
                "sgemm_ladder": (I, [I, I, I, I, F, P, I, P, I, F, P, I, P]),
                "sgemm_3xtf32_set_kernel_form": (I, [I]),
                "sgemm_3xtf32_plan": (I, [I, I, I, I, I, I, IP]),
                "sgemm_host_set_pipeline": (I, [I, I, I, I]),
                "sgemm_config_layouts": (I, [I]),
                "sgemm_diag_tf32_mma_rate": (I, [I, ctypes.POINTER(ctypes.c_double)]),
                "sgemm_diag_tf32_pair_mma_rate": (I, [I, ctypes.POINTER(ctypes.c_double)]),
                "sgemm_grouped": (I, [I, I, I, I, I, I, I, F, P, I, P, I, LL, P, F, P, I, P]),
                "sgemm_grouped_wgrad": (I, [I, I, I, I, I, I, F, P, I, P, I, P, F, P, I, LL, P]),
                "sgemm_i8_quantize": (I, [I, I, I, P, I, P, I, P, P]),
                "sgemm_i8": (I, [I, I, I, P, I, P, P, I, P, I, P, I, P]),
                "sgemm_grouped_set_tile": (I, [I, I]),
                "sgemm_grad_clip": (I, [I, P, P, P, P, F, P, P]),
                "sgemm_rms_norm": (I, [I, I, I, P, I, P, I, P, I, F, P, I, P, I, P, P]),
                "sgemm_rms_norm_i8": (I, [I, I, I, P, I, P, I, P, I, F, P, I, P, I, P, P]),
                "sgemm_rms_norm_grad": (I, [I, I, I, P, I, P, I, P, I, P, P, I, P, I, P, P]),
                "sgemm_linear_ce": (I, [I, I, I, I, P, I, P, I, P, LL, P, P, P]),
                "sgemm_linear_ce_grad": (I, [I, I, I, I, P, I, P, I, P, LL, P, P, P, I, P, I, P]),
                "sgemm_mx4_quantize": (I, [I, I, I, P, I, P, I, P, P]),
                "sgemm_mx4_dequantize": (I, [I, I, P, I, P, I, P, I, P]),
                "sgemm_mx4": (I, [I, I, I, P, I, P, P, I, P, I, P, I, P]),
                "sgemm_strided_batched": (I, [I, I, I, I, I, F, P, I, LL, P, I, LL, F, P, I, LL,
                                              I, P]),
            }
            for name, (res, args) in sig.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
        return _lib


def _ints(n, values=None):
    arr = (ctypes.c_int * n)()
    if values is not None:
        for i, v in enumerate(values):
            arr[i] = int(v)
    return arr


# ---- the C ABI, same names ------------------------------------------------------
def sgemm(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> int:
    """Raw call: A, B, C are device addresses (ints), stream a cudaStream_t
    handle (int) or None. Returns the status code."""
    return lib().sgemm(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def sgemm_host(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> int:
    """C = alpha*A*B + beta*C on HOST matrices (addresses as ints), copies
    overlapped with the GEMM; C is final once `stream` is synchronised."""
    return lib().sgemm_host(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def sgemm_host_set_pipeline(first: int, mid: int, last: int, panels: int) -> int:
    """K-chunk widths (first, middle, last) and the row panels of the last
    chunk for later sgemm_host calls; 0 picks the default. Returns a status."""
    return lib().sgemm_host_set_pipeline(first, mid, last, panels)


def sgemm_ex(opA, opB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> int:
    """C = alpha*op(A)*op(B) + beta*C (ops SGEMM_OP_N / SGEMM_OP_T)."""
    return lib().sgemm_ex(opA, opB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def sgemm_strided_batched(opA, opB, M, N, K, alpha, A, lda, strideA, B, ldb, strideB, beta, C,
                          ldc, strideC, batch, stream=None) -> int:
    """`batch` products C_i = alpha*op(A_i)*op(B_i) + beta*C_i, one launch."""
    return lib().sgemm_strided_batched(opA, opB, M, N, K, alpha, A, lda, strideA, B, ldb, strideB,
                                       beta, C, ldc, strideC, batch, stream)


def sgemm_3xtf32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> int:
    """Opt-in tensor-core path (three TF32 products per FP32 product), same
    arguments as sgemm(). Returns the status code."""
    return lib().sgemm_3xtf32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def sgemm_status_string(status: int) -> str:
    return lib().sgemm_status_string(status).decode()


def sgemm_last_config() -> str:
    buf = ctypes.create_string_buffer(256)
    lib().sgemm_last_config(buf, 256)
    return buf.value.decode()


def sgemm_poll_device_status(stream=None):
    """(status, device detail code)."""
    detail = ctypes.c_int(0)
    st = lib().sgemm_poll_device_status(stream, ctypes.byref(detail))
    return st, detail.value


def sgemm_shutdown() -> None:
    lib().sgemm_shutdown()


def sgemm_config_count() -> int:
    return lib().sgemm_config_count()


def sgemm_set_staged_a(on: int) -> int:
    """Row-major A through the staging ring and producer warp: 1 where allowed
    and each CTA runs at least 8 k-slices (default), 2 wherever allowed, 0
    never (the transposing copy). Returns the previous setting."""
    return lib().sgemm_set_staged_a(on)


def sgemm_config_info(cid: int):
    name = ctypes.create_string_buffer(128)
    params = _ints(13)
    st = lib().sgemm_config_info(cid, name, 128, params)
    if st != SGEMM_OK:
        raise SgemmError(st, "sgemm_config_info")
    return name.value.decode(), dict(zip(PARAM_NAMES, list(params)))


def sgemm_diag_tf32_mma_rate(iters: int = 20000):
    """(status, TFLOP/s): the measured TF32 tensor-core throughput of the
    current device (synchronous, about 6 ms)."""
    v = ctypes.c_double(0.0)
    st = lib().sgemm_diag_tf32_mma_rate(iters, ctypes.byref(v))
    return st, v.value


def sgemm_diag_tf32_pair_mma_rate(iters: int = 20000):
    """(status, TFLOP/s): the same for two-SM (cta_group::2) MMAs issued by
    CTA pairs."""
    v = ctypes.c_double(0.0)
    st = lib().sgemm_diag_tf32_pair_mma_rate(iters, ctypes.byref(v))
    return st, v.value


def sgemm_config_layouts(cid: int) -> int:
    """1: configuration `cid` is built for every operand layout; 0: row-major
    operands only; negative: an error status."""
    return lib().sgemm_config_layouts(cid)


def sgemm_force_config(cid: int) -> int:
    return lib().sgemm_force_config(cid)


SHAPE_CLASSES = ("square_large", "square_small", "k_dominant", "skinny_n", "skinny_m", "tiny",
                 "square_mid")


def sgemm_choose_config(M, N, K):
    """(config id, shape class name) of the automatic choice."""
    cls = ctypes.c_int(-1)
    cid = lib().sgemm_choose_config(M, N, K, ctypes.byref(cls))
    if cid < 0:
        raise SgemmError(cid, "sgemm_choose_config")
    return cid, SHAPE_CLASSES[cls.value]


def sgemm_cfg_check(params):
    """(rule, derived): rule 0 = legal; derived = {WMITER, WSUBM, WSUBN,
    acc_per_thread, smem_bytes} for a legal tuple."""
    if isinstance(params, dict):
        params = [params[k] for k in PARAM_NAMES]
    p = _ints(13, params)
    d = _ints(5)
    rule = lib().sgemm_cfg_check(p, d)
    derived = dict(zip(("WMITER", "WSUBM", "WSUBN", "acc", "smem_bytes"), list(d))) if rule == 0 else None
    return rule, derived


SCHED_FIELDS = ("tiles_m", "tiles_n", "kiters", "grid", "dp_tiles", "sk_q", "sk_r", "group_m")
PIECE_FIELDS = ("tile", "kb", "ke", "tile_m", "tile_n", "contributors", "is_partial")


def sgemm_schedule_query(M, N, K, cid, capacity):
    out = _ints(8)
    st = lib().sgemm_schedule_query(M, N, K, cid, capacity, out)
    if st != SGEMM_OK:
        raise SgemmError(st, "sgemm_schedule_query")
    return dict(zip(SCHED_FIELDS, list(out)))


SCHED_HYBRID, SCHED_HYBRID_TAIL, SCHED_DATA_PARALLEL, SCHED_STREAM_K, SCHED_SPLIT_K = 0, 1, 2, 3, 4
SCHED_MODES = (SCHED_HYBRID, SCHED_HYBRID_TAIL, SCHED_DATA_PARALLEL, SCHED_STREAM_K, SCHED_SPLIT_K)


def sgemm_schedule_plan(M, N, K, BM, BN, BK, capacity, policy):
    """The schedule for BM x BN x BK tiles under `policy` = (mode, group_m,
    min_units, splits), host arithmetic only; raises on an argument error."""
    out = _ints(8)
    st = lib().sgemm_schedule_plan(M, N, K, BM, BN, BK, capacity, _ints(4, policy), out)
    if st != SGEMM_OK:
        raise SgemmError(st, "sgemm_schedule_plan")
    return dict(zip(SCHED_FIELDS, list(out)))


def sgemm_force_schedule(policy=None) -> int:
    """Force (mode, group_m, min_units, splits) on later calls; None restores
    the tuned per-class policy. Returns the status code."""
    return lib().sgemm_force_schedule(None if policy is None else _ints(4, policy))


def sgemm_choose_policy(M, N, K):
    """(status, (mode, group_m, min_units, splits)) that sgemm() takes by itself."""
    out = _ints(4)
    st = lib().sgemm_choose_policy(M, N, K, out)
    return st, tuple(out)


def sgemm_schedule_piece(sched: dict, b: int, i: int):
    """(number of pieces of CTA b, piece i as a dict)."""
    v = _ints(8, [sched[k] for k in SCHED_FIELDS])
    out = _ints(7)
    n = lib().sgemm_schedule_piece(v, b, i, out)
    if n < 0:
        raise SgemmError(n, "sgemm_schedule_piece")
    return n, dict(zip(PIECE_FIELDS, list(out)))


def sgemm_diag_wait_timeout(timeout_ns: int, stream=None) -> int:
    return lib().sgemm_diag_wait_timeout(timeout_ns, stream)


def sgemm_set_wait_timeout_ns(ns: int) -> int:
    return lib().sgemm_set_wait_timeout_ns(ns)


def sgemm_noalloc(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> int:
    """Same call as sgemm() for callers that cannot allocate device memory:
    the kernel's scratch comes from a fixed buffer inside the library.
    Returns the status code."""
    return lib().sgemm_noalloc(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def sgemm_noalloc_poll_status(stream=None):
    """(status, device detail code) of the sgemm_noalloc calls on this device
    since the last poll; synchronises `stream` first."""
    detail = ctypes.c_int(0)
    st = lib().sgemm_noalloc_poll_status(stream, ctypes.byref(detail))
    return st, detail.value


def sgemm_ladder(kernel, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> int:
    """One of the pages' kernels (3: shared-memory tiling, 7: vectorized
    block tiling, 8: warp tiling) on device matrices; same arguments and
    result as sgemm(). Returns the status code."""
    return lib().sgemm_ladder(kernel, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


LADDER_KERNELS = (3, 7, 8)


SGEMM_X3_SINGLE, SGEMM_X3_PAIR = 1, 2
X3_FORMS = (SGEMM_X3_PAIR, SGEMM_X3_SINGLE)


X3_PLAN_FIELDS = ("form", "bk", "stages", "ctas", "units", "dp_units", "split_units", "kiters",
                  "bn")


def sgemm_3xtf32_plan(M: int, N: int, K: int, form: int, pairs: int, sms: int):
    """(status, {field: value}) of the plan sgemm_3xtf32 follows (host only)."""
    out = _ints(len(X3_PLAN_FIELDS))
    st = lib().sgemm_3xtf32_plan(M, N, K, form, pairs, sms, out)
    return st, dict(zip(X3_PLAN_FIELDS, list(out)))


def sgemm_3xtf32_set_kernel_form(form: int) -> int:
    """SGEMM_X3_PAIR (default): CTA pairs with two-SM MMAs; SGEMM_X3_SINGLE: single
    CTAs. Returns the previous setting (or an error status)."""
    return lib().sgemm_3xtf32_set_kernel_form(form)


# ---- products grouped by expert, 8-bit products, gradient clipping -------------------
def sgemm_grouped(op, type, out_type, E, T, N, K, alpha, X, ldx, W, ldw, strideW, offsets, beta, Y,
                  ldy, stream=None) -> int:
    """Y[r] = alpha*X[r]*op(W_e) + beta*Y[r] for the rows r of group e, whose
    bounds are E + 1 ints on the device. Returns the status code."""
    return lib().sgemm_grouped(op, type, out_type, E, T, N, K, alpha, X, ldx, W, ldw, strideW,
                               offsets, beta, Y, ldy, stream)


def sgemm_grouped_wgrad(type, out_type, E, T, M, N, alpha, A, lda, B, ldb, offsets, beta, C, ldc,
                        strideC, stream=None) -> int:
    """C_e = alpha*A_e^T*B_e + beta*C_e over the rows of each group. Returns the
    status code."""
    return lib().sgemm_grouped_wgrad(type, out_type, E, T, M, N, alpha, A, lda, B, ldb, offsets,
                                     beta, C, ldc, strideC, stream)


def sgemm_i8_quantize(M, K, type, X, ldx, Q, ldq, scale, stream=None) -> int:
    """Rows of X to 8-bit integers Q with one FP32 scale a row. Returns the
    status code."""
    return lib().sgemm_i8_quantize(M, K, type, X, ldx, Q, ldq, scale, stream)


def sgemm_i8(M, N, K, A, lda, scaleA, B, ldb, scaleB, out_type, C, ldc, stream=None) -> int:
    """C = (A B^T) * scaleA[:, None] * scaleB on 8-bit integers (B is N x K).
    Returns the status code."""
    return lib().sgemm_i8(M, N, K, A, lda, scaleA, B, ldb, scaleB, out_type, C, ldc, stream)


def sgemm_grouped_set_tile(width: int, ctas: int = 1) -> int:
    """Tile width and CTAs per tile of later grouped and 8-bit products; 0
    restores the choice by size. Returns the status code."""
    return lib().sgemm_grouped_set_tile(width, ctas)


def sgemm_grad_clip(grads, out, sizes, types, max_norm, norm, stream=None) -> int:
    """The 2-norm of tensors taken together, and out_i = grads_i * min(1,
    max_norm / (norm + 1e-6)): sequences of device addresses, element counts
    and SGEMM_TYPE_* codes. out None: the norm only. Returns the status code."""
    n = len(grads)
    vp = (ctypes.c_void_p * n)(*grads)
    vo = None if out is None else (ctypes.c_void_p * n)(*out)
    return lib().sgemm_grad_clip(n, vp, vo, (ctypes.c_longlong * n)(*sizes),
                                 (ctypes.c_int * n)(*types), max_norm, norm, stream)


# ---- the output end of a model: norm, loss over the vocabulary ----------------------
def sgemm_rms_norm(M, N, type, X, ldx, R, ldr, weight, weight_type, eps, H, ldh, Y, ldy, rstd=None,
                   stream=None) -> int:
    """H = X + R (R None: X itself), Y = H / sqrt(mean(H^2) + eps) * weight row by
    row; rstd (may be None) receives 1 / sqrt(...). Returns the status code."""
    return lib().sgemm_rms_norm(M, N, type, X, ldx, R, ldr, weight, weight_type, eps, H, ldh, Y, ldy,
                                rstd, stream)


def sgemm_rms_norm_i8(M, N, type, X, ldx, R, ldr, weight, weight_type, eps, H, ldh, Q, ldq, scale,
                      stream=None) -> int:
    """The same with the norm as 8-bit integers Q and one FP32 scale a row.
    Returns the status code."""
    return lib().sgemm_rms_norm_i8(M, N, type, X, ldx, R, ldr, weight, weight_type, eps, H, ldh, Q,
                                   ldq, scale, stream)


def sgemm_rms_norm_grad(M, N, type, dY, lddy, H, ldh, weight, weight_type, rstd, dH, lddh, dX, lddx,
                        dweight, stream=None) -> int:
    """Gradients of sgemm_rms_norm; dH, dX and dweight may be None. Returns the
    status code."""
    return lib().sgemm_rms_norm_grad(M, N, type, dY, lddy, H, ldh, weight, weight_type, rstd, dH,
                                     lddh, dX, lddx, dweight, stream)


def sgemm_linear_ce(type, T, V, H, X, ldx, W, ldw, target, ignore_index, loss, lse=None, stream=None) -> int:
    """loss[t] = log(sum_v exp(X[t] . W[v])) - X[t] . W[target[t]], 0 where the
    target is ignore_index; lse (may be None) receives the logarithms. Returns
    the status code."""
    return lib().sgemm_linear_ce(type, T, V, H, X, ldx, W, ldw, target, ignore_index, loss, lse, stream)


def sgemm_linear_ce_grad(type, T, V, H, X, ldx, W, ldw, target, ignore_index, lse, dloss, dX, lddx, dW,
                         lddw, stream=None) -> int:
    """Gradients of sgemm_linear_ce for dloss; dX or dW may be None. Returns the
    status code."""
    return lib().sgemm_linear_ce_grad(type, T, V, H, X, ldx, W, ldw, target, ignore_index, lse, dloss,
                                      dX, lddx, dW, lddw, stream)


# ---- 4-bit floating point in blocks of 32 with a power of two each ------------------
def sgemm_mx4_quantize(M, K, type, X, ldx, Q, ldq, scale, stream=None) -> int:
    """Rows of X to 4-bit codes Q (16 bytes for every 32 values) and the blocks'
    powers in tiles of 128 rows x 4 blocks. Returns the status code."""
    return lib().sgemm_mx4_quantize(M, K, type, X, ldx, Q, ldq, scale, stream)


def sgemm_mx4_dequantize(M, K, Q, ldq, scale, type, X, ldx, stream=None) -> int:
    """The values that Q and scale stand for. Returns the status code."""
    return lib().sgemm_mx4_dequantize(M, K, Q, ldq, scale, type, X, ldx, stream)


def sgemm_mx4(M, N, K, A, lda, scaleA, B, ldb, scaleB, out_type, C, ldc, stream=None) -> int:
    """C = A B^T on 4-bit codes with their blocks' powers (B is N x K). Returns the
    status code."""
    return lib().sgemm_mx4(M, N, K, A, lda, scaleA, B, ldb, scaleB, out_type, C, ldc, stream)


# ---- torch conveniences (marshalling only) ------------------------------------------
def _stream_handle(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _ld(t, name):
    if t.dim() != 2 or t.dtype.__repr__() != "torch.float32":
        raise ValueError(f"{name} must be a 2-D float32 tensor")
    if t.is_neg():
        raise ValueError(f"{name} is a negated view: call resolve_neg() first")
    if t.size(1) > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be row-major (unit stride along rows)")
    least = max(t.size(1), 1)
    if t.size(0) < 2 or t.numel() == 0:
        return least
    if t.stride(0) < least:
        raise ValueError(f"{name} has overlapping rows (a row stride below the row length)")
    return t.stride(0)


def gemm(A, B, C, alpha=1.0, beta=0.0, stream=None):
    """C <- alpha*A@B + beta*C on CUDA float32 tensors (row-major views with
    any row stride). Raises SgemmError on a non-zero status. Returns C."""
    import torch
    M, K = A.shape
    K2, N = B.shape
    if K2 != K or tuple(C.shape) != (M, N):
        raise ValueError("shape mismatch")
    for t, nm in ((A, "A"), (B, "B"), (C, "C")):
        if not t.is_cuda:
            raise ValueError(f"{nm} must be a CUDA tensor")
    st = sgemm(M, N, K, float(alpha), A.data_ptr(), _ld(A, "A"), B.data_ptr(), _ld(B, "B"),
               float(beta), C.data_ptr(), _ld(C, "C"), _stream_handle(stream))
    if st != SGEMM_OK:
        raise SgemmError(st, "sgemm")
    if not C.is_inference():
        torch.autograd.graph.increment_version(C)
    return C


# (csrc_torch/marshal.cpp: checks, allocation and the C call in native code.
# Autograd does not see through them: results carry no graph, layers.py has the
# differentiable form. A tensor that is given to be written counts as changed.)
@functools.cache
def _native():
    """The marshalling module, bound to the loaded library."""
    import torch  # noqa: F401  (its libraries come first)
    path = _build.marshal_path()
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build the CUDA library first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    loader = importlib.machinery.ExtensionFileLoader("_marshal", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_marshal", loader))
    loader.exec_module(module)
    names = ("sgemm_grouped", "sgemm_grouped_wgrad", "sgemm_i8_quantize", "sgemm_i8", "sgemm_grad_clip",
             "sgemm_rms_norm", "sgemm_rms_norm_i8", "sgemm_rms_norm_grad", "sgemm_linear_ce",
             "sgemm_linear_ce_grad", "sgemm_mx4_quantize", "sgemm_mx4_dequantize", "sgemm_mx4")
    module.bind(tuple(ctypes.cast(getattr(lib(), n), ctypes.c_void_p).value for n in names), SgemmError)
    return module


def grouped_gemm(X, W, offsets, Y=None, op="T", alpha=1.0, beta=0.0, out_dtype=None, stream=None):
    """Y[r] = alpha * X[r] @ op(W[e]) + beta * Y[r] for the rows r of group e,
    offsets[e] <= r < offsets[e + 1] (int32, on the device). W is (E, N, K) with
    op "T" and (E, K, N) with op "N"; the gradient of X is grouped_gemm(dY, W,
    offsets, op=the other). Without Y a new tensor of out_dtype (default: X's)
    is returned, in which rows outside every group are not set."""
    if op != "N" and op != "T":
        raise ValueError('op must be "N" or "T"')
    return _native().grouped_gemm(X, W, offsets, Y, op == "T", alpha, beta, out_dtype, stream)


def grouped_wgrad(A, B, offsets, C=None, alpha=1.0, beta=0.0, out_dtype=None, stream=None):
    """C[e] = alpha * A_e.T @ B_e + beta * C[e] over the rows of each group: the
    gradient of W (E, N, K) with A = dY, B = X, of W (E, K, N) with A = X, B = dY.
    Without C a new (E, M, N) tensor of out_dtype (default: A's) is returned."""
    return _native().grouped_wgrad(A, B, offsets, C, alpha, beta, out_dtype, stream)


def i8_quantize(X, Q=None, scale=None, stream=None):
    """(Q, scale): the rows of X as 8-bit integers with one FP32 scale a row,
    scale = max|X[m]| / 127. A new Q has rows padded to 16 bytes."""
    return _native().i8_quantize(X, Q, scale, stream)


def i8_gemm(A, scaleA, B, scaleB, C=None, out_dtype=None, stream=None):
    """C = (A @ B.T) * scaleA[:, None] * scaleB on int8 A (M, K) and B (N, K), the
    sum an exact integer. Without C a new tensor of out_dtype (default bfloat16)
    is returned."""
    return _native().i8_gemm(A, scaleA, B, scaleB, C, out_dtype, stream)


def clip_grad_norm(grads, max_norm, out=None, stream=None):
    """The 2-norm (a float32 scalar tensor) of contiguous CUDA tensors taken
    together, before clipping; out[i] = grads[i] * min(1, max_norm / (norm +
    1e-6)), in place without `out`."""
    return _native().clip_grad_norm(grads, max_norm, out, stream)


def rms_norm(X, weight, residual=None, eps=1e-6, Y=None, H=None, rstd=None, stream=None):
    """(Y, H, rstd): H = X + residual in X's type (X itself without a residual),
    rstd = 1 / sqrt(mean(H^2) + eps) of each row in float32, Y = H * rstd *
    weight. weight is of X's type or float32. Y and H may be X or the residual
    itself."""
    return _native().rms_norm(X, weight, residual, eps, Y, H, rstd, stream)


def rms_norm_i8(X, weight, residual=None, eps=1e-6, Q=None, scale=None, H=None, stream=None):
    """(Q, scale, H): the same norm as 8-bit integers with one float32 scale a row,
    as i8_gemm takes them: Q * scale[:, None] stands for H * rstd * weight. A new
    Q has rows padded to 16 bytes."""
    return _native().rms_norm_i8(X, weight, residual, eps, Q, scale, H, stream)


def rms_norm_grad(dY, H, weight, rstd, dH=None, dX=None, dweight=None, want=(True, True), stream=None):
    """(dX, dweight): gradients of rms_norm. dX is that of X and of the residual
    alike; dH is the gradient that reaches H itself. What is not wanted is None."""
    return _native().rms_norm_grad(dY, H, weight, rstd, dH, dX, dweight, bool(want[0]), bool(want[1]),
                                   stream)


def linear_cross_entropy(X, W, target, ignore_index=-100, loss=None, lse=None, stream=None):
    """(loss, lse), float32 with a value for each row of X: the softmax cross
    entropy of the logits X @ W.T with the words target (int64), 0 where target
    is ignore_index, and the logarithm of the sum of the logits' exponentials.
    The logits are not kept. A target that is no word gives NaN. Logits of
    -infinity have no share; an infinite float32 operand gives NaN."""
    return _native().linear_cross_entropy(X, W, target, ignore_index, loss, lse, stream)


def linear_cross_entropy_grad(X, W, target, lse, dloss, ignore_index=-100, dX=None, dW=None,
                              want=(True, True), stream=None):
    """(dX, dW): gradients of linear_cross_entropy for dloss, the gradient of each
    row's loss (float32). What is not wanted is None. X must hold finite numbers in
    rows that are not counted, too, and W in words that have no share: the products
    add 0 times them."""
    return _native().linear_cross_entropy_grad(X, W, target, lse, dloss, ignore_index, dX, dW,
                                               bool(want[0]), bool(want[1]), stream)


def mx4_quantize(X, Q=None, scale=None, stream=None):
    """(Q, scale): the rows of X as 4-bit floating point (E2M1) in blocks of 32
    values with a power of two each. Q is uint8, (rows, 16 * blocks), the first
    of two values in a byte's low half; scale is uint8, the biased powers in the
    tiles that mx4_gemm reads (see mx4_tile_scales)."""
    return _native().mx4_quantize(X, Q, scale, stream)


def mx4_dequantize(Q, scale, K, X=None, out_dtype=None, stream=None):
    """The (rows, K) values that Q and scale stand for, as out_dtype (default
    bfloat16)."""
    return _native().mx4_dequantize(Q, scale, K, X, out_dtype, stream)


def mx4_gemm(A, scaleA, B, scaleB, C=None, out_dtype=None, stream=None):
    """C = A @ B.T on the 4-bit values of A (M rows) and B (N rows), added up in
    FP32. Without C a new tensor of out_dtype (default bfloat16) is returned."""
    return _native().mx4_gemm(A, scaleA, B, scaleB, C, out_dtype, stream)


def mx4_tile_scales(scales):
    """Biased powers of two, uint8 (rows, blocks), as the vector that mx4_gemm
    reads: tiles of 128 rows x 4 blocks of 512 bytes, row of tiles after row of
    tiles; in a tile row r and block b stand at (r % 32) * 16 + (r // 32) * 4 + b.
    Places that belong to no block are 0."""
    import torch
    if scales.dim() != 2 or scales.dtype != torch.uint8:
        raise ValueError("scales must be a 2-D uint8 tensor")
    rows, blocks = scales.shape
    tiles = torch.nn.functional.pad(scales, (0, -blocks % 4, 0, -rows % 128))
    return tiles.view((rows + 127) // 128, 4, 32, (blocks + 3) // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)
