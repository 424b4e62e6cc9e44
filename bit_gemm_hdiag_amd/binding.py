"""ctypes binding of libmxsens (include/mxsens.h), same names as the C ABI.

Argument marshalling only: tensors must already live in GPU memory; the
binding checks dtypes and layouts, allocates outputs and workspaces with
torch when the caller passes none, and enqueues the C call on the current
HIP stream. Every step of the method runs in the library's kernels. There
is no CPU fallback: a missing library raises at import.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, Structure, c_char_p, c_double, c_float, c_int32, c_int64, c_size_t, c_void_p
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_lib", "libmxsens.so")

MXS_F32, MXS_BF16 = 0, 1
STATUS = {0: "MXS_OK", -1: "MXS_ERR_ARG", -2: "MXS_ERR_SHAPE", -3: "MXS_ERR_BUDGET",
          -4: "MXS_ERR_WORKSPACE", -5: "MXS_ERR_DEVICE", -6: "MXS_ERR_UNSUPPORTED"}


class MxsError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}: {msg}")
        self.status = status


class _QMat(Structure):
    _fields_ = [("rows", c_int64), ("K", c_int64), ("n8", c_int32), ("n6", c_int32),
                ("n4", c_int32), ("reserved", c_int32),
                ("q8", c_void_p), ("ld8", c_int64), ("q6", c_void_p), ("ld6", c_int64),
                ("q4", c_void_p), ("ld4", c_int64), ("sc", c_void_p), ("lds", c_int64)]


class _Lora(Structure):
    _fields_ = [("K", c_int64), ("N", c_int64), ("n", c_int32), ("R", c_int32), ("dtype", c_int32),
                ("reserved", c_int32), ("A", c_void_p), ("B", c_void_p), ("scale", c_void_p), ("rank", c_void_p)]


class _Kv4Cache(Structure):
    _fields_ = [("pages", c_int64), ("page_size", c_int32), ("H", c_int32), ("D", c_int32), ("reserved", c_int32),
                ("kc", c_void_p), ("ks", c_void_p), ("vc", c_void_p), ("vs", c_void_p)]


def library_path() -> str:
    return _LIB_PATH


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"libmxsens.so is not built ({_LIB_PATH}); run __graft_entry__.build() "
                          "or python -m bit_gemm_hdiag_amd.build")
    lib = ctypes.CDLL(_LIB_PATH)
    P, S = c_void_p, c_int32
    sig = {
        "mxs_status_string": (c_char_p, [S]),
        "mxs_last_error": (c_char_p, []),
        "mxs_version": (c_int32, []),
        "mxs_budget_blocks": (S, [c_int64, c_int32, c_int32, P]),
        "mxs_calibrate_workspace": (c_size_t, [c_int64, c_int64]),
        "mxs_score_workspace": (c_size_t, [c_int64, c_int64]),
        "mxs_calibrate": (S, [P, c_int32, c_int64, c_int64, c_int64, P, P, c_size_t, P]),
        "mxs_score": (S, [P, c_int32, c_int64, c_int64, c_int64, P, P, P, c_size_t, P]),
        "mxs_allocate": (S, [P, c_int64, c_int32, c_int32, P, P, P]),
        "mxs_quantize": (S, [P, c_int32, c_int64, P, POINTER(_QMat), P]),
        "mxs_mixed_gemm_workspace": (c_size_t, [POINTER(_QMat), POINTER(_QMat)]),
        "mxs_mixed_gemm": (S, [POINTER(_QMat), POINTER(_QMat), P, c_int64, P, c_size_t, P]),
        "mxs_mixed_gemm_noalloc": (S, [POINTER(_QMat), POINTER(_QMat), P, c_int64, P]),
        "mxs_mixed_gemm_mx_workspace": (c_size_t, [POINTER(_QMat), POINTER(_QMat)]),
        "mxs_mixed_gemm_mx": (S, [POINTER(_QMat), POINTER(_QMat), P, c_int64, P, c_size_t, P]),
        "mxs_quantize_kv": (S, [P, c_int32, c_int64, c_int64, c_int64, P, P, P]),
        "mxs_allocate_blocks": (S, [P, c_int64, c_int32, c_int32, P, P, P]),
        "mxs_output_error_workspace": (c_size_t, [c_int64, c_int64]),
        "mxs_output_error": (S, [P, P, c_int32, c_int64, c_int64, c_int64, c_int64, c_int64, P, c_int64, P, P,
                                 c_size_t, P]),
        "mxs_layer_budget": (S, [c_int32, P, P, P, c_double, P, P]),
        "mxs_attend_kv4_workspace": (c_size_t, [c_int64, c_int64, c_int64, c_int64]),
        "mxs_attend_kv4": (S, [P, P, P, P, P, c_int64, c_int64, c_int64, c_int64, ctypes.c_float, P, P, c_size_t, P]),
        "mxs_mixed_gemm_fused_workspace": (c_size_t, [c_int64, c_int32, POINTER(_QMat)]),
        "mxs_mixed_gemm_fused": (S, [P, c_int32, c_int64, c_int64, P, POINTER(_QMat), P, c_int64, P, c_size_t, P]),
        "mxs_prepare_weights_size": (c_size_t, [POINTER(_QMat)]),
        "mxs_prepare_weights": (S, [POINTER(_QMat), P, c_size_t, P]),
        "mxs_mixed_gemm_prepared_workspace": (c_size_t, [POINTER(_QMat), POINTER(_QMat)]),
        "mxs_mixed_gemm_prepared": (S, [POINTER(_QMat), POINTER(_QMat), P, c_size_t, P, c_int64, P, c_size_t, P]),
        "mxs_mixed_gemm_fused_prepared_workspace": (c_size_t, [c_int64, c_int32, POINTER(_QMat)]),
        "mxs_mixed_gemm_fused_prepared": (S, [P, c_int32, c_int64, c_int64, P, POINTER(_QMat), P, c_size_t, P,
                                              c_int64, P, c_size_t, P]),
        "mxs_rope_frequencies": (S, [c_int32, c_double, c_int32, c_double, c_double, c_double, c_double, P]),
        "mxs_rope": (S, [P, c_int32, c_int64, c_int64, c_int64, c_int64, c_int64, P, P, c_int32, c_int32, c_float, P,
                         c_int64, c_int64, P]),
        "mxs_kv4_append": (S, [P, P, P, c_int32, c_int64, c_int64, c_int64, c_int64, c_int64, P, P, P, c_int32, c_int32,
                               c_float, P]),
        "mxs_kv4_read": (S, [P, P, c_int64, c_int32, P, c_int64, c_int64, P, c_int64, c_int64, P]),
        "mxs_kv4_copy": (S, [P, P, P, P, c_int64, P]),
        "mxs_kv4_fork": (S, [P, P, P, c_int64, c_int64, P, P, P, c_int64, P]),
        "mxs_kv4_reserve_workspace": (c_size_t, [c_int64, c_int64]),
        "mxs_kv4_reserve": (S, [P, P, P, c_int64, c_int64, P, P, c_int64, P, P, P, c_size_t, P]),
        "mxs_kv4_compact": (S, [P, P, c_int64, c_int64, P, P, P, P, c_int64, P, P]),
        "mxs_kv4_compact_granted": (S, [P, P, c_int64, c_int64, P, P, P, P, P, c_int64, P, P]),
        "mxs_kv4_release": (S, [P, P, P, c_int64, c_int64, P, P, P, P]),
        "mxs_verify_tree_workspace": (c_size_t, [c_int64] * 4),
        "mxs_verify_tree": (S, [P, c_int32, c_int64, c_int64, P, P, P, c_int64, c_int64, c_int64, P, c_int64, c_int32,
                                P, P, P, P, P, P, c_size_t, P]),
        "mxs_lora_add_workspace": (c_size_t, [c_int64, P]),
        "mxs_lora_add": (S, [P, c_int64, c_int64, P, P, P, c_int64, P, c_size_t, P]),
        "mxs_attend_kv4_tree_workspace": (c_size_t, [c_int32] + [c_int64] * 7),
        "mxs_attend_kv4_tree": (S, [P, c_int32, c_int64, P, P, c_int64, P, P, P, c_int64, c_int64, c_int64, c_int64,
                                    c_int64, c_int64, c_float, P, c_int64, P, c_size_t, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    return lib


_lib = _load()
EXPORTED = ("mxs_status_string", "mxs_last_error", "mxs_version", "mxs_budget_blocks",
            "mxs_calibrate_workspace", "mxs_score_workspace", "mxs_calibrate", "mxs_score",
            "mxs_allocate", "mxs_quantize", "mxs_mixed_gemm_workspace", "mxs_mixed_gemm", "mxs_mixed_gemm_noalloc",
            "mxs_mixed_gemm_mx_workspace", "mxs_mixed_gemm_mx", "mxs_quantize_kv", "mxs_allocate_blocks",
            "mxs_output_error_workspace", "mxs_output_error", "mxs_layer_budget", "mxs_attend_kv4_workspace",
            "mxs_attend_kv4", "mxs_mixed_gemm_fused_workspace", "mxs_mixed_gemm_fused",
            "mxs_prepare_weights_size", "mxs_prepare_weights", "mxs_mixed_gemm_prepared_workspace",
            "mxs_mixed_gemm_prepared", "mxs_mixed_gemm_fused_prepared_workspace", "mxs_mixed_gemm_fused_prepared",
            "mxs_rope_frequencies", "mxs_rope", "mxs_kv4_append", "mxs_kv4_read", "mxs_attend_kv4_tree_workspace",
            "mxs_attend_kv4_tree", "mxs_kv4_copy", "mxs_kv4_fork", "mxs_kv4_reserve_workspace", "mxs_kv4_reserve",
            "mxs_kv4_compact", "mxs_kv4_compact_granted", "mxs_kv4_release", "mxs_verify_tree_workspace", "mxs_verify_tree",
            "mxs_lora_add_workspace", "mxs_lora_add")


def _check(status: int, where: str):
    if status != 0:
        raise MxsError(status, where, _lib.mxs_last_error().decode())


def _stream(dev) -> c_void_p:
    return c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return MXS_BF16
    if t.dtype == torch.float32:
        return MXS_F32
    raise TypeError(f"unsupported element type {t.dtype} (bf16 or fp32)")


def _dev2d(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    return t.data_ptr(), t.stride(0)


def _ptr(t):
    return None if t is None or t.numel() == 0 else t.data_ptr()


def _workspace(nbytes: int, dev, ws):
    """(tensor, pointer, bytes). The caller keeps the tensor until the library
    function has returned: given back earlier, the block could go to a call of
    another thread that enqueues between this call's launches."""
    if nbytes == 0:
        return ws, None, 0
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


# --------------------------------------------------------------------- plain calls
def mxs_version() -> int:
    return _lib.mxs_version()


def mxs_status_string(status: int) -> str:
    return _lib.mxs_status_string(status).decode()


def mxs_last_error() -> str:
    return _lib.mxs_last_error().decode()


def mxs_budget_blocks(K: int, bp8: int, bp6: int):
    out = (c_int32 * 3)()
    _check(_lib.mxs_budget_blocks(K, bp8, bp6, ctypes.cast(out, c_void_p)), "mxs_budget_blocks")
    return int(out[0]), int(out[1]), int(out[2])


def mxs_calibrate_workspace(M: int, K: int) -> int:
    return int(_lib.mxs_calibrate_workspace(M, K))


def mxs_score_workspace(N: int, K: int) -> int:
    return int(_lib.mxs_score_workspace(N, K))


def mxs_calibrate(X: torch.Tensor, hdiag: torch.Tensor | None = None, ws=None) -> torch.Tensor:
    """hdiag[k] += sum_t X[t, k]^2 (fp64, fixed order). X [M, K] bf16/fp32 on the GPU."""
    px, ldx = _dev2d(X, "X")
    M, K = X.shape
    if hdiag is None:
        hdiag = torch.zeros(K, dtype=torch.float64, device=X.device)
    if hdiag.dtype != torch.float64 or not hdiag.is_contiguous() or hdiag.numel() != K:
        raise ValueError("hdiag must be a contiguous fp64 [K] tensor")
    ws, pw, nw = _workspace(mxs_calibrate_workspace(M, K), X.device, ws)
    _check(_lib.mxs_calibrate(px, _dtype(X), M, K, ldx, hdiag.data_ptr(), pw, nw, _stream(X.device)),
           "mxs_calibrate")
    return hdiag


def mxs_score(W: torch.Tensor, hdiag: torch.Tensor, score: torch.Tensor | None = None, ws=None):
    """score[k] = hdiag[k] * sum_n (W - Q4(W))[n, k]^2, fp64 [K]."""
    pw_, ldw = _dev2d(W, "W")
    N, K = W.shape
    if score is None:
        score = torch.empty(K, dtype=torch.float64, device=W.device)
    if hdiag.dtype != torch.float64 or not hdiag.is_contiguous() or hdiag.numel() != K:
        raise ValueError("hdiag must be a contiguous fp64 [K] tensor")
    ws, p, n = _workspace(mxs_score_workspace(N, K), W.device, ws)
    _check(_lib.mxs_score(pw_, _dtype(W), N, K, ldw, hdiag.data_ptr(), score.data_ptr(), p, n,
                          _stream(W.device)), "mxs_score")
    return score


def mxs_allocate(score: torch.Tensor, bp8: int, bp6: int, bits=None, perm=None):
    """(bits uint8 [K] in {8, 6, 4}, perm int32 [K] gather form)."""
    if not score.is_cuda or score.dtype != torch.float64 or not score.is_contiguous():
        raise ValueError("score must be a contiguous fp64 GPU tensor")
    K = score.numel()
    if bits is None:
        bits = torch.empty(K, dtype=torch.uint8, device=score.device)
    if perm is None:
        perm = torch.empty(K, dtype=torch.int32, device=score.device)
    _check(_lib.mxs_allocate(score.data_ptr(), K, bp8, bp6, bits.data_ptr(), perm.data_ptr(),
                             _stream(score.device)), "mxs_allocate")
    return bits, perm


@dataclass(frozen=True)
class QMat:
    """Planes of a matrix quantised with one bit map (see mxs_qmat). Frozen:
    the C struct is built once, on first use, and reused by every call."""
    rows: int
    K: int
    n8: int
    n6: int
    n4: int
    q8: torch.Tensor
    q6: torch.Tensor
    q4: torch.Tensor
    sc: torch.Tensor

    def c_struct(self) -> _QMat:
        q = self.__dict__.get("_c")
        if q is not None:
            return q

        def ld(t, width):
            return t.stride(0) if t.numel() else max(width, 1)
        for t in (self.q8, self.q6, self.q4, self.sc):
            if t.numel() and t.stride(1) != 1:
                raise ValueError("planes need unit column stride")
        q = _QMat(self.rows, self.K, self.n8, self.n6, self.n4, 0,
                  _ptr(self.q8), ld(self.q8, 32 * self.n8), _ptr(self.q6), ld(self.q6, 24 * self.n6),
                  _ptr(self.q4), ld(self.q4, 16 * self.n4), _ptr(self.sc), ld(self.sc, self.K // 32))
        object.__setattr__(self, "_c", q)
        return q

    def rows_slice(self, r0: int, r1: int) -> "QMat":
        return QMat(r1 - r0, self.K, self.n8, self.n6, self.n4, self.q8[r0:r1], self.q6[r0:r1],
                    self.q4[r0:r1], self.sc[r0:r1])


def qmat_alloc(rows: int, K: int, n8: int, n6: int, n4: int, device) -> QMat:
    kw = dict(device=device)
    return QMat(rows, K, n8, n6, n4,
                torch.empty((rows, 32 * n8), dtype=torch.int8, **kw),
                torch.empty((rows, 24 * n6), dtype=torch.uint8, **kw),
                torch.empty((rows, 16 * n4), dtype=torch.uint8, **kw),
                torch.empty((rows, K // 32), dtype=torch.uint8, **kw))


def mxs_quantize(X: torch.Tensor, perm: torch.Tensor | None, n8: int, n6: int, n4: int,
                 out: QMat | None = None) -> QMat:
    """MXINT 8/6/4 planes of X[:, perm] (perm None = identity)."""
    px, ldx = _dev2d(X, "X")
    R, K = X.shape
    if perm is not None and (perm.dtype != torch.int32 or not perm.is_contiguous() or perm.numel() != K
                             or not perm.is_cuda):
        raise ValueError("perm must be a contiguous int32 [K] GPU tensor")
    if out is None:
        out = qmat_alloc(R, K, n8, n6, n4, X.device)
    if out.rows != R or out.K != K:
        raise ValueError("output planes do not match X")
    q = out.c_struct()
    _check(_lib.mxs_quantize(px, _dtype(X), ldx, _ptr(perm), ctypes.byref(q), _stream(X.device)),
           "mxs_quantize")
    return out


def mxs_mixed_gemm_workspace(A: QMat, W: QMat) -> int:
    a, w = A.c_struct(), W.c_struct()
    return int(_lib.mxs_mixed_gemm_workspace(ctypes.byref(a), ctypes.byref(w)))


def _gemm(fn, wsfn, name, A: QMat, W: QMat, Y, ws) -> torch.Tensor:
    dev = A.sc.device
    if Y is None:
        Y = torch.empty((A.rows, W.rows), dtype=torch.float32, device=dev)
    if Y.dtype != torch.float32:
        raise TypeError("Y must be fp32")
    py, ldy = _dev2d(Y, "Y")
    a, w = ctypes.byref(A.c_struct()), ctypes.byref(W.c_struct())
    if ws is None:
        ws, p, n = _workspace(int(wsfn(a, w)), dev, None)
    else:
        p, n = ws.data_ptr(), ws.numel() * ws.element_size()
    _check(fn(a, w, py, ldy, p, n, _stream(dev)), name)
    return Y


def mxs_mixed_gemm(A: QMat, W: QMat, Y: torch.Tensor | None = None, ws=None) -> torch.Tensor:
    """Y [M, N] fp32 = Qa(X) Qw(W)^T with per-block MX scales."""
    return _gemm(_lib.mxs_mixed_gemm, _lib.mxs_mixed_gemm_workspace, "mxs_mixed_gemm", A, W, Y, ws)


# bytes of the device scratch array behind mxs_mixed_gemm_noalloc (per GPU)
NOALLOC_SCRATCH_BYTES = 48 << 20


def mxs_mixed_gemm_noalloc(A: QMat, W: QMat, Y: torch.Tensor) -> torch.Tensor:
    """mxs_mixed_gemm with its workspace in the library's per-GPU scratch
    array: the C call allocates nothing (Y is the caller's fp32 [M, N])."""
    if Y.dtype != torch.float32:
        raise TypeError("Y must be fp32")
    py, ldy = _dev2d(Y, "Y")
    a, w = ctypes.byref(A.c_struct()), ctypes.byref(W.c_struct())
    _check(_lib.mxs_mixed_gemm_noalloc(a, w, py, ldy, _stream(Y.device)), "mxs_mixed_gemm_noalloc")
    return Y


def mxs_mixed_gemm_fused_workspace(M: int, dtype: torch.dtype, W: QMat) -> int:
    dt = MXS_BF16 if dtype == torch.bfloat16 else MXS_F32
    return int(_lib.mxs_mixed_gemm_fused_workspace(M, dt, ctypes.byref(W.c_struct())))


def _fused_args(X: torch.Tensor, perm, W: QMat, Y):
    px, ldx = _dev2d(X, "X")
    M, K = X.shape
    if K != W.K:
        raise ValueError("X and W differ in K")
    if perm is not None and (perm.dtype != torch.int32 or not perm.is_contiguous() or perm.numel() != K
                             or not perm.is_cuda):
        raise ValueError("perm must be a contiguous int32 [K] GPU tensor")
    if Y is None:
        Y = torch.empty((M, W.rows), dtype=torch.float32, device=X.device)
    if Y.dtype != torch.float32:
        raise TypeError("Y must be fp32")
    py, ldy = _dev2d(Y, "Y")
    return px, ldx, M, Y, py, ldy


def mxs_mixed_gemm_fused(X: torch.Tensor, perm: torch.Tensor | None, W: QMat, Y: torch.Tensor | None = None,
                         ws=None) -> torch.Tensor:
    """Y [M, N] fp32 = mixed_gemm(quantize(X[:, perm] at W's block counts), W), X quantized inside the call."""
    px, ldx, M, Y, py, ldy = _fused_args(X, perm, W, Y)
    w = W.c_struct()
    dt = _dtype(X)
    if ws is None:
        ws, p, n = _workspace(int(_lib.mxs_mixed_gemm_fused_workspace(M, dt, ctypes.byref(w))), X.device, None)
    else:
        p, n = ws.data_ptr(), ws.numel() * ws.element_size()
    _check(_lib.mxs_mixed_gemm_fused(px, dt, M, ldx, _ptr(perm), ctypes.byref(w), py, ldy, p, n,
                                     _stream(X.device)), "mxs_mixed_gemm_fused")
    return Y


# ------------------------------------------------------------ prepared weights
def mxs_prepare_weights_size(W: QMat) -> int:
    return int(_lib.mxs_prepare_weights_size(ctypes.byref(W.c_struct())))


def mxs_prepare_weights(W: QMat, out: torch.Tensor | None = None) -> torch.Tensor:
    """W's prefill operand built once (uint8 device buffer, contents private
    to the library), for mxs_mixed_gemm_prepared / mxs_mixed_gemm_fused_prepared."""
    n = mxs_prepare_weights_size(W)
    if out is None:
        out = torch.empty(max(n, 1), dtype=torch.uint8, device=W.sc.device)
    if out.dtype != torch.uint8 or not out.is_cuda or not out.is_contiguous():
        raise ValueError("out must be a contiguous uint8 GPU tensor")
    _check(_lib.mxs_prepare_weights(ctypes.byref(W.c_struct()), out.data_ptr(), out.numel(),
                                    _stream(out.device)), "mxs_prepare_weights")
    return out


def mxs_mixed_gemm_prepared_workspace(A: QMat, W: QMat) -> int:
    return int(_lib.mxs_mixed_gemm_prepared_workspace(ctypes.byref(A.c_struct()), ctypes.byref(W.c_struct())))


def mxs_mixed_gemm_prepared(A: QMat, W: QMat, wprep: torch.Tensor, Y: torch.Tensor | None = None,
                            ws=None) -> torch.Tensor:
    """mxs_mixed_gemm with W's operand taken from mxs_prepare_weights(W)."""
    dev = A.sc.device
    if Y is None:
        Y = torch.empty((A.rows, W.rows), dtype=torch.float32, device=dev)
    if Y.dtype != torch.float32:
        raise TypeError("Y must be fp32")
    py, ldy = _dev2d(Y, "Y")
    a, w = ctypes.byref(A.c_struct()), ctypes.byref(W.c_struct())
    if ws is None:
        ws, p, n = _workspace(int(_lib.mxs_mixed_gemm_prepared_workspace(a, w)), dev, None)
    else:
        p, n = ws.data_ptr(), ws.numel() * ws.element_size()
    _check(_lib.mxs_mixed_gemm_prepared(a, w, wprep.data_ptr(), wprep.numel() * wprep.element_size(), py, ldy,
                                        p, n, _stream(dev)), "mxs_mixed_gemm_prepared")
    return Y


def mxs_mixed_gemm_fused_prepared_workspace(M: int, dtype: torch.dtype, W: QMat) -> int:
    dt = MXS_BF16 if dtype == torch.bfloat16 else MXS_F32
    return int(_lib.mxs_mixed_gemm_fused_prepared_workspace(M, dt, ctypes.byref(W.c_struct())))


def mxs_mixed_gemm_fused_prepared(X: torch.Tensor, perm: torch.Tensor | None, W: QMat, wprep: torch.Tensor,
                                  Y: torch.Tensor | None = None, ws=None) -> torch.Tensor:
    """mxs_mixed_gemm_fused with W's operand taken from mxs_prepare_weights(W)."""
    px, ldx, M, Y, py, ldy = _fused_args(X, perm, W, Y)
    w = W.c_struct()
    dt = _dtype(X)
    if ws is None:
        ws, p, n = _workspace(int(_lib.mxs_mixed_gemm_fused_prepared_workspace(M, dt, ctypes.byref(w))), X.device,
                              None)
    else:
        p, n = ws.data_ptr(), ws.numel() * ws.element_size()
    _check(_lib.mxs_mixed_gemm_fused_prepared(px, dt, M, ldx, _ptr(perm), ctypes.byref(w), wprep.data_ptr(),
                                              wprep.numel() * wprep.element_size(), py, ldy, p, n,
                                              _stream(X.device)), "mxs_mixed_gemm_fused_prepared")
    return Y


def mxs_mixed_gemm_mx_workspace(A: QMat, W: QMat) -> int:
    a, w = A.c_struct(), W.c_struct()
    return int(_lib.mxs_mixed_gemm_mx_workspace(ctypes.byref(a), ctypes.byref(w)))


def mxs_mixed_gemm_mx(A: QMat, W: QMat, Y: torch.Tensor | None = None, ws=None) -> torch.Tensor:
    """The same product, prefill on the block-scaled fp6 matrix cores."""
    return _gemm(_lib.mxs_mixed_gemm_mx, _lib.mxs_mixed_gemm_mx_workspace, "mxs_mixed_gemm_mx", A, W, Y, ws)


def mxs_quantize_kv(kv: torch.Tensor, codes=None, scales=None):
    """codes uint8 [T, H, D/2], scales uint8 [T, H, D/32] for kv [T, H, D]."""
    if not kv.is_cuda or kv.dim() != 3 or not kv.is_contiguous():
        raise ValueError("kv must be a contiguous [T, H, D] GPU tensor")
    T, H, D = kv.shape
    if codes is None:
        codes = torch.empty((T, H, D // 2), dtype=torch.uint8, device=kv.device)
    if scales is None:
        scales = torch.empty((T, H, D // 32), dtype=torch.uint8, device=kv.device)
    _check(_lib.mxs_quantize_kv(kv.data_ptr(), _dtype(kv), T, H, D, _ptr(codes), _ptr(scales),
                                _stream(kv.device)), "mxs_quantize_kv")
    return codes, scales


# ------------------------------------------------------------ layer-wise budget
def mxs_allocate_blocks(score: torch.Tensor, n8: int, n6: int, bits=None, perm=None):
    """mxs_allocate with the block counts given: (bits, perm)."""
    if not score.is_cuda or score.dtype != torch.float64 or not score.is_contiguous():
        raise ValueError("score must be a contiguous fp64 GPU tensor")
    K = score.numel()
    if bits is None:
        bits = torch.empty(K, dtype=torch.uint8, device=score.device)
    if perm is None:
        perm = torch.empty(K, dtype=torch.int32, device=score.device)
    _check(_lib.mxs_allocate_blocks(score.data_ptr(), K, n8, n6, bits.data_ptr(), perm.data_ptr(),
                                    _stream(score.device)), "mxs_allocate_blocks")
    return bits, perm


def mxs_output_error_workspace(M: int, N: int) -> int:
    return int(_lib.mxs_output_error_workspace(M, N))


def mxs_output_error(X: torch.Tensor, W: torch.Tensor, Yq: torch.Tensor, err=None, ws=None) -> torch.Tensor:
    """err (fp64 [1] on the GPU) = sum over (t, n) of (X W^T - Yq)^2."""
    px, ldx = _dev2d(X, "X")
    pw, ldw = _dev2d(W, "W")
    py, ldy = _dev2d(Yq, "Yq")
    if X.dtype != W.dtype:
        raise TypeError("X and W must have the same element type")
    if Yq.dtype != torch.float32:
        raise TypeError("Yq must be fp32")
    M, K = X.shape
    N = W.shape[0]
    if W.shape[1] != K or tuple(Yq.shape) != (M, N):
        raise ValueError("shapes do not match: X [M, K], W [N, K], Yq [M, N]")
    if err is None:
        err = torch.empty(1, dtype=torch.float64, device=X.device)
    ws, p, n = _workspace(mxs_output_error_workspace(M, N), X.device, ws)
    _check(_lib.mxs_output_error(px, pw, _dtype(X), M, N, K, ldx, ldw, py, ldy, err.data_ptr(), p, n,
                                 _stream(X.device)), "mxs_output_error")
    return err


def mxs_layer_budget(S, rows, K, B: float):
    """(blocks [L][3] as (n8, n6, n4) lists, R) for layer sensitivities S."""
    L = len(S)
    s_arr = (ctypes.c_double * L)(*[float(x) for x in S])
    r_arr = (c_int64 * L)(*[int(x) for x in rows])
    k_arr = (c_int64 * L)(*[int(x) for x in K])
    out = (c_int32 * (3 * L))()
    R = c_double(0.0)
    _check(_lib.mxs_layer_budget(L, ctypes.cast(s_arr, c_void_p), ctypes.cast(r_arr, c_void_p),
                                 ctypes.cast(k_arr, c_void_p), float(B), ctypes.cast(out, c_void_p),
                                 ctypes.byref(R)), "mxs_layer_budget")
    return [[out[3 * i], out[3 * i + 1], out[3 * i + 2]] for i in range(L)], R.value


# ------------------------------------------------------- attention over KV4
def mxs_attend_kv4_workspace(T: int, Hq: int, Hkv: int, D: int) -> int:
    return int(_lib.mxs_attend_kv4_workspace(T, Hq, Hkv, D))


def mxs_attend_kv4(q: torch.Tensor, k_cache, v_cache, scale: float, out=None, ws=None) -> torch.Tensor:
    """out [Hq, D] fp32: attention of one query token q [Hq, D] (fp32) over K/V
    caches given as (codes [T, Hkv, D/2], scales [T, Hkv, D/32]) from
    mxs_quantize_kv."""
    kc, ks = k_cache
    vc, vs = v_cache
    if not q.is_cuda or q.dtype != torch.float32 or q.dim() != 2 or not q.is_contiguous():
        raise ValueError("q must be a contiguous fp32 [Hq, D] GPU tensor")
    for t in (kc, ks, vc, vs):
        if not t.is_cuda or t.dtype != torch.uint8 or t.dim() != 3 or not t.is_contiguous():
            raise ValueError("caches must be contiguous uint8 [T, Hkv, ...] GPU tensors")
    Hq, D = q.shape
    T, Hkv = kc.shape[0], kc.shape[1]
    if tuple(kc.shape) != (T, Hkv, D // 2) or tuple(vc.shape) != (T, Hkv, D // 2) \
            or tuple(ks.shape) != (T, Hkv, D // 32) or tuple(vs.shape) != (T, Hkv, D // 32):
        raise ValueError("cache shapes do not match q")
    if out is None:
        out = torch.empty((Hq, D), dtype=torch.float32, device=q.device)
    ws, p, n = _workspace(mxs_attend_kv4_workspace(T, Hq, Hkv, D), q.device, ws)
    _check(_lib.mxs_attend_kv4(q.data_ptr(), kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), T, Hq,
                               Hkv, D, float(scale), out.data_ptr(), p, n, _stream(q.device)), "mxs_attend_kv4")
    return out


# ------------------------------------- serving on the 4-bit cache: rotary positions
ROPE_LAYOUTS = {"half": 0, "pairs": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "parts": 3}


def _int32(n: int, name: str) -> int:
    """n, which the C interface takes in 32 bits (a larger one would lose its upper half)."""
    if n > 0x7FFFFFFF:
        raise ValueError(f"{name} must be less than 2^31")
    return n


def mxs_rope_frequencies(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                         low: float = 1.0, high: float = 4.0, original_length: float = 8192.0,
                         device="cuda") -> torch.Tensor:
    """Radians per position of the rot / 2 rotated pairs, fp64, copied to `device`.

    scaling stretches them for long contexts: "linear" divides by factor, "ntk"
    raises the base, "parts" divides only the pairs that turn few times within
    original_length tokens (none above `high` turns, all below `low`)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
    out = torch.empty(max(_int32(int(rot), "rot") // 2, 1), dtype=torch.float64)
    _check(_lib.mxs_rope_frequencies(rot, base, ROPE_SCALINGS[scaling], factor, low, high, original_length,
                                     out.data_ptr()), "mxs_rope_frequencies")
    return out.to(device)


# The calls of a decode step are short, so their checks avoid what is slow in
# Python: device objects are compared by index, strides read once.
def _gpu(t: torch.Tensor, name: str) -> int:
    """Index of the GPU that holds t."""
    i = t.get_device()
    if i < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    return i


def _rows(t: torch.Tensor, name: str, gpu: int):
    """(pointer, token stride, head stride) of a [T, H, D] tensor on that GPU with adjacent dims."""
    if t.dim() != 3 or t.get_device() != gpu:
        raise ValueError(f"{name} must be a [T, H, D] tensor on cuda:{gpu}")
    s = t.stride()
    if s[2] != 1:
        raise ValueError(f"{name} must have unit stride in the last dimension")
    return t.data_ptr(), s[0], s[1]


def _vector(t: torch.Tensor, name: str, dtype, n: int, gpu: int) -> int:
    """Pointer of a contiguous [n] tensor of `dtype` on that GPU."""
    if t.dtype is not dtype or t.dim() != 1 or t.numel() != n or t.get_device() != gpu or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements on cuda:{gpu}")
    return t.data_ptr()


def _call(gpu: int, fn, name: str, *args):
    """The C call on the current stream of that GPU, with the GPU current (HIP launches there)."""
    if torch._C._cuda_getDevice() == gpu:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(gpu))
    else:
        with torch.cuda.device(gpu):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(gpu))
    if status:
        _check(status, name)


def _layout(layout: str) -> int:
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}")
    return ROPE_LAYOUTS[layout]


def mxs_rope(x: torch.Tensor, positions: torch.Tensor, freq: torch.Tensor, layout: str = "half", mscale: float = 1.0,
             out: torch.Tensor | None = None) -> torch.Tensor:
    """x [T, H, D] (bf16 or fp32, any token and head strides) with the first
    2 * len(freq) dims of every head turned by positions [T] (int64) times freq
    (fp64, from mxs_rope_frequencies). out may be x. The gradient with respect
    to x is the same call on the output's gradient at -positions."""
    gpu = _gpu(x, "x")
    px, xt, xh = _rows(x, "x", gpu)
    T, H, D = x.shape
    if out is None:
        out = torch.empty((T, H, D), dtype=x.dtype, device=x.device)
    elif out.shape != x.shape or out.dtype is not x.dtype:
        raise ValueError("out must have x's shape and type")
    py, yt, yh = _rows(out, "out", gpu)
    n = freq.numel()
    _call(gpu, _lib.mxs_rope, "mxs_rope", px, _dtype(x), T, H, D, xt, xh,
          _vector(positions, "positions", torch.int64, T, gpu), _vector(freq, "freq", torch.float64, n, gpu),
          _int32(2 * n, "2 * len(freq)"), _layout(layout), mscale, py, yt, yh)
    return out


# ------------------------------------------------------- paged 4-bit K/V cache
@dataclass(frozen=True)
class KV4Cache:
    """A pool of pages of 4-bit keys and values (see mxs_kv4_cache): codes kc,
    vc uint8 [pages, page_size, H, D / 2], E8M0 bytes ks, vs uint8 [pages,
    page_size, H, D / 32], contiguous. Slot = page * page_size + offset.
    Frozen: checked and its C struct built once."""
    kc: torch.Tensor
    ks: torch.Tensor
    vc: torch.Tensor
    vs: torch.Tensor

    def __post_init__(self):
        if self.kc.dim() != 4 or not self.kc.is_cuda:
            raise ValueError("kc must be a [pages, page_size, H, D / 2] GPU tensor")
        P, S, H, h = self.kc.shape
        for t, w in ((self.kc, h), (self.ks, h // 16), (self.vc, h), (self.vs, h // 16)):
            if t.dtype != torch.uint8 or tuple(t.shape) != (P, S, H, w) or not t.is_contiguous() \
                    or t.device != self.kc.device:
                raise ValueError("cache planes must be contiguous uint8 [pages, page_size, H, D / 2] codes and "
                                 "[pages, page_size, H, D / 32] scales on one GPU")
        c = _Kv4Cache(P, _int32(S, "page_size"), _int32(H, "H"), _int32(2 * h, "D"), 0, self.kc.data_ptr(),
                      self.ks.data_ptr(), self.vc.data_ptr(), self.vs.data_ptr())
        for k, v in (("_c", c), ("_ref", ctypes.pointer(c)), ("gpu", self.kc.get_device()), ("page_size", S),
                     ("H", H), ("D", 2 * h)):
            object.__setattr__(self, k, v)


def kv4_cache_alloc(pages: int, page_size: int, H: int, D: int, device="cuda") -> KV4Cache:
    """An empty pool (contents undefined until written)."""
    if D < 32 or D % 32:
        raise ValueError("D must be a positive multiple of 32")
    kw = dict(dtype=torch.uint8, device=device)
    return KV4Cache(*(torch.empty((pages, page_size, H, D // w), **kw) for w in (2, 32, 2, 32)))


def _kv_rows(cache: KV4Cache, t: torch.Tensor, name: str, T: int, dtype):
    if t.dtype is not dtype or t.shape != (T, cache.H, cache.D):
        raise ValueError(f"{name} must be a {dtype} [{T}, {cache.H}, {cache.D}] tensor")
    return _rows(t, name, cache.gpu)


def mxs_kv4_append(cache: KV4Cache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                   positions: torch.Tensor | None = None, freq: torch.Tensor | None = None, layout: str = "half",
                   mscale: float = 1.0) -> None:
    """Quantises k, v [T, H, D] into the cache at slots [T] (int64, distinct;
    negative or past the pool: skipped). With positions and freq, the keys are
    rotated first, as by mxs_rope but without rounding in between."""
    gpu, T = cache.gpu, slots.numel()
    pk, kt, kh = _kv_rows(cache, k, "k", T, k.dtype)
    pv, vt, vh = _kv_rows(cache, v, "v", T, k.dtype)
    if (positions is None) != (freq is None):
        raise ValueError("positions and freq go together")
    n, pp, pf = 0, None, None
    if positions is not None:
        n = freq.numel()
        pp, pf = _vector(positions, "positions", torch.int64, T, gpu), _vector(freq, "freq", torch.float64, n, gpu)
    _call(gpu, _lib.mxs_kv4_append, "mxs_kv4_append", cache._ref, pk, pv, _dtype(k), T, kt, kh, vt, vh,
          _vector(slots, "slots", torch.int64, T, gpu), pp, pf, _int32(2 * n, "2 * len(freq)"), _layout(layout), mscale)


def mxs_kv4_read(cache: KV4Cache, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                 k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None, keys: bool = True,
                 values: bool = True):
    """(k, v), each [T, H, D]: the values of slots [T] (int64), exact. Rows of
    slots that are negative or past the pool are left as they were (zero in
    outputs that the call allocates). dtype is that of outputs not given. keys
    or values False: that one is not read, and None is returned for it."""
    gpu, T = cache.gpu, slots.numel()
    if not (keys or values) or (k_out is not None and not keys) or (v_out is not None and not values):
        raise ValueError("keys, values or both are read, and no output is given for what is not")
    if k_out is not None or v_out is not None:
        dtype = (k_out if k_out is not None else v_out).dtype
    if keys and k_out is None:
        k_out = torch.zeros((T, cache.H, cache.D), dtype=dtype, device=cache.kc.device)
    if values and v_out is None:
        v_out = torch.zeros((T, cache.H, cache.D), dtype=dtype, device=cache.kc.device)
    pk, kt, kh = _kv_rows(cache, k_out, "k_out", T, dtype) if keys else (None, 0, 0)
    pv, vt, vh = _kv_rows(cache, v_out, "v_out", T, dtype) if values else (None, 0, 0)
    _call(gpu, _lib.mxs_kv4_read, "mxs_kv4_read", cache._ref, _vector(slots, "slots", torch.int64, T, gpu), T,
          _dtype(k_out if keys else v_out), pk, kt, kh, pv, vt, vh)
    return k_out, v_out


# ------------------------------------------------------------ pages of the cache
def _table(cache: KV4Cache, table: torch.Tensor):
    """(pointer, width, rows) of a page table."""
    if table.dtype is not torch.int32 or table.dim() != 2 or table.get_device() != cache.gpu \
            or not table.is_contiguous():
        raise ValueError(f"table must be a contiguous int32 [B, pages] tensor on cuda:{cache.gpu}")
    B, width = table.shape
    return table.data_ptr(), width, B


def _given_ws(ws, gpu: int, dev, query, *args):
    """(tensor, pointer, bytes) of a workspace, allocated if the caller passes none."""
    if ws is None:
        return _workspace(int(query(*args)), dev, None)
    if ws.get_device() != gpu or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on cuda:{gpu}")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def mxs_kv4_copy(dst: KV4Cache, dst_slots: torch.Tensor, src: KV4Cache, src_slots: torch.Tensor) -> None:
    """Copies the tokens of src_slots [T] in one pool to dst_slots [T] in another
    or the same (int64; pairs with a negative or too large slot are skipped).
    Destinations are distinct and, in one pool, no token's source."""
    gpu, T = dst.gpu, src_slots.numel()
    if src.gpu != gpu:
        raise ValueError("both pools must be on one GPU")
    _call(gpu, _lib.mxs_kv4_copy, "mxs_kv4_copy", dst._ref, _vector(dst_slots, "dst_slots", torch.int64, T, gpu),
          src._ref, _vector(src_slots, "src_slots", torch.int64, T, gpu), T)


def mxs_kv4_fork(cache: KV4Cache, refs: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, src: torch.Tensor,
                 dst: torch.Tensor) -> None:
    """Row dst[i] of the page table becomes a fork of row src[i]: the same pages
    for its tokens (refs [pages] counts them), the same length. The rows dst
    hold no pages before. table [B, pages], lens [B], src and dst [n] int32."""
    gpu, n = cache.gpu, src.numel()
    pt, width, B = _table(cache, table)
    _call(gpu, _lib.mxs_kv4_fork, "mxs_kv4_fork", cache._ref,
          _vector(refs, "refs", torch.int32, cache.kc.shape[0], gpu), pt, width, B,
          _vector(lens, "lens", torch.int32, B, gpu), _vector(src, "src", torch.int32, n, gpu),
          _vector(dst, "dst", torch.int32, n, gpu), n)


def mxs_kv4_reserve_workspace(pages: int, B: int) -> int:
    return int(_lib.mxs_kv4_reserve_workspace(pages, B))


def mxs_kv4_reserve(cache: KV4Cache, refs: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, cu: torch.Tensor,
                    total: int | None = None, slots: torch.Tensor | None = None, lens_out: torch.Tensor | None = None,
                    ws=None):
    """(slots [total] int64, lens_out [B] int32): room for cu[b + 1] - cu[b] tokens
    behind the lens[b] of every sequence, in the lowest free pages (refs 0) where
    its row of the table has none or shares one (whose tokens are copied first).
    slots are those of the new tokens, -1 where the pool or the row has no room
    (that sequence is left as it was). total: the rows of slots, needed where the
    call allocates them. lens_out may be lens."""
    gpu, dev = cache.gpu, cache.kc.device
    pt, width, B = _table(cache, table)
    pages = cache.kc.shape[0]
    if slots is None:
        if total is None:
            raise ValueError("total or slots must be given")
        slots = torch.full((total,), -1, dtype=torch.int64, device=dev)
    elif total is not None and total != slots.numel():
        raise ValueError("slots must have total elements")
    n = slots.numel()
    if lens_out is None:
        lens_out = torch.empty(B, dtype=torch.int32, device=dev)
    ws, p, nbytes = _given_ws(ws, gpu, dev, _lib.mxs_kv4_reserve_workspace, pages, B)
    _call(gpu, _lib.mxs_kv4_reserve, "mxs_kv4_reserve", cache._ref, _vector(refs, "refs", torch.int32, pages, gpu), pt,
          width, B, _vector(lens, "lens", torch.int32, B, gpu), _vector(cu, "cu", torch.int32, B + 1, gpu), n,
          _vector(slots, "slots", torch.int64, n, gpu), _vector(lens_out, "lens_out", torch.int32, B, gpu), p, nbytes)
    return slots, lens_out


def _compact(cache: KV4Cache, table, lens, cu, path, count, lens_out):
    """(lens_out, arguments before and behind the slots) of a compaction."""
    gpu, total = cache.gpu, path.numel()
    pt, width, B = _table(cache, table)
    if lens_out is None:
        lens_out = torch.empty(B, dtype=torch.int32, device=cache.kc.device)
    return lens_out, (cache._ref, pt, width, B, _vector(lens, "lens", torch.int32, B, gpu),
                      _vector(cu, "cu", torch.int32, B + 1, gpu), _vector(path, "path", torch.int32, total, gpu),
                      _vector(count, "count", torch.int32, B, gpu)), \
        (total, _vector(lens_out, "lens_out", torch.int32, B, gpu))


def mxs_kv4_compact(cache: KV4Cache, table: torch.Tensor, lens: torch.Tensor, cu: torch.Tensor, path: torch.Tensor,
                    count: torch.Tensor, lens_out: torch.Tensor | None = None) -> torch.Tensor:
    """lens_out [B]: of the last cu[b + 1] - cu[b] tokens of every sequence, those
    numbered path[cu[b]] .. path[cu[b] + count[b] - 1] (ascending) are moved together
    behind the others, and the length ends there. path and count as
    mxs_verify_tree returns them. lens_out may be lens. For steps in which every
    sequence was granted its room; otherwise mxs_kv4_compact_granted."""
    lens_out, front, back = _compact(cache, table, lens, cu, path, count, lens_out)
    _call(cache.gpu, _lib.mxs_kv4_compact, "mxs_kv4_compact", *front, *back)
    return lens_out


def mxs_kv4_compact_granted(cache: KV4Cache, table: torch.Tensor, lens: torch.Tensor, cu: torch.Tensor,
                            path: torch.Tensor, count: torch.Tensor, slots: torch.Tensor,
                            lens_out: torch.Tensor | None = None) -> torch.Tensor:
    """As mxs_kv4_compact, with the slots [total] that mxs_kv4_reserve left for this
    cu: a sequence that it refused (a first slot of -1) has none of its new tokens
    in the cache and is left as it is, its length with it. total is path's."""
    lens_out, front, back = _compact(cache, table, lens, cu, path, count, lens_out)
    _call(cache.gpu, _lib.mxs_kv4_compact_granted, "mxs_kv4_compact_granted", *front,
          _vector(slots, "slots", torch.int64, path.numel(), cache.gpu), *back)
    return lens_out


def mxs_kv4_release(cache: KV4Cache, refs: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, keep: torch.Tensor,
                    lens_out: torch.Tensor | None = None) -> torch.Tensor:
    """lens_out [B] = min(lens, keep): the pages behind the first keep[b] tokens of
    every sequence are given back (0 frees it, a negative keep leaves it as it
    is). lens_out may be lens."""
    gpu = cache.gpu
    pt, width, B = _table(cache, table)
    if lens_out is None:
        lens_out = torch.empty(B, dtype=torch.int32, device=cache.kc.device)
    _call(gpu, _lib.mxs_kv4_release, "mxs_kv4_release", cache._ref,
          _vector(refs, "refs", torch.int32, cache.kc.shape[0], gpu), pt, width, B,
          _vector(lens, "lens", torch.int32, B, gpu), _vector(keep, "keep", torch.int32, B, gpu),
          _vector(lens_out, "lens_out", torch.int32, B, gpu))
    return lens_out


# ------------------------------------------- attention of drafted tokens over it
def mxs_attend_kv4_tree_workspace(dtype: torch.dtype, B: int, total_q: int, max_q: int, max_len: int, Hq: int,
                                  Hkv: int, D: int) -> int:
    dt = MXS_BF16 if dtype == torch.bfloat16 else MXS_F32
    return int(_lib.mxs_attend_kv4_tree_workspace(dt, B, total_q, max_q, max_len, Hq, Hkv, D))


def mxs_attend_kv4_tree(q: torch.Tensor, cache: KV4Cache, table: torch.Tensor, lens: torch.Tensor, cu: torch.Tensor,
                        scale: float, mask: torch.Tensor | None = None, max_q: int | None = None,
                        max_len: int | None = None, out: torch.Tensor | None = None, ws=None) -> torch.Tensor:
    """out [total_q, Hq, D]: attention of the query tokens q (bf16 or fp32) of B
    sequences over the cache. Sequence b has lens[b] cached tokens in the pages
    table[b]; its query rows cu[b] .. cu[b + 1] - 1 are the last of them. mask
    [total_q, words] int64 holds, for every row, the bits of the drafted tokens
    it sees (None: those up to itself). table [B, pages], lens [B] and cu
    [B + 1] are int32. max_q and max_len bound the query and cached tokens of a
    sequence (default: total_q and what the table can hold). max_q chooses the
    kernel: plain decode of a batch should pass max_q=1 (with the default, 32
    sequences take more than twice the time). Rows of no sequence are left as
    they were in `out` (zero in an output that the call allocates)."""
    gpu = _gpu(q, "q")
    pq, qt, qh = _rows(q, "q", gpu)
    total, Hq, D = q.shape
    if out is None:
        out = torch.zeros((total, Hq, D), dtype=q.dtype, device=q.device)
    elif out.shape != q.shape or out.dtype is not q.dtype:
        raise ValueError("out must have q's shape and type")
    po, ot, oh = _rows(out, "out", gpu)
    if (qh != D or oh != D) and Hq > 1:
        raise ValueError("the heads of q and of out must be adjacent")
    if cache.D != D or cache.gpu != gpu:
        raise ValueError("q and the cache must have one head dimension and one device")
    if table.dtype is not torch.int32 or table.dim() != 2 or table.get_device() != gpu or not table.is_contiguous():
        raise ValueError(f"table must be a contiguous int32 [B, pages] tensor on cuda:{gpu}")
    B, width = table.shape
    pm, words = None, 0
    if mask is not None:
        if mask.dtype is not torch.int64 or mask.dim() != 2 or mask.shape[0] != total or mask.get_device() != gpu \
                or not mask.is_contiguous():
            raise ValueError(f"mask must be a contiguous int64 [total_q, words] tensor on cuda:{gpu}")
        pm, words = mask.data_ptr(), mask.shape[1]
    if max_q is None:
        max_q = total
    if max_len is None:
        max_len = width * cache.page_size
    dt = _dtype(q)
    if ws is None:
        ws, p, n = _workspace(int(_lib.mxs_attend_kv4_tree_workspace(dt, B, total, max_q, max_len, Hq, cache.H, D)),
                              q.device, None)
    else:
        if ws.get_device() != gpu or not ws.is_contiguous():
            raise ValueError(f"ws must be a contiguous tensor on cuda:{gpu}")
        p, n = ws.data_ptr(), ws.numel() * ws.element_size()
    _call(gpu, _lib.mxs_attend_kv4_tree, "mxs_attend_kv4_tree", pq, dt, qt, cache._ref, table.data_ptr(), width,
          _vector(lens, "lens", torch.int32, B, gpu), _vector(cu, "cu", torch.int32, B + 1, gpu), pm, words, B, total,
          max_q, max_len, Hq, scale, po, ot, p, n)
    return out


# ------------------------------------------------- verification of drafted tokens
def mxs_verify_tree_workspace(B: int, total: int, max_n: int, V: int) -> int:
    return int(_lib.mxs_verify_tree_workspace(B, total, max_n, V))


def _matrix(t: torch.Tensor, name: str, rows: int, cols: int, gpu: int):
    """(pointer, row stride) of a [rows, cols] tensor on that GPU with adjacent columns."""
    if t.dim() != 2 or t.shape != (rows, cols) or t.get_device() != gpu or (cols > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a [{rows}, {cols}] tensor on cuda:{gpu} with unit column stride")
    return t.data_ptr(), t.stride(0)


def mxs_verify_tree(logits: torch.Tensor, tokens: torch.Tensor, cu: torch.Tensor, uniform: torch.Tensor,
                    parents: torch.Tensor | None = None, draft: torch.Tensor | None = None, replacement: bool = False,
                    temperature: torch.Tensor | None = None, max_n: int | None = None,
                    path: torch.Tensor | None = None, count: torch.Tensor | None = None,
                    next_token: torch.Tensor | None = None, ws=None):
    """(path int32 [total], count int32 [B], next_token int64 [B]): drafted tokens
    accepted or rejected against the target's logits [total, V] (bf16 or fp32), so
    that every token is distributed as the target alone would draw it.

    Rows cu[b] .. cu[b + 1] - 1 (cu int32 [B + 1]) are the nodes of sequence b: its
    last token, then the drafted ones, tokens [total] (int64) below parents [total]
    (int32, counted within the sequence; None: a chain). draft [total, V] (fp32):
    row i is the distribution from which the children of node i were drawn, without
    replacement unless `replacement` is set; None: they were proposed without one.
    temperature [B] (fp32; 0: greedy; None: 1). uniform [total] (fp64, in [0, 1)):
    the number that decides on each node; the root's draws the next token. max_n
    bounds a sequence's nodes (default: total, and at most 1024).
    path holds the kept nodes of each sequence, the root first, then -1; count
    their number; next_token what follows the last of them."""
    gpu = _gpu(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be a [total, V] tensor")
    total, V = logits.shape
    pl, ldl = _matrix(logits, "logits", total, V, gpu)
    dt, dev, B = _dtype(logits), logits.device, cu.numel() - 1
    if B < 0:
        raise ValueError("cu must have B + 1 elements")
    pd, ldd = None, 0
    if draft is not None:
        if draft.dtype is not torch.float32:
            raise TypeError("draft must be fp32")
        pd, ldd = _matrix(draft, "draft", total, V, gpu)
    if max_n is None:
        max_n = min(total, 1024)
    if path is None:
        path = torch.full((total,), -1, dtype=torch.int32, device=dev)
    if count is None:
        count = torch.empty(B, dtype=torch.int32, device=dev)
    if next_token is None:
        next_token = torch.empty(B, dtype=torch.int64, device=dev)
    ws, p, n = _given_ws(ws, gpu, dev, _lib.mxs_verify_tree_workspace, B, total, max_n, V)
    _call(gpu, _lib.mxs_verify_tree, "mxs_verify_tree", pl, dt, ldl, V,
          _vector(tokens, "tokens", torch.int64, total, gpu),
          None if parents is None else _vector(parents, "parents", torch.int32, total, gpu),
          _vector(cu, "cu", torch.int32, B + 1, gpu), B, total, max_n, pd, ldd, int(bool(replacement)),
          None if temperature is None else _vector(temperature, "temperature", torch.float32, B, gpu),
          _vector(uniform, "uniform", torch.float64, total, gpu), _vector(path, "path", torch.int32, total, gpu),
          _vector(count, "count", torch.int32, B, gpu), _vector(next_token, "next_token", torch.int64, B, gpu), p, n)
    return path, count, next_token


# ------------------------------------------- adapters beside a shared projection
@dataclass(frozen=True)
class LoraSet:
    """Low-rank adapters of one linear layer (see mxs_lora): A [n, R, K] and B
    [n, N, R] (bf16 or fp32), scale fp32 [n] (None: 1), rank int32 [n] (None: R),
    contiguous, on one GPU. Frozen: checked and its C struct built once."""
    A: torch.Tensor
    B: torch.Tensor
    scale: torch.Tensor | None = None
    rank: torch.Tensor | None = None

    def __post_init__(self):
        A, B = self.A, self.B
        gpu = _gpu(A, "A")
        if A.dim() != 3 or B.dim() != 3 or B.dtype is not A.dtype or B.get_device() != gpu \
                or not A.is_contiguous() or not B.is_contiguous():
            raise ValueError("A [n, R, K] and B [n, N, R] must be contiguous tensors of one type on one GPU")
        n, R, K = A.shape
        N = B.shape[1]
        if B.shape[0] != n or B.shape[2] != R:
            raise ValueError("A [n, R, K] and B [n, N, R] do not match")
        c = _Lora(K, N, _int32(n, "n"), _int32(R, "R"), _dtype(A), 0, _ptr(A), _ptr(B),
                  None if self.scale is None else _vector(self.scale, "scale", torch.float32, n, gpu),
                  None if self.rank is None else _vector(self.rank, "rank", torch.int32, n, gpu))
        for k, v in (("_c", c), ("_ref", ctypes.pointer(c)), ("gpu", gpu), ("K", K), ("N", N)):
            object.__setattr__(self, k, v)


def mxs_lora_add_workspace(M: int, adapters: LoraSet) -> int:
    return int(_lib.mxs_lora_add_workspace(M, adapters._ref))


def mxs_lora_add(Y: torch.Tensor, X: torch.Tensor, ids: torch.Tensor, adapters: LoraSet, ws=None) -> torch.Tensor:
    """Y[t] += scale[a] B[a] (A[a] X[t]) with a = ids[t] (int32 [M]; outside the
    set: the row is left as it was). X [M, K] of the adapters' type, Y [M, N] fp32,
    as mxs_mixed_gemm writes it. Returns Y."""
    gpu = adapters.gpu
    M = ids.numel()
    if X.dtype is not adapters.A.dtype or Y.dtype is not torch.float32:
        raise TypeError("X must have the adapters' type, and Y must be fp32")
    px, ldx = _matrix(X, "X", M, adapters.K, gpu)
    py, ldy = _matrix(Y, "Y", M, adapters.N, gpu)
    ws, p, n = _given_ws(ws, gpu, Y.device, _lib.mxs_lora_add_workspace, M, adapters._ref)
    _call(gpu, _lib.mxs_lora_add, "mxs_lora_add", px, M, ldx, _vector(ids, "ids", torch.int32, M, gpu), adapters._ref, py,
          ldy, p, n)
    return Y
