"""ctypes binding of libsignmuon.so (argument marshalling only).

Every step of the Sign-Muon path runs in the HIP library; this module turns
torch tensors (device memory) and the current torch stream into the plain
pointers and sizes of the C ABI declared in ``include/signmuon.h``, and
raises ``SignMuonError`` on a non-zero status.  There is no fallback: if the
library is missing, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import os
from typing import Optional, Sequence, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
# SIGNMUON_LIB may name another build of the same library (e.g. a tuning
# variant); the default is the in-tree build.
LIB_PATH = os.environ.get("SIGNMUON_LIB") or os.path.join(_HERE, "libsignmuon.so")

SM_OK, SM_EINVAL, SM_EWORKSPACE, SM_EHIP, SM_ENONFINITE, SM_ERANGE, SM_EUNSUPPORTED = \
    0, -1, -2, -3, -4, -5, -6
SM_F32, SM_BF16 = 0, 1
NS_F32, NS_BF16, NS_BF16X3 = 0, 1, 2
SCALE_FRO, SCALE_SPECTRAL = 0, 1
SIGNS_PACKED, SIGNS_TERNARY = 0, 1
ACTIVATIONS = {"silu": 0, "gelu": 1}
REDUCTIONS = {"none": 0, "sum": 1, "mean": 2}
MAX_WORKERS = 32767
_NO_SIZE = ctypes.c_size_t(-1).value    # a workspace query refused its arguments

EXPORTS = (
    "signmuon_strerror", "signmuon_abi_version", "signmuon_momentum",
    "signmuon_polar_ns_workspace", "signmuon_polar_ns", "signmuon_sign_pack",
    "signmuon_majority_vote", "signmuon_apply", "signmuon_step_workspace",
    "signmuon_step", "signmuon_step_profiled", "signmuon_get_status",
    "signmuon_worker_pipeline", "signmuon_sign_ternary", "signmuon_majority_vote_ternary",
    "signmuon_executor_create", "signmuon_executor_destroy", "signmuon_reset_status",
    "signmuon_polar_ns_static",
)
# include/signmuon_layers.h
LAYER_EXPORTS = (
    "signmuon_layer_norm", "signmuon_layer_norm_backward",
    "signmuon_layer_norm_backward_workspace", "signmuon_embedding",
    "signmuon_embedding_backward", "signmuon_embedding_backward_workspace",
    "signmuon_linear_cross_entropy", "signmuon_linear_cross_entropy_backward",
    "signmuon_linear_cross_entropy_workspace", "signmuon_rms_norm", "signmuon_rms_norm_e4m3",
    "signmuon_rms_norm_backward", "signmuon_rms_norm_backward_workspace", "signmuon_gated_mlp",
    "signmuon_gated_mlp_backward", "signmuon_gated_mlp_workspace",
)
PHASES = {0: "start", 1: "momentum", 2: "prescale", 3: "gemm", 4: "pack", 5: "vote",
          6: "gram", 7: "square", 8: "update", 9: "gap"}


class SignMuonError(RuntimeError):
    def __init__(self, func: str, status: int, msg: str):
        super().__init__(f"{func}: {msg} (status {status})")
        self.status = status


class SmHparams(ctypes.Structure):
    _fields_ = [("eta", ctypes.c_float), ("beta", ctypes.c_float),
                ("lambda_", ctypes.c_float), ("eps", ctypes.c_float),
                ("K", ctypes.c_int32), ("scale", ctypes.c_int32),
                ("P", ctypes.c_int32), ("ns_a", ctypes.c_float),
                ("ns_b", ctypes.c_float), ("ns_c", ctypes.c_float),
                ("ns_precision", ctypes.c_int32), ("tie_value", ctypes.c_int32),
                ("sign_encoding", ctypes.c_int32)]


class SmProfile(ctypes.Structure):
    _fields_ = [("events", ctypes.POINTER(ctypes.c_void_p)),
                ("kinds", ctypes.POINTER(ctypes.c_int32)),
                ("capacity", ctypes.c_int32), ("count", ctypes.c_int32)]


class SmMatrix(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("elem_off", ctypes.c_int64), ("word_off", ctypes.c_int64)]


@dataclasses.dataclass
class HParams:
    eta: float = 0.02
    beta: float = 0.9
    lam: float = 0.01
    eps: float = 1e-7
    K: int = 5
    scale: str = "fro"              # "fro" | "spectral"
    P: int = 0
    coeffs: Tuple[float, float, float] = (1.5, -0.5, 0.0)
    precision: str = "bf16"         # "f32" | "bf16" | "bf16x3"
    tie_value: int = 0
    encoding: str = "packed"        # worker sign buffers: "packed" | "ternary"

    def to_c(self) -> SmHparams:
        prec = {"f32": NS_F32, "bf16": NS_BF16, "bf16x3": NS_BF16X3}[self.precision]
        scale = {"fro": SCALE_FRO, "spectral": SCALE_SPECTRAL}[self.scale]
        enc = {"packed": SIGNS_PACKED, "ternary": SIGNS_TERNARY}[self.encoding]
        a, b, c = self.coeffs
        return SmHparams(self.eta, self.beta, self.lam, self.eps, int(self.K), scale,
                         int(self.P), a, b, c, prec, int(self.tie_value), enc)


_LIB = None


def lib():
    """Load libsignmuon.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m distributed_bit_matrix_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                 ctypes.c_float, ctypes.c_size_t)
        hp = ctypes.POINTER(SmHparams)
        mats = ctypes.POINTER(SmMatrix)
        sig = {
            "signmuon_strerror": (ctypes.c_char_p, [ctypes.c_int]),
            "signmuon_abi_version": (i32, []),
            "signmuon_momentum": (i32, [vp, vp, i32, vp, i64, f32, f32, vp]),
            "signmuon_polar_ns_workspace": (sz, [i64, i64, hp]),
            "signmuon_polar_ns": (i32, [vp, vp, i64, i64, hp, vp, vp, sz, vp]),
            "signmuon_polar_ns_static": (i32, [vp, vp, i64, i64, hp, vp, vp]),
            "signmuon_sign_pack": (i32, [vp, vp, i64, vp]),
            "signmuon_majority_vote": (i32, [vp, i64, i32, i64, i32, vp, vp, vp]),
            "signmuon_sign_ternary": (i32, [vp, vp, i64, vp]),
            "signmuon_majority_vote_ternary": (i32, [vp, i64, i32, i64, i32, vp, vp, vp]),
            "signmuon_apply": (i32, [vp, i32, vp, vp, f32, i64, vp]),
            "signmuon_step_workspace": (sz, [mats, i32, hp, i32]),
            "signmuon_step": (i32, [mats, i32, hp, vp, vp, i32, vp, vp, i64, i32,
                                    i32, i32, vp, vp, sz, vp, vp]),
            "signmuon_worker_pipeline": (i32, [mats, i32, hp, vp, vp, i32, vp, vp, i64,
                                               i32, i32, i32, vp, vp, sz, vp, vp]),
            "signmuon_step_profiled": (i32, [mats, i32, hp, vp, vp, i32, vp, vp, i64,
                                             i32, i32, i32, vp, vp, sz,
                                             ctypes.POINTER(SmProfile), vp, vp]),
            "signmuon_get_status": (i32, [vp, vp]),
            "signmuon_executor_create": (i32, [ctypes.POINTER(vp)]),
            "signmuon_executor_destroy": (i32, [vp]),
            "signmuon_reset_status": (i32, [vp, vp]),
            "signmuon_layer_norm": (i32, [vp, i32, i64, vp, vp, i32, i64, i64, f32, vp, vp, vp,
                                          vp]),
            "signmuon_layer_norm_backward_workspace": (sz, [i64, i64]),
            "signmuon_layer_norm_backward": (i32, [vp, i64, vp, i32, i64, vp, i32, vp, vp, i64,
                                                   i64, vp, vp, vp, i32, i32, vp, sz, vp]),
            "signmuon_embedding": (i32, [vp, i32, i64, i64, vp, i32, i64, f32, vp, i32, vp]),
            "signmuon_embedding_backward_workspace": (sz, [i64, i64, i64]),
            "signmuon_embedding_backward": (i32, [vp, i32, i64, vp, i32, i64, i64, f32, vp, i32,
                                                  i64, i64, i32, vp, sz, vp]),
        }
        sig.update({
            "signmuon_linear_cross_entropy_workspace": (sz, [i64, i64, i64, i32, i32]),
            "signmuon_linear_cross_entropy": (i32, [vp, i64, vp, i32, vp, i32, i64, i64, i64, i64,
                                                    i32, vp, vp, vp, sz, vp]),
            "signmuon_linear_cross_entropy_backward": (i32, [vp, vp, i64, vp, i32, vp, i32, vp,
                                                             i64, i64, i64, i64, i32, vp, vp, i32,
                                                             i32, vp, sz, vp]),
            "signmuon_rms_norm": (i32, [vp, i64, vp, i64, i32, vp, i32, i64, i64, f32, vp, vp, vp,
                                        vp]),
            "signmuon_rms_norm_e4m3": (i32, [vp, i64, vp, i64, i32, vp, i32, i64, i64, f32, i64,
                                             vp, vp, vp, vp, vp]),
            "signmuon_rms_norm_backward_workspace": (sz, [i64, i64]),
            "signmuon_rms_norm_backward": (i32, [vp, i64, vp, i64, vp, i64, i32, vp, i32, vp, i64,
                                                 i64, vp, vp, i32, i32, vp, sz, vp]),
            "signmuon_gated_mlp_workspace": (sz, [i64, i64, i64, i32, i32]),
            "signmuon_gated_mlp": (i32, [vp, i64, vp, vp, vp, i32, i32, i64, i64, i64, vp, vp, vp,
                                         sz, vp]),
            "signmuon_gated_mlp_backward": (i32, [vp, i64, vp, i64, vp, vp, vp, vp, i32, i32, i64,
                                                  i64, i64, vp, vp, vp, vp, i32, i32, vp, sz,
                                                  vp]),
        })
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


def strerror(status: int) -> str:
    return lib().signmuon_strerror(int(status)).decode()


def _check(func: str, status: int):
    if status != SM_OK:
        raise SignMuonError(func, status, strerror(status))


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _wdtype(W) -> int:
    import torch
    if W.dtype == torch.float32:
        return SM_F32
    if W.dtype == torch.bfloat16:
        return SM_BF16
    raise TypeError("W must be float32 or bfloat16")


def _require(t, dtype, name):
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} CUDA tensor")


def mats_array(mats: Sequence[Tuple[int, int, int, int]]):
    arr = (SmMatrix * len(mats))()
    for i, (r, c, eo, wo) in enumerate(mats):
        arr[i] = SmMatrix(r, c, eo, wo)
    return arr


def default_layout(shapes: Sequence[Tuple[int, int]]):
    """Back-to-back layout: (rows, cols, elem_off, word_off) per matrix, the
    entry count d and the packed words per worker (int8 sign buffers take d
    bytes per worker, each matrix at its elem_off)."""
    out, eo, wo = [], 0, 0
    for r, c in shapes:
        out.append((r, c, eo, wo))
        eo += r * c
        wo += (r * c + 31) // 32
    return out, eo, wo


# ---------------------------------------------------------------------------
# Entry points
# ---------------------------------------------------------------------------
def momentum(G, W, Mom, beta: float, lam: float, stream=None):
    import torch
    _require(G, torch.float32, "G")
    _require(Mom, torch.float32, "Mom")
    n = Mom.numel()
    if G.numel() != n or W.numel() != n:
        raise ValueError("G, W and Mom must have the same size")
    _check("signmuon_momentum", lib().signmuon_momentum(
        _ptr(G), _ptr(W), _wdtype(W), _ptr(Mom), n, beta, lam, _stream(stream)))


def polar_ns_workspace(rows: int, cols: int, hp: HParams) -> int:
    return int(lib().signmuon_polar_ns_workspace(rows, cols, ctypes.byref(hp.to_c())))


def polar_ns(X, hp: HParams, u0=None, U=None, ws=None, stream=None):
    import torch
    _require(X, torch.float32, "X")
    rows, cols = X.shape
    if U is None:
        U = torch.empty_like(X)
    nbytes = polar_ns_workspace(rows, cols, hp)
    if nbytes == 0:
        raise SignMuonError("signmuon_polar_ns_workspace", SM_EINVAL, "invalid arguments")
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=X.device)
    if u0 is not None:
        _require(u0, torch.float32, "u0")
    _check("signmuon_polar_ns", lib().signmuon_polar_ns(
        _ptr(X), _ptr(U), rows, cols, ctypes.byref(hp.to_c()), _ptr(u0), _ptr(ws),
        ws.numel(), _stream(stream)))
    return U


STATIC_SCRATCH_BYTES = 64 << 20


def polar_ns_static(X, hp: HParams, u0=None, U=None, stream=None):
    """PolarNS with the library's own per-GPU scratch array (no workspace,
    no allocation by the library; calls on one GPU must not overlap)."""
    import torch
    _require(X, torch.float32, "X")
    rows, cols = X.shape
    if U is None:
        U = torch.empty_like(X)
    _require(U, torch.float32, "U")
    if u0 is not None:
        _require(u0, torch.float32, "u0")
    _check("signmuon_polar_ns_static", lib().signmuon_polar_ns_static(
        _ptr(X), _ptr(U), rows, cols, ctypes.byref(hp.to_c()), _ptr(u0), _stream(stream)))
    return U


def sign_pack(U, bits=None, stream=None):
    import torch
    _require(U, torch.float32, "U")
    n = U.numel()
    if bits is None:
        bits = torch.empty((n + 31) // 32, dtype=torch.int32, device=U.device)
    _check("signmuon_sign_pack", lib().signmuon_sign_pack(_ptr(U), _ptr(bits), n,
                                                          _stream(stream)))
    return bits


def majority_vote(bits, M: int, n: int, tie_value: int = 0, stride: Optional[int] = None,
                  D=None, sums=None, want_sums: bool = False, stream=None):
    """bits: int32 tensor holding M worker buffers of `stride` words each."""
    import torch
    if stride is None:
        stride = (n + 31) // 32
    if D is None:
        D = torch.empty(n, dtype=torch.int8, device=bits.device)
    if want_sums and sums is None:
        sums = torch.empty(n, dtype=torch.int16, device=bits.device)
    _check("signmuon_majority_vote", lib().signmuon_majority_vote(
        _ptr(bits), stride, M, n, tie_value, _ptr(D), _ptr(sums), _stream(stream)))
    return (D, sums) if want_sums else D


def sign_ternary(U, S=None, stream=None):
    """int8 signs of U: +1, -1, or 0 for zero / NaN."""
    import torch
    _require(U, torch.float32, "U")
    n = U.numel()
    if S is None:
        S = torch.empty(n, dtype=torch.int8, device=U.device)
    _check("signmuon_sign_ternary", lib().signmuon_sign_ternary(_ptr(U), _ptr(S), n,
                                                                _stream(stream)))
    return S


def majority_vote_ternary(S, M: int, n: int, tie_value: int = 0,
                          stride: Optional[int] = None, D=None, sums=None,
                          want_sums: bool = False, stream=None):
    """S: int8 tensor holding M worker sign buffers of `stride` bytes each."""
    import torch
    if stride is None:
        stride = n
    if D is None:
        D = torch.empty(n, dtype=torch.int8, device=S.device)
    if want_sums and sums is None:
        sums = torch.empty(n, dtype=torch.int16, device=S.device)
    _check("signmuon_majority_vote_ternary", lib().signmuon_majority_vote_ternary(
        _ptr(S), stride, M, n, tie_value, _ptr(D), _ptr(sums), _stream(stream)))
    return (D, sums) if want_sums else D


def apply(W, eta: float, D=None, Df=None, stream=None):
    n = W.numel()
    _check("signmuon_apply", lib().signmuon_apply(
        _ptr(W), _wdtype(W), _ptr(D), _ptr(Df), eta, n, _stream(stream)))
    return W


# ---------------------------------------------------------------------------
# Layers (include/signmuon_layers.h).  Calls run on the device of their first
# tensor, on `stream` (default: that device's current stream); what they
# allocate belongs to that stream.  The checks are written for speed: small
# calls take as long as their host side.
# ---------------------------------------------------------------------------
def _here(t, stream) -> int:
    """The device of t if a call can go straight to its current stream, -1 if
    device and stream have to be set first."""
    import torch
    dev = t.get_device()
    if dev < 0:
        raise TypeError("tensors must be on a GPU")
    return dev if stream is None and dev == torch.cuda.current_device() else -1


@contextlib.contextmanager
def _placed(t, stream):
    import torch
    if stream is not None and stream.device != t.device:
        raise ValueError("the stream is not on the tensors' device")
    with torch.cuda.device(t.device), torch.cuda.stream(stream):
        yield


def _raw_stream(dev: int) -> int:
    """Handle of the device's current stream (0.1 us; building a torch Stream
    object for it takes 2 us)."""
    import torch
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return get(dev) if get else torch.cuda.current_stream(dev).cuda_stream


def _code(dtype, name) -> int:
    import torch
    if dtype is torch.bfloat16:
        return SM_BF16
    if dtype is torch.float32:
        return SM_F32
    raise TypeError(f"{name} must be float32 or bfloat16")


def _rows(t, name) -> Tuple[int, int, int]:
    """(rows, cols, row stride) of a tensor whose last dimension is dense:
    any contiguous one, or a 2-D one with longer row strides."""
    shape = t.shape
    if not shape:
        raise ValueError(f"{name} must have at least one dimension")
    cols = shape[-1]
    if t.is_contiguous():
        return (t.numel() // cols if cols else 0), cols, cols
    if len(shape) == 2 and (cols == 1 or t.stride(1) == 1):
        if shape[0] == 1:
            return 1, cols, cols
        if t.stride(0) >= cols:
            return shape[0], cols, t.stride(0)
    raise TypeError(f"{name} must be contiguous, or 2-D with contiguous rows that do not overlap")


def _check_arg(t, shape, dtype, dev, name):
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is not on the first tensor's device")


def _dense_like(t):
    import torch
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _workspace(ws, nbytes, like, dev):
    """(ws, pointer, bytes) of the workspace: the caller's, or a new one where
    one is needed."""
    import torch
    if nbytes == 0:
        return None, None, 0
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    elif not ws.is_contiguous():
        raise TypeError("ws must be contiguous")
    elif ws.get_device() != dev:
        raise ValueError("ws is not on the first tensor's device")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def layer_norm(X, weight=None, bias=None, eps: float = 1e-5, want_stats: bool = False, Y=None,
               mean=None, rstd=None, stream=None):
    """Layer norm over the last dimension of X (float32 or bfloat16): Y, or
    with want_stats (Y, mean, rstd), the latter float32 of X's leading shape.
    weight and bias: float32 or bfloat16, one dtype for both; None stands for
    ones and zeros.  Y may be X."""
    import torch
    dev = _here(X, stream)
    if dev < 0:
        with _placed(X, stream):
            return layer_norm(X, weight, bias, eps, want_stats, Y, mean, rstd)
    rows, cols, xs = _rows(X, "X")
    xd = wd = _code(X.dtype, "X")
    if weight is not None:
        wd = _code(weight.dtype, "weight")
        _check_arg(weight, (cols,), weight.dtype, dev, "weight")
        if bias is not None:
            _check_arg(bias, (cols,), weight.dtype, dev, "bias")
    elif bias is not None:
        wd = _code(bias.dtype, "bias")
        _check_arg(bias, (cols,), bias.dtype, dev, "bias")
    if Y is None:
        Y = _dense_like(X)
    else:
        _check_arg(Y, X.shape, X.dtype, dev, "Y")
    if mean is not None:
        _check_arg(mean, X.shape[:-1], torch.float32, dev, "mean")
    elif want_stats:
        mean = torch.empty(rows, dtype=torch.float32, device=X.device)
        if X.dim() != 2:
            mean = mean.view(X.shape[:-1])
    if rstd is not None:
        _check_arg(rstd, X.shape[:-1], torch.float32, dev, "rstd")
    elif want_stats:
        rstd = torch.empty_like(mean)
    _check("signmuon_layer_norm", lib().signmuon_layer_norm(
        X.data_ptr(), xd, xs, _ptr(weight), _ptr(bias), wd, rows, cols, eps, Y.data_ptr(),
        _ptr(mean), _ptr(rstd), _raw_stream(dev)))
    return (Y, mean, rstd) if want_stats else Y


def layer_norm_backward_workspace(rows: int, cols: int) -> int:
    n = lib().signmuon_layer_norm_backward_workspace(rows, cols)
    if n == _NO_SIZE:
        _check("signmuon_layer_norm_backward_workspace", SM_EINVAL)
    return n


def layer_norm_backward(dY, X, weight, mean, rstd, want_x: bool = True, want_weight: bool = True,
                        want_bias: bool = True, dX=None, dweight=None, dbias=None, dtype=None,
                        accumulate: bool = False, ws=None, stream=None):
    """(dX, dweight, dbias) of layer_norm, None in the place of one that is
    not wanted.  mean and rstd are the forward pass's; dX may be dY.  dtype:
    that of dweight and dbias (default: what dweight or dbias has, else
    float32).  accumulate adds to the dweight and dbias passed in (float32);
    dX is overwritten."""
    import torch
    dev = _here(dY, stream)
    if dev < 0:
        with _placed(dY, stream):
            return layer_norm_backward(dY, X, weight, mean, rstd, want_x, want_weight, want_bias,
                                       dX, dweight, dbias, dtype, accumulate, ws)
    rows, cols, dys = _rows(dY, "dY")
    xd = wd = _code(X.dtype, "X")
    if X.dtype != dY.dtype or X.shape != dY.shape:
        raise TypeError("dY must have X's dtype and shape")
    if X.get_device() != dev:
        raise ValueError("X is not on the first tensor's device")
    xs = _rows(X, "X")[2]
    if weight is not None:
        wd = _code(weight.dtype, "weight")
        _check_arg(weight, (cols,), weight.dtype, dev, "weight")
    _check_arg(mean, X.shape[:-1], torch.float32, dev, "mean")
    _check_arg(rstd, X.shape[:-1], torch.float32, dev, "rstd")
    if not want_x:
        dX = None
    elif dX is None:
        dX = _dense_like(X)
    else:
        _check_arg(dX, X.shape, X.dtype, dev, "dX")
    if not want_weight:
        dweight = None
    if not want_bias:
        dbias = None
    if accumulate and ((want_weight and dweight is None) or (want_bias and dbias is None)):
        raise ValueError("accumulate needs the dweight and dbias to add to")
    if dtype is None:
        dtype = (dweight.dtype if dweight is not None else
                 dbias.dtype if dbias is not None else torch.float32)
    dwd = SM_F32
    if want_weight:
        if dweight is None:
            dweight = torch.empty(cols, dtype=dtype, device=X.device)
        else:
            _check_arg(dweight, (cols,), dtype, dev, "dweight")
        dwd = _code(dweight.dtype, "dweight")
    if want_bias:
        if dbias is None:
            dbias = torch.empty(cols, dtype=dtype, device=X.device)
        else:
            _check_arg(dbias, (cols,), dtype, dev, "dbias")
        dwd = _code(dbias.dtype, "dbias")
    ws, wsp, nbytes = _workspace(ws, layer_norm_backward_workspace(rows, cols), X, dev)
    _check("signmuon_layer_norm_backward", lib().signmuon_layer_norm_backward(
        dY.data_ptr(), dys, X.data_ptr(), xd, xs, _ptr(weight), wd, mean.data_ptr(),
        rstd.data_ptr(), rows, cols, _ptr(dX), _ptr(dweight), _ptr(dbias), dwd, accumulate,
        wsp, nbytes, _raw_stream(dev)))
    return dX, dweight, dbias


def _token_bits(t) -> int:
    import torch
    if t.dtype == torch.int64:
        bits = 64
    elif t.dtype == torch.int32:
        bits = 32
    else:
        raise TypeError("tokens must be int32 or int64")
    if not t.is_contiguous():
        raise TypeError("tokens must be contiguous")
    return bits


def embedding(tokens, weight, scale: float = 1.0, out=None, out_dtype=None, stream=None):
    """scale * weight[tokens], of shape tokens.shape + (dim,), in out_dtype
    (default: weight's).  A token outside the table makes its row NaN."""
    import torch
    dev = _here(tokens, stream)
    if dev < 0:
        with _placed(tokens, stream):
            return embedding(tokens, weight, scale, out, out_dtype)
    bits = _token_bits(tokens)
    shape = weight.shape
    if len(shape) != 2 or not weight.is_contiguous():
        raise TypeError("weight must be a contiguous 2-D tensor")
    if weight.get_device() != dev:
        raise ValueError("weight is not on the first tensor's device")
    vocab, dim = shape
    wd = _code(weight.dtype, "weight")
    if out is None:
        out = torch.empty(*tokens.shape, dim, dtype=out_dtype or weight.dtype,
                          device=weight.device)
    else:
        _check_arg(out, tokens.shape + (dim,), out_dtype or out.dtype, dev, "out")
    _check("signmuon_embedding", lib().signmuon_embedding(
        weight.data_ptr(), wd, vocab, dim, tokens.data_ptr(), bits, tokens.numel(), scale,
        out.data_ptr(), _code(out.dtype, "out"), _raw_stream(dev)))
    return out


def embedding_backward_workspace(n: int, vocab: int, dim: int) -> int:
    nbytes = lib().signmuon_embedding_backward_workspace(n, vocab, dim)
    if nbytes == _NO_SIZE:
        _check("signmuon_embedding_backward_workspace", SM_EINVAL)
    return nbytes


def embedding_backward(dY, tokens, vocab: int, scale: float = 1.0, padding: Optional[int] = None,
                       dW=None, dtype=None, accumulate: bool = False, ws=None, stream=None):
    """Gradient of the table: dW[v] = scale * the sum of dY's rows whose token
    is v, for all v < vocab, in dtype (default: dW's, else float32).  Tokens
    equal to padding or outside the table add nothing.  accumulate adds to
    the float32 dW passed in, and touches only the rows of present tokens."""
    import torch
    dev = _here(dY, stream)
    if dev < 0:
        with _placed(dY, stream):
            return embedding_backward(dY, tokens, vocab, scale, padding, dW, dtype, accumulate,
                                      ws)
    bits = _token_bits(tokens)
    n = tokens.numel()
    rows, dim, dys = _rows(dY, "dY")
    if rows != n and dim:
        raise ValueError("dY must have one row for each token")
    if tokens.get_device() != dev:
        raise ValueError("tokens are not on the first tensor's device")
    dyd = _code(dY.dtype, "dY")
    if dW is None:
        if accumulate:
            raise ValueError("accumulate needs the dW to add to")
        dW = torch.empty(vocab, dim, dtype=dtype or torch.float32, device=dY.device)
    else:
        _check_arg(dW, (vocab, dim), dtype or dW.dtype, dev, "dW")
    ws, wsp, nbytes = _workspace(ws, embedding_backward_workspace(n, vocab, dim), dY, dev)
    _check("signmuon_embedding_backward", lib().signmuon_embedding_backward(
        dY.data_ptr(), dyd, dys, tokens.data_ptr(), bits, n,
        -1 if padding is None else int(padding), scale, dW.data_ptr(), _code(dW.dtype, "dW"), vocab,
        dim, accumulate, wsp, nbytes, _raw_stream(dev)))
    return dW


def _rms_args(X, weight, residual, H, rstd, want_stats, dev):
    """(rows, cols, x stride, residual stride, x code, weight code, H, rstd)."""
    import torch
    rows, cols, xs = _rows(X, "X")
    xd = wd = _code(X.dtype, "X")
    rs = xs
    if weight is not None:
        wd = _code(weight.dtype, "weight")
        _check_arg(weight, (cols,), weight.dtype, dev, "weight")
    if residual is not None:
        if residual.dtype is not X.dtype or residual.shape != X.shape:
            raise TypeError("residual must have X's dtype and shape")
        if residual.get_device() != dev:
            raise ValueError("residual is not on the first tensor's device")
        rs = cols if residual.is_contiguous() else _rows(residual, "residual")[2]
        if H is None:
            H = _dense_like(X)
        else:
            _check_arg(H, X.shape, X.dtype, dev, "H")
    elif H is not None:
        raise ValueError("H is the sum with a residual")
    if rstd is not None:
        _check_arg(rstd, X.shape[:-1], torch.float32, dev, "rstd")
    elif want_stats:
        rstd = torch.empty(rows, dtype=torch.float32, device=X.device)
        if X.dim() != 2:
            rstd = rstd.view(X.shape[:-1])
    return rows, cols, xs, rs, xd, wd, H, rstd


def rms_norm(X, weight=None, residual=None, eps: float = 1e-6, want_stats: bool = False, Y=None,
             H=None, rstd=None, stream=None):
    """Root-mean-square norm over the last dimension of X, or of X + residual: Y
    without a residual, else (Y, H) with H the sum, rounded to X's dtype, that the
    norm is taken of.  With want_stats always (Y, H, rstd), H being X without a
    residual; rstd is float32 of X's leading shape.  X and residual: float32 or
    bfloat16; weight: float32 or bfloat16, None for ones.  H may be X or residual, Y
    may be X."""
    dev = _here(X, stream)
    if dev < 0:
        with _placed(X, stream):
            return rms_norm(X, weight, residual, eps, want_stats, Y, H, rstd)
    rows, cols, xs, rs, xd, wd, H, rstd = _rms_args(X, weight, residual, H, rstd, want_stats, dev)
    if Y is None:
        Y = _dense_like(X)
    else:
        _check_arg(Y, X.shape, X.dtype, dev, "Y")
    _check("signmuon_rms_norm", lib().signmuon_rms_norm(
        X.data_ptr(), xs, _ptr(residual), rs, xd, _ptr(weight), wd, rows, cols, eps, _ptr(H),
        Y.data_ptr(), _ptr(rstd), _raw_stream(dev)))
    if want_stats:
        return Y, X if H is None else H, rstd
    return Y if H is None else (Y, H)


def rms_norm_e4m3(X, weight=None, residual=None, eps: float = 1e-6, block: Optional[int] = 128,
                  want_stats: bool = False, Q=None, scales=None, H=None, rstd=None, stream=None):
    """rms_norm with its output in 8 bits: (Q, scales), (Q, scales, H) with a
    residual, and with want_stats (Q, scales, H, rstd).  Q: float8_e4m3fn of X's
    shape; scales: float32, one for each `block` = 128 columns of a row (None: one a
    row); Q * scale stands for Y, the largest value of a block for 448 * scale.  Rows
    of up to 16384 columns."""
    import torch
    dev = _here(X, stream)
    if dev < 0:
        with _placed(X, stream):
            return rms_norm_e4m3(X, weight, residual, eps, block, want_stats, Q, scales, H, rstd)
    rows, cols, xs, rs, xd, wd, H, rstd = _rms_args(X, weight, residual, H, rstd, want_stats, dev)
    if Q is None:
        Q = torch.empty(X.shape, dtype=torch.float8_e4m3fn, device=X.device)
    else:
        _check_arg(Q, X.shape, torch.float8_e4m3fn, dev, "Q")
    if block is not None and block != 128:
        raise ValueError("block must be 128, or None for a whole row")
    shape = X.shape[:-1] + (1 if block is None else -(-cols // 128),)
    if scales is None:
        scales = torch.empty(shape, dtype=torch.float32, device=X.device)
    else:
        _check_arg(scales, shape, torch.float32, dev, "scales")
    _check("signmuon_rms_norm_e4m3", lib().signmuon_rms_norm_e4m3(
        X.data_ptr(), xs, _ptr(residual), rs, xd, _ptr(weight), wd, rows, cols, eps, block or 0,
        _ptr(H), Q.data_ptr(), scales.data_ptr(), _ptr(rstd), _raw_stream(dev)))
    if want_stats:
        return Q, scales, X if H is None else H, rstd
    return (Q, scales) if H is None else (Q, scales, H)


def rms_norm_backward_workspace(rows: int, cols: int) -> int:
    n = lib().signmuon_rms_norm_backward_workspace(rows, cols)
    if n == _NO_SIZE:
        _check("signmuon_rms_norm_backward_workspace", SM_EINVAL)
    return n


def rms_norm_backward(dY, H, weight, rstd, dH=None, want_x: bool = True, want_weight: bool = True,
                      dX=None, dweight=None, dtype=None, accumulate: bool = False, ws=None,
                      stream=None):
    """(dX, dweight) of rms_norm for the gradients dY of Y and dH of H (None: H has
    no other use), None in the place of one that is not wanted.  dX is the gradient
    of X and of the residual.  H and rstd are the forward pass's; dX may be dY or dH.
    dtype: dweight's (default: what dweight has, else float32).  accumulate adds to
    the float32 dweight passed in; dX is overwritten."""
    import torch
    dev = _here(dY, stream)
    if dev < 0:
        with _placed(dY, stream):
            return rms_norm_backward(dY, H, weight, rstd, dH, want_x, want_weight, dX, dweight,
                                     dtype, accumulate, ws)
    rows, cols, dys = _rows(dY, "dY")
    xd = wd = _code(H.dtype, "H")
    strides = []
    for t, name in ((H, "H"), (dH, "dH")):
        if t is None:
            strides.append(cols)
            continue
        if t.dtype != dY.dtype or t.shape != dY.shape:
            raise TypeError(f"{name} must have dY's dtype and shape")
        if t.get_device() != dev:
            raise ValueError(f"{name} is not on the first tensor's device")
        strides.append(_rows(t, name)[2])
    if weight is not None:
        wd = _code(weight.dtype, "weight")
        _check_arg(weight, (cols,), weight.dtype, dev, "weight")
    _check_arg(rstd, H.shape[:-1], torch.float32, dev, "rstd")
    if not want_x:
        dX = None
    elif dX is None:
        dX = _dense_like(H)
    else:
        _check_arg(dX, H.shape, H.dtype, dev, "dX")
    dwd = SM_F32
    if not want_weight:
        dweight = None
    elif dweight is None:
        if accumulate:
            raise ValueError("accumulate needs the dweight to add to")
        dweight = torch.empty(cols, dtype=dtype or torch.float32, device=H.device)
    else:
        _check_arg(dweight, (cols,), dtype or dweight.dtype, dev, "dweight")
    if want_weight:
        dwd = _code(dweight.dtype, "dweight")
    ws, wsp, nbytes = _workspace(ws, rms_norm_backward_workspace(rows, cols), H, dev)
    _check("signmuon_rms_norm_backward", lib().signmuon_rms_norm_backward(
        dY.data_ptr(), dys, H.data_ptr(), strides[0], _ptr(dH), strides[1], xd, _ptr(weight), wd,
        rstd.data_ptr(), rows, cols, _ptr(dX), _ptr(dweight), dwd, bool(accumulate and want_weight),
        wsp, nbytes, _raw_stream(dev)))
    return dX, dweight


def _mlp_args(X, w_gate, w_up, w_down, activation, dev):
    """(rows, dim, row stride, hidden, dtype code, activation code)."""
    rows, dim, xs = _rows(X, "X")
    code = _code(X.dtype, "X")
    if w_gate.dim() != 2:
        raise TypeError("w_gate must be a 2-D tensor")
    hidden = w_gate.shape[0]
    for t, shape, name in ((w_gate, (hidden, dim), "w_gate"), (w_up, (hidden, dim), "w_up"),
                           (w_down, (dim, hidden), "w_down")):
        _check_arg(t, shape, X.dtype, dev, name)
    if activation not in ACTIVATIONS:
        raise ValueError("activation must be silu or gelu")
    return rows, dim, xs, hidden, code, ACTIVATIONS[activation]


def gated_mlp_workspace(rows: int, dim: int, hidden: int, dtype, backward: bool) -> int:
    nbytes = lib().signmuon_gated_mlp_workspace(rows, dim, hidden, _code(dtype, "dtype"),
                                                bool(backward))
    if nbytes == _NO_SIZE:
        _check("signmuon_gated_mlp_workspace", SM_EINVAL)
    return nbytes


def gated_mlp(X, w_gate, w_up, w_down, activation: str = "silu", want_pre: bool = False, Y=None,
              pre=None, ws=None, stream=None):
    """Gated feed-forward block (act(X w_gate^T) * (X w_up^T)) w_down^T over the last
    dimension of X: Y, or with want_pre (Y, pre), the float32 pre-activations (...,
    2 hidden), gate and then up, that the backward pass needs.  X: float32 or
    bfloat16, (..., dim); w_gate, w_up: (hidden, dim) and w_down: (dim, hidden) of
    the same dtype.  activation: "silu" or "gelu"."""
    import torch
    dev = _here(X, stream)
    if dev < 0:
        with _placed(X, stream):
            return gated_mlp(X, w_gate, w_up, w_down, activation, want_pre, Y, pre, ws)
    rows, dim, xs, hidden, code, act = _mlp_args(X, w_gate, w_up, w_down, activation, dev)
    if Y is None:
        Y = _dense_like(X)
    else:
        _check_arg(Y, X.shape, X.dtype, dev, "Y")
    if pre is not None:
        _check_arg(pre, X.shape[:-1] + (2 * hidden,), torch.float32, dev, "pre")
    elif want_pre:
        pre = torch.empty(X.shape[:-1] + (2 * hidden,), dtype=torch.float32, device=X.device)
    ws, wsp, nbytes = _workspace(ws, gated_mlp_workspace(rows, dim, hidden, X.dtype, False), X,
                                 dev)
    _check("signmuon_gated_mlp", lib().signmuon_gated_mlp(
        X.data_ptr(), xs, w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(), code, act, rows,
        dim, hidden, Y.data_ptr(), _ptr(pre), wsp, nbytes, _raw_stream(dev)))
    return (Y, pre) if want_pre else Y


def gated_mlp_backward(dY, X, w_gate, w_up, w_down, pre, activation: str = "silu",
                       want=(True, True, True, True), dX=None, dw_gate=None, dw_up=None,
                       dw_down=None, dtype=None, accumulate: bool = False, ws=None, stream=None):
    """(dX, dw_gate, dw_up, dw_down) of gated_mlp, None in the place of one whose entry
    of want is False.  pre is the forward pass's.  dtype: that of the weights'
    gradients (default: what those passed in have, else float32).  accumulate adds to
    the float32 ones, which have to be passed in then; dX is overwritten."""
    import torch
    dev = _here(X, stream)
    if dev < 0:
        with _placed(X, stream):
            return gated_mlp_backward(dY, X, w_gate, w_up, w_down, pre, activation, want, dX,
                                      dw_gate, dw_up, dw_down, dtype, accumulate, ws)
    rows, dim, xs, hidden, code, act = _mlp_args(X, w_gate, w_up, w_down, activation, dev)
    if dY.dtype != X.dtype or dY.shape != X.shape:
        raise TypeError("dY must have X's dtype and shape")
    if dY.get_device() != dev:
        raise ValueError("dY is not on the first tensor's device")
    dys = _rows(dY, "dY")[2]
    _check_arg(pre, X.shape[:-1] + (2 * hidden,), torch.float32, dev, "pre")
    if not want[0]:
        dX = None
    elif dX is None:
        dX = _dense_like(X)
    else:
        _check_arg(dX, X.shape, X.dtype, dev, "dX")
    grads = [g if w else None for g, w in zip((dw_gate, dw_up, dw_down), want[1:])]
    if dtype is None:
        dtype = next((g.dtype for g in grads if g is not None), torch.float32)
    for i, (w, like) in enumerate(zip(want[1:], (w_gate, w_up, w_down))):
        if w and grads[i] is None:
            if accumulate:
                raise ValueError("accumulate needs the weights' gradients to add to")
            grads[i] = torch.empty(like.shape, dtype=dtype, device=X.device)
        elif w:
            _check_arg(grads[i], like.shape, dtype, dev, ("dw_gate", "dw_up", "dw_down")[i])
    ws, wsp, nbytes = _workspace(ws, gated_mlp_workspace(rows, dim, hidden, X.dtype, True), X, dev)
    _check("signmuon_gated_mlp_backward", lib().signmuon_gated_mlp_backward(
        dY.data_ptr(), dys, X.data_ptr(), xs, w_gate.data_ptr(), w_up.data_ptr(),
        w_down.data_ptr(), pre.data_ptr(), code, act, rows, dim, hidden, _ptr(dX),
        _ptr(grads[0]), _ptr(grads[1]), _ptr(grads[2]), _code(dtype, "dtype"),
        bool(accumulate and any(want[1:])), wsp, nbytes, _raw_stream(dev)))
    return (dX, *grads)


def _loss_args(X, weight, targets, ignore_index, reduction, dev):
    """(rows, dim, row stride, vocab, dtype code, target bits, reduction code)."""
    rows, dim, xs = _rows(X, "X")
    code = _code(X.dtype, "X")
    if weight.dim() != 2 or weight.shape[1] != dim:
        raise TypeError("weight must be a 2-D tensor with X's last dimension")
    _check_arg(weight, weight.shape, X.dtype, dev, "weight")
    bits = _token_bits(targets)
    if targets.shape != X.shape[:-1]:
        raise ValueError("targets must have X's leading shape")
    if targets.get_device() != dev:
        raise ValueError("targets are not on the first tensor's device")
    if reduction not in REDUCTIONS:
        raise ValueError("reduction must be none, sum or mean")
    if not -1 << 63 <= ignore_index < 1 << 63:      # (ctypes would take its low 64 bits)
        raise ValueError("ignore_index must be a 64-bit integer")
    return rows, dim, xs, weight.shape[0], code, bits, REDUCTIONS[reduction]


def linear_cross_entropy_workspace(rows: int, dim: int, vocab: int, dtype, backward: bool) -> int:
    nbytes = lib().signmuon_linear_cross_entropy_workspace(rows, dim, vocab,
                                                           _code(dtype, "dtype"), bool(backward))
    if nbytes == _NO_SIZE:
        _check("signmuon_linear_cross_entropy_workspace", SM_EINVAL)
    return nbytes


def linear_cross_entropy(X, weight, targets, ignore_index: int = -100, reduction: str = "mean",
                         want_lse: bool = False, loss=None, lse=None, ws=None, stream=None):
    """Softmax cross entropy of the logits X weight^T, which are not kept: loss,
    or with want_lse (loss, lse).  X: float32 or bfloat16, (..., dim); weight:
    (vocab, dim) of the same dtype; targets: int32 or int64 of X's leading shape.
    loss is a float32 scalar for reduction "mean" (over the rows whose target is
    not ignore_index; 0 where none is left) and "sum", and of the targets' shape
    for "none"; lse, float32 of the targets' shape, is what the backward pass
    needs."""
    import torch
    dev = _here(X, stream)
    if dev < 0:
        with _placed(X, stream):
            return linear_cross_entropy(X, weight, targets, ignore_index, reduction, want_lse,
                                        loss, lse, ws)
    rows, dim, xs, vocab, code, bits, red = _loss_args(X, weight, targets, ignore_index,
                                                        reduction, dev)
    shape = targets.shape if red == 0 else targets.shape[:0]
    if loss is None:
        loss = torch.empty(shape, dtype=torch.float32, device=X.device)
    else:
        _check_arg(loss, shape, torch.float32, dev, "loss")
    if lse is None:
        lse = torch.empty(targets.shape, dtype=torch.float32, device=X.device)
    else:
        _check_arg(lse, targets.shape, torch.float32, dev, "lse")
    ws, wsp, nbytes = _workspace(ws, linear_cross_entropy_workspace(rows, dim, vocab, X.dtype,
                                                                    False), X, dev)
    _check("signmuon_linear_cross_entropy", lib().signmuon_linear_cross_entropy(
        X.data_ptr(), xs, weight.data_ptr(), code, targets.data_ptr(), bits, rows, dim, vocab,
        int(ignore_index), red, loss.data_ptr(), lse.data_ptr(), wsp, nbytes, _raw_stream(dev)))
    return (loss, lse) if want_lse else loss


def linear_cross_entropy_backward(dloss, X, weight, targets, lse, ignore_index: int = -100,
                                  reduction: str = "mean", want_x: bool = True,
                                  want_weight: bool = True, dX=None, dweight=None, dtype=None,
                                  accumulate: bool = False, ws=None, stream=None):
    """(dX, dweight) of linear_cross_entropy for the float32 gradient dloss of its
    loss, None in the place of one that is not wanted.  lse is the forward
    pass's.  dX may be X.  dtype: dweight's (default: what dweight has, else
    float32).  accumulate adds to the float32 dweight passed in; dX is
    overwritten."""
    import torch
    dev = _here(X, stream)
    if dev < 0:
        with _placed(X, stream):
            return linear_cross_entropy_backward(dloss, X, weight, targets, lse, ignore_index,
                                                 reduction, want_x, want_weight, dX, dweight,
                                                 dtype, accumulate, ws)
    rows, dim, xs, vocab, code, bits, red = _loss_args(X, weight, targets, ignore_index,
                                                        reduction, dev)
    _check_arg(dloss, targets.shape if red == 0 else targets.shape[:0], torch.float32, dev,
               "dloss")
    _check_arg(lse, targets.shape, torch.float32, dev, "lse")
    if not want_x:
        dX = None
    elif dX is None:
        dX = _dense_like(X)
    else:
        _check_arg(dX, X.shape, X.dtype, dev, "dX")
    dwd = SM_F32
    if not want_weight:
        dweight = None
    elif dweight is None:
        if accumulate:
            raise ValueError("accumulate needs the dweight to add to")
        dweight = torch.empty(weight.shape, dtype=dtype or torch.float32, device=X.device)
    else:
        _check_arg(dweight, weight.shape, dtype or dweight.dtype, dev, "dweight")
    if want_weight:
        dwd = _code(dweight.dtype, "dweight")
    ws, wsp, nbytes = _workspace(ws, linear_cross_entropy_workspace(rows, dim, vocab, X.dtype,
                                                                    True), X, dev)
    _check("signmuon_linear_cross_entropy_backward",
           lib().signmuon_linear_cross_entropy_backward(
               dloss.data_ptr(), X.data_ptr(), xs, weight.data_ptr(), code, targets.data_ptr(),
               bits, lse.data_ptr(), rows, dim, vocab, int(ignore_index), red, _ptr(dX),
               _ptr(dweight), dwd, bool(accumulate) and want_weight, wsp, nbytes,
               _raw_stream(dev)))
    return dX, dweight


def step_workspace(mats, hp: HParams, post_vote: int) -> int:
    arr = mats_array(mats)
    return int(lib().signmuon_step_workspace(arr, len(mats), ctypes.byref(hp.to_c()),
                                             int(post_vote)))


class Executor:
    """Owner of a signmuon_executor (the streams and events of the concurrent
    PolarNS chains), created on the current device; freed on close() or
    garbage collection."""

    def __init__(self):
        h = ctypes.c_void_p()
        _check("signmuon_executor_create", lib().signmuon_executor_create(ctypes.byref(h)))
        self.handle = h

    def close(self):
        if self.handle is not None and self.handle.value:
            _check("signmuon_executor_destroy", lib().signmuon_executor_destroy(self.handle))
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class StepPlan:
    """Cached ctypes arguments of one parameter set for repeated steps.

    concurrent: run the PolarNS chains concurrently on an executor owned by
    the plan (default); False enqueues every kernel on the caller's stream."""

    def __init__(self, mats, hp: HParams, post_vote: int, device=None,
                 concurrent: bool = True):
        import torch
        self.mats = list(mats)
        self.arr = mats_array(self.mats)
        self.hp = hp
        self.hpc = hp.to_c()
        # 0: Algorithm 2; 1: polar step after the vote; 2: both
        self.post_vote = int(post_vote)
        nbytes = step_workspace(self.mats, hp, post_vote)
        if nbytes == 0:
            raise SignMuonError("signmuon_step_workspace", SM_EINVAL, "invalid arguments")
        dev = torch.device(device or "cuda")
        # zero-filled: the first bytes carry the non-finite flags
        self.ws = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
        self.executor = None
        if concurrent:
            with torch.cuda.device(self.ws.device):
                self.executor = Executor()

    def _ex(self):
        return None if self.executor is None else self.executor.handle

    def set_eta(self, eta: float):
        self.hp.eta = eta
        self.hpc.eta = eta

    def __call__(self, G, W, Mom, bits, stride: int, M: int, local_worker: int = 0,
                 u0=None, stream=None):
        _check("signmuon_step", lib().signmuon_step(
            self.arr, len(self.mats), ctypes.byref(self.hpc), _ptr(G), _ptr(W),
            _wdtype(W), _ptr(Mom), _ptr(bits), stride, M, local_worker,
            int(self.post_vote), _ptr(u0), _ptr(self.ws), self.ws.numel(),
            self._ex(), _stream(stream)))

    def worker_pipeline(self, G, W, Mom, bits, stride: int, M: int, worker: int,
                        u0=None, stream=None):
        """Worker `worker`'s momentum, PolarNS and sign packing (no vote,
        W unchanged)."""
        _check("signmuon_worker_pipeline", lib().signmuon_worker_pipeline(
            self.arr, len(self.mats), ctypes.byref(self.hpc), _ptr(G), _ptr(W),
            _wdtype(W), _ptr(Mom), _ptr(bits), stride, M, worker,
            int(self.post_vote), _ptr(u0), _ptr(self.ws), self.ws.numel(),
            self._ex(), _stream(stream)))

    def profiled(self, prof: "SmProfile", G, W, Mom, bits, stride: int, M: int,
                 local_worker: int = 0, u0=None, stream=None):
        """Same step, recording prof's events after each phase."""
        _check("signmuon_step_profiled", lib().signmuon_step_profiled(
            self.arr, len(self.mats), ctypes.byref(self.hpc), _ptr(G), _ptr(W),
            _wdtype(W), _ptr(Mom), _ptr(bits), stride, M, local_worker,
            int(self.post_vote), _ptr(u0), _ptr(self.ws), self.ws.numel(),
            ctypes.byref(prof), self._ex(), _stream(stream)))

    def status(self, stream=None) -> int:
        return int(lib().signmuon_get_status(_ptr(self.ws), _stream(stream)))

    def reset_status(self, stream=None):
        _check("signmuon_reset_status", lib().signmuon_reset_status(_ptr(self.ws),
                                                                    _stream(stream)))

    def capture(self, G, W, Mom, bits, stride: int, M: int, local_worker: int = 0,
                u0=None):
        """Recording the step into a HIP graph is switched off: with this
        ROCm release, ending the capture of a step (torch.cuda.graph around
        one call) ended the process with a segmentation fault inside the
        runtime, also for sets that run as one chain on the capturing stream
        (so the fork and join of the executor's streams is not the cause),
        and no cause in the library has been found.  Steps are enqueued
        eagerly."""
        raise SignMuonError("StepPlan.capture", SM_EUNSUPPORTED,
                            "HIP graph capture of the step is disabled")
