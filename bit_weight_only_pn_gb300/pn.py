"""Python binding of the PN CUDA library (include/pn.h): argument marshalling only.

PyTorch supplies device memory and the current CUDA stream; every step of the
computation runs in the library's kernels.  There is no CPU path: if the
library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple

import torch

PN3T = 124
PN4T = 125
ALGO_AUTO, ALGO_TENSOR_CORE, ALGO_CUDA_CORE, ALGO_CUDA_CORE_STAGED = 0, 1, 2, 3
NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2
MAX_M = 16
MAX_LAYER = 8
STATUS = {0: "PN_OK", 1: "PN_EINVAL", 2: "PN_EALIGN", 3: "PN_EUNSUPPORTED", 4: "PN_ECUDA",
          5: "PN_ETIMEOUT"}

LIBRARY = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpn_gb300.so")

_lock = threading.Lock()
_lib = None


class PnError(RuntimeError):
    def __init__(self, status: int, what: str, cuda_error: str | None = None):
        detail = f" ({cuda_error})" if cuda_error else ""
        super().__init__(f"{what}: {STATUS.get(status, status)}{detail}")
        self.status = status
        self.cuda_error = cuda_error


class _Desc(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int), ("W", ctypes.c_void_p), ("N", ctypes.c_int64),
                ("K", ctypes.c_int64), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p)]


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIBRARY):
                raise RuntimeError(f"PN CUDA library not built ({LIBRARY}); run "
                                   "`python -m bit_weight_only_pn_gb300.build`")
            L = ctypes.CDLL(LIBRARY)
            vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
            L.pn_abi_version.restype = i32
            L.pn_status_string.restype = ctypes.c_char_p
            L.pn_status_string.argtypes = [i32]
            L.pn_last_cuda_error.restype = ctypes.c_char_p
            L.pn_last_cuda_error.argtypes = []
            L.pn_weights_per_block.restype = i32
            L.pn_weights_per_block.argtypes = [i32]
            L.pn_row_bytes.restype = sz
            L.pn_row_bytes.argtypes = [i32, i64]
            L.pn_pack.restype = i32
            L.pn_pack.argtypes = [i32, vp, i64, i64, vp, vp]
            L.pn_unpack.restype = i32
            L.pn_unpack.argtypes = [i32, vp, i64, i64, vp, vp]
            L.pn_workspace_bytes.restype = sz
            L.pn_workspace_bytes.argtypes = [i64]
            L.pn_workspace_init.restype = i32
            L.pn_workspace_init.argtypes = [vp, sz, vp]
            L.pn_workspace_status.restype = i32
            L.pn_workspace_status.argtypes = [vp, sz, vp]
            L.pn_gemv.restype = i32
            L.pn_gemv.argtypes = [i32, vp, i64, i64, vp, i32, vp, vp, sz, vp]
            L.pn_gemv_ex.restype = i32
            L.pn_gemv_ex.argtypes = [i32, vp, i64, i64, vp, i32, vp, vp, sz, i32, vp]
            L.pn_gemv_layer.restype = i32
            L.pn_gemv_layer.argtypes = [ctypes.POINTER(_Desc), i32, i32, vp, sz, vp]
            L.pn_gptq_scratch_bytes.restype = sz
            L.pn_gptq_scratch_bytes.argtypes = [i64, i64]
            L.pn_gptq.restype = i32
            L.pn_gptq.argtypes = [i32, vp, i64, i64, vp, i64, ctypes.c_double, vp, vp, sz, vp]
            L.pn_gemv_layer_host.restype = i32
            L.pn_gemv_layer_host.argtypes = [ctypes.POINTER(_Desc), i32, i32, vp, vp, vp, sz, vp]
            L.pn_gemv_hadamard.restype = i32
            L.pn_gemv_hadamard.argtypes = [i32, vp, i64, i64, vp, i32, i32, vp, vp, sz, vp]
            L.pn_gemv_layer_hadamard.restype = i32
            L.pn_gemv_layer_hadamard.argtypes = [ctypes.POINTER(_Desc), i32, i32, i32, vp, sz, vp]
            L.pn_gemv_layer_ex.restype = i32
            L.pn_gemv_layer_ex.argtypes = [ctypes.POINTER(_Desc), i32, i32, vp, sz, i32, vp]
            L.pn_unpack_f16.restype = i32
            L.pn_unpack_f16.argtypes = [i32, vp, i64, i64, vp, vp]
            L.pn_gemm_f16.restype = i32
            L.pn_gemm_f16.argtypes = [vp, i64, i64, vp, i64, vp, i64, vp, sz, vp]
            L.pn_prefill.restype = i32
            L.pn_prefill.argtypes = [i32, vp, i64, i64, vp, i64, vp, vp, sz, vp, sz, vp]
            f32 = ctypes.c_float
            L.pn_kv_cache_bytes.restype = sz
            L.pn_kv_cache_bytes.argtypes = [i64, i32, i32, i32]
            L.pn_kv_plan.restype = i32
            L.pn_kv_plan.argtypes = [vp, vp, vp, i32, vp, i64, i32, vp, i64, vp, i32, i64, vp, vp, vp, vp, vp, vp, vp,
                                     vp, vp]
            L.pn_kv_append.restype = i32
            L.pn_kv_append.argtypes = [vp, i64, vp, i64, vp, i64, i32, i64, i32, vp, vp, f32, vp, vp, i64, i32, i32,
                                       vp, vp, vp, i64, i32, i32, i32, vp, vp]
            L.pn_kv_read.restype = i32
            L.pn_kv_read.argtypes = [vp, i64, i32, i32, i32, vp, i64, vp, vp, vp]
            L.pn_attention_workspace_bytes.restype = sz
            L.pn_attention_workspace_bytes.argtypes = []
            L.pn_attention.restype = i32
            L.pn_attention.argtypes = [vp, i64, i64, i32, vp, i64, i32, i32, i32, vp, i64, i32, vp, vp, i32, i32, f32,
                                       i32, i32, vp, vp, vp, sz, vp]
            L.pn_verify.restype = i32
            L.pn_verify.argtypes = [vp, vp, i64, vp, i64, vp, vp, i32, i32, i32, vp, vp, vp]
            L.pn_logprobs.restype = i32
            L.pn_logprobs.argtypes = [vp, i64, i32, i64, i32, f32, vp, i32, vp, vp, i32, vp, vp, vp]
            L.pn_norm.restype = i32
            L.pn_norm.argtypes = [vp, i64, i32, vp, i64, i32, vp, i64, f32, i64, i32, i32, vp, vp, i32, vp, vp, f32, vp, i64, vp, vp]
            L.pn_kv_weigh.restype = i32
            L.pn_kv_weigh.argtypes = [vp, i64, i64, i32, vp, i64, i32, i32, i32, vp, i64, i32, vp, vp, i32, i32, vp, f32, i32, i32,
                                      vp, f32, vp, vp]
            L.pn_kv_weigh_ex.restype = i32
            L.pn_kv_weigh_ex.argtypes = [*L.pn_kv_weigh.argtypes[:-1], vp, sz, vp]
            L.pn_kv_evict.restype = i32
            L.pn_kv_evict.argtypes = [vp, i64, i32, i32, i32, vp, vp, i64, i32, vp, vp, i32, i32, i32, i32, i32, vp, i64, vp, vp,
                                      i64, vp, vp, vp, vp, vp, vp]
            L.pn_read_ranges.restype = i32
            L.pn_read_ranges.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(sz), i32, vp, vp]
            L.pn_hadamard.restype = i32
            L.pn_hadamard.argtypes = [vp, i32, i64, i32, vp, vp]
            L.pn_set_wait_timeout_ns.restype = None
            L.pn_set_wait_timeout_ns.argtypes = [ctypes.c_uint64]
            L.pn_set_test_stall.restype = None
            L.pn_set_test_stall.argtypes = [ctypes.c_int]
            L.pn_tc_split.restype = i32
            L.pn_tc_split.argtypes = [ctypes.POINTER(i32), ctypes.POINTER(i64), ctypes.POINTER(i64), i32, i32,
                                      i32, ctypes.POINTER(ctypes.c_uint32), ctypes.POINTER(i32)]
            _lib = L
        return _lib


def _check(status: int, what: str) -> None:
    if status != 0:
        cuda = lib().pn_last_cuda_error().decode() if status == 4 else None
        raise PnError(status, what, cuda)


def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _require(t: torch.Tensor, dtype, name: str) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def weights_per_block(pn_type: int) -> int:
    return int(lib().pn_weights_per_block(pn_type))


def row_bytes(pn_type: int, K: int) -> int:
    return int(lib().pn_row_bytes(pn_type, K))


def pack(pn_type: int, w: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """fp32 weights [N][K] -> PN rows uint8 [N][row_bytes]."""
    _require(w, torch.float32, "w")
    N, K = w.shape
    rb = row_bytes(pn_type, K)
    if rb == 0:
        raise ValueError(f"K={K} is not a whole number of blocks")
    if out is None:
        out = torch.empty((N, rb), dtype=torch.uint8, device=w.device)
    _require(out, torch.uint8, "out")
    _check(lib().pn_pack(pn_type, _ptr(w), N, K, _ptr(out), _stream(stream)), "pn_pack")
    return out


def unpack(pn_type: int, W: torch.Tensor, K: int, out: torch.Tensor | None = None,
           stream=None) -> torch.Tensor:
    """PN rows uint8 [N][row_bytes] -> fp32 weights [N][K] (exact)."""
    _require(W, torch.uint8, "W")
    N = W.shape[0]
    if out is None:
        out = torch.empty((N, K), dtype=torch.float32, device=W.device)
    _require(out, torch.float32, "out")
    _check(lib().pn_unpack(pn_type, _ptr(W), N, K, _ptr(out), _stream(stream)), "pn_unpack")
    return out


class Workspace:
    """Zeroed device scratch for GEMV calls on one device (see pn_workspace_bytes)."""

    def __init__(self, total_rows: int, device=None, stream=None):
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        with torch.cuda.device(self.device):
            self.nbytes = int(lib().pn_workspace_bytes(int(total_rows)))
            if self.nbytes == 0:
                raise PnError(4, "pn_workspace_bytes")
            self.buffer = torch.zeros(self.nbytes, dtype=torch.uint8, device=self.device)
        self.total_rows = int(total_rows)

    @property
    def ptr(self) -> int:
        return self.buffer.data_ptr()

    def status(self, stream=None) -> int:
        """Synchronise, read and clear the device status word (0 = ok)."""
        return int(lib().pn_workspace_status(self.ptr, self.nbytes, _stream(stream)))


def gemv(pn_type: int, W: torch.Tensor, K: int, x: torch.Tensor, y: torch.Tensor | None = None,
         workspace: Workspace | None = None, algo: int = ALGO_AUTO, stream=None) -> torch.Tensor:
    """y[M][N] = decode(W)[N][K] @ x[M][K]^T with fp32 accumulation (1 <= M <= 16)."""
    _require(W, torch.uint8, "W")
    _require(x, torch.float16, "x")
    if x.dim() == 1:
        x = x.view(1, -1)
    M = x.shape[0]
    N = W.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=W.device)
    _require(y, torch.float32, "y")
    ws_ptr, ws_bytes = (workspace.ptr, workspace.nbytes) if workspace is not None else (None, 0)
    _check(lib().pn_gemv_ex(pn_type, _ptr(W), N, K, _ptr(x), M, _ptr(y), ws_ptr, ws_bytes, algo,
                            _stream(stream)), "pn_gemv")
    return y


def gemv_layer(entries, M: int, workspace: Workspace | None = None, algo: int = ALGO_AUTO,
               stream=None):
    """Several independent GEMVs in one launch.

    ``entries`` is a sequence of (pn_type, W, K, x, y) with x fp16 [M][K] and y
    fp32 [M][N] preallocated.  Returns the list of y tensors.
    """
    entries = list(entries)
    arr = (_Desc * len(entries))()
    for i, (t, W, K, x, y) in enumerate(entries):
        _require(W, torch.uint8, "W")
        _require(x, torch.float16, "x")
        _require(y, torch.float32, "y")
        arr[i] = _Desc(t, _ptr(W), W.shape[0], K, _ptr(x), _ptr(y))
    ws_ptr, ws_bytes = (workspace.ptr, workspace.nbytes) if workspace is not None else (None, 0)
    _check(lib().pn_gemv_layer_ex(arr, len(entries), M, ws_ptr, ws_bytes, algo, _stream(stream)),
           "pn_gemv_layer")
    return [e[4] for e in entries]


def gemv_hadamard(pn_type: int, W: torch.Tensor, K: int, x: torch.Tensor, block: int,
                  y: torch.Tensor | None = None, workspace: Workspace | None = None, stream=None) -> torch.Tensor:
    """y = decode(W) @ hadamard(x, block)^T in one launch (see pn_gemv_hadamard)."""
    _require(W, torch.uint8, "W")
    _require(x, torch.float16, "x")
    if x.dim() == 1:
        x = x.view(1, -1)
    M, N = x.shape[0], W.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=W.device)
    _require(y, torch.float32, "y")
    ws_ptr, ws_bytes = (workspace.ptr, workspace.nbytes) if workspace is not None else (None, 0)
    _check(lib().pn_gemv_hadamard(pn_type, _ptr(W), N, K, _ptr(x), M, block, _ptr(y), ws_ptr, ws_bytes,
                                  _stream(stream)), "pn_gemv_hadamard")
    return y


class LayerCall:
    """The marshalled arguments of one layer call (pn_gemv_layer /
    pn_gemv_layer_host) over fixed buffers, built once and reused: a serving
    loop that calls with the same tensors every step pays one ctypes call per
    step.  The entries' tensors are kept alive by this object."""

    def __init__(self, entries, M: int, workspace: Workspace):
        self.entries = list(entries)
        self.M = M
        self.workspace = workspace
        self._arr = (_Desc * len(self.entries))()
        for i, (t, W, K, x, y) in enumerate(self.entries):
            _require(W, torch.uint8, "W")
            _require(x, torch.float16, "x")
            _require(y, torch.float32, "y")
            self._arr[i] = _Desc(t, _ptr(W), W.shape[0], K, _ptr(x), _ptr(y))
        self._n = len(self.entries)
        self.x_elems = sum(M * K for _, _, K, _, _ in self.entries)
        self.y_elems = sum(M * W.shape[0] for _, W, _, _, _ in self.entries)

    def device(self, stream=None) -> None:
        """pn_gemv_layer on the entries' device buffers (enqueued on `stream`)."""
        _check(lib().pn_gemv_layer(self._arr, self._n, self.M, self.workspace.ptr, self.workspace.nbytes,
                                   _stream(stream)), "pn_gemv_layer")

    def host(self, x_host: torch.Tensor, y_host: torch.Tensor, stream=None) -> torch.Tensor:
        """pn_gemv_layer_host: x from host memory, y back to it; returns when
        y_host is written."""
        if x_host.is_cuda or y_host.is_cuda or x_host.dtype != torch.float16 or y_host.dtype != torch.float32:
            raise TypeError("x_host must be a CPU float16 tensor and y_host a CPU float32 tensor")
        if not (x_host.is_contiguous() and y_host.is_contiguous()):
            raise ValueError("host buffers must be contiguous")
        if x_host.numel() < self.x_elems or y_host.numel() < self.y_elems:
            raise ValueError("host buffers are too small")
        _check(lib().pn_gemv_layer_host(self._arr, self._n, self.M, x_host.data_ptr(), y_host.data_ptr(),
                                        self.workspace.ptr, self.workspace.nbytes, _stream(stream)),
               "pn_gemv_layer_host")
        return y_host


def gemv_layer_host(entries, M: int, x_host: torch.Tensor, y_host: torch.Tensor, workspace: Workspace,
                    stream=None) -> torch.Tensor:
    """pn_gemv_layer_host: x from host memory (every entry's x [M][K] in
    order, fp16), the GEMVs, y back to host memory (fp32), in one call that
    returns when y_host is written.  (LayerCall keeps the marshalled
    arguments for repeated calls.)"""
    return LayerCall(entries, M, workspace).host(x_host, y_host, stream)


def gemv_layer_hadamard(entries, M: int, block: int, workspace: Workspace | None = None, stream=None):
    """Several independent GEMVs on rotated activations in one launch (see pn_gemv_layer_hadamard)."""
    entries = list(entries)
    arr = (_Desc * len(entries))()
    for i, (t, W, K, x, y) in enumerate(entries):
        _require(W, torch.uint8, "W")
        _require(x, torch.float16, "x")
        _require(y, torch.float32, "y")
        arr[i] = _Desc(t, _ptr(W), W.shape[0], K, _ptr(x), _ptr(y))
    ws_ptr, ws_bytes = (workspace.ptr, workspace.nbytes) if workspace is not None else (None, 0)
    _check(lib().pn_gemv_layer_hadamard(arr, len(entries), M, block, ws_ptr, ws_bytes, _stream(stream)),
           "pn_gemv_layer_hadamard")
    return [e[4] for e in entries]


def gptq(pn_type: int, w: torch.Tensor, X: torch.Tensor, damp: float = 0.01, stream=None) -> torch.Tensor:
    """GPTQ-style quantisation (see pn_gptq): fp32 w [N][K] and calibration
    inputs X fp32 [n][K] -> PN rows [N][row_bytes].  Synchronous."""
    _require(w, torch.float32, "w")
    _require(X, torch.float32, "X")
    N, K = w.shape
    if X.dim() != 2 or X.shape[1] != K:
        raise ValueError("X must be [n][K]")
    rb = row_bytes(pn_type, K)
    if rb == 0:
        raise ValueError("K is not a whole number of blocks")
    W = torch.empty((N, rb), dtype=torch.uint8, device=w.device)
    nbytes = int(lib().pn_gptq_scratch_bytes(N, K))
    scratch = torch.empty(nbytes + 256, dtype=torch.uint8, device=w.device)
    base = (scratch.data_ptr() + 255) // 256 * 256
    _check(lib().pn_gptq(pn_type, _ptr(w), N, K, _ptr(X), X.shape[0], float(damp), _ptr(W), base, nbytes,
                         _stream(stream)), "pn_gptq")
    return W


def hadamard(x: torch.Tensor, block: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Block Hadamard rotation of fp16 activations [M][K] (see pn_hadamard)."""
    _require(x, torch.float16, "x")
    if x.dim() == 1:
        x = x.view(1, -1)
    M, K = x.shape
    if out is None:
        out = torch.empty_like(x)
    _require(out, torch.float16, "out")
    _check(lib().pn_hadamard(_ptr(x), M, K, block, _ptr(out), _stream(stream)), "pn_hadamard")
    return out


def unpack_f16(pn_type: int, W: torch.Tensor, K: int, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """PN rows uint8 [N][row_bytes] -> fp16 weights [N][K] (exact decode, one rounding)."""
    _require(W, torch.uint8, "W")
    N = W.shape[0]
    if out is None:
        out = torch.empty((N, K), dtype=torch.float16, device=W.device)
    _require(out, torch.float16, "out")
    _check(lib().pn_unpack_f16(pn_type, _ptr(W), N, K, _ptr(out), _stream(stream)), "pn_unpack_f16")
    return out


def gemm_f16(w16: torch.Tensor, x: torch.Tensor, y: torch.Tensor | None = None,
             workspace: Workspace | None = None, stream=None) -> torch.Tensor:
    """y[M][N] = x[M][K] @ w16[N][K]^T, fp16 products, fp32 accumulation (tcgen05)."""
    _require(w16, torch.float16, "w16")
    _require(x, torch.float16, "x")
    N, K = w16.shape
    M = x.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=w16.device)
    _require(y, torch.float32, "y")
    if workspace is None:
        workspace = Workspace(N, w16.device)
    _check(lib().pn_gemm_f16(_ptr(w16), N, K, _ptr(x), M, _ptr(y), y.shape[1], workspace.ptr,
                             workspace.nbytes, _stream(stream)), "pn_gemm_f16")
    return y


def prefill(pn_type: int, W: torch.Tensor, K: int, x: torch.Tensor, y: torch.Tensor | None = None,
            scratch: torch.Tensor | None = None, workspace: Workspace | None = None,
            stream=None) -> torch.Tensor:
    """y[M][N] for large M: PN rows rebuilt as fp16 chunk by chunk into
    ``scratch`` (default: room for every row), then the fp16 GEMM."""
    _require(W, torch.uint8, "W")
    _require(x, torch.float16, "x")
    N = W.shape[0]
    M = x.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=W.device)
    _require(y, torch.float32, "y")
    if scratch is None:
        rows = max(128, (N + 127) // 128 * 128)
        scratch = torch.empty(rows * K, dtype=torch.float16, device=W.device)
    _require(scratch, torch.float16, "scratch")
    if workspace is None:
        workspace = Workspace(N, W.device)
    _check(lib().pn_prefill(pn_type, _ptr(W), N, K, _ptr(x), M, _ptr(y), _ptr(scratch),
                            scratch.numel() * 2, workspace.ptr, workspace.nbytes, _stream(stream)),
           "pn_prefill")
    return y


# ------------------------------------------------- 4-bit cache, serving step --

_step_module = None


def _step():
    """The compiled entry of these calls (csrc/pn_step_binding.cpp): checks,
    outputs and the C call in one go."""
    global _step_module
    if _step_module is None:
        lib()                                        # a missing library is reported by its own name
        try:
            from bit_weight_only_pn_gb300 import _step as module
        except ImportError as e:
            raise RuntimeError("the Python entry of the serving-step calls is not built; run "
                               "`python -m bit_weight_only_pn_gb300.build`") from e
        _step_module = module
    return _step_module


def _call(stream, function, what: str, *args):
    """function(*args) on `stream` (None: the current one), whose memory the outputs are taken from."""
    if stream is None:
        r = function(*args)
    else:
        with torch.cuda.stream(stream):
            r = function(*args)
    if r[0]:
        _check(r[0], what)
    return r


def kv_cache(pages: int, page_size: int, kv_heads: int, head_dim: int, device=None) -> torch.Tensor:
    """A zeroed 4-bit key/value cache (layout: include/pn.h, "4-bit cache"):
    uint8 [pages][kv_heads][page_size / 16][17 * head_dim]."""
    if lib().pn_kv_cache_bytes(pages, page_size, kv_heads, head_dim) == 0:
        raise ValueError("page_size must be a power of two from 16 to 1024 and head_dim 64, 128 or 256")
    return torch.zeros((pages, kv_heads, page_size // 16, 17 * head_dim), dtype=torch.uint8,
                       device=device if device is not None else "cuda")


class KvPlan(NamedTuple):
    """A step's bookkeeping (see pn_kv_plan).  Unless given as `out`, the eight share
    one allocation, which lasts as long as any of them: clone what is to outlive
    the slot maps (16 bytes a slot)."""
    slots: torch.Tensor         # int64 [capacity]: where each token goes in the cache, -1 nowhere
    positions: torch.Tensor     # int32 [capacity]: its position in its request, -1 none
    requests: torch.Tensor      # int32 [capacity]: its request, -1 behind the step's tokens
    starts: torch.Tensor        # int32 [batch + 1]: tokens before each request
    lens: torch.Tensor          # int32 [batch]: lengths after the step
    held: torch.Tensor          # int32 [batch]: pages held after the step
    ring: torch.Tensor          # int64 [2]: head and tail of the free pages after the step
    refused: torch.Tensor       # int32 [1]: requests that did not fit


def kv_plan(lens: torch.Tensor, add: torch.Tensor, held: torch.Tensor, table: torch.Tensor, free: torch.Tensor,
            ring: torch.Tensor, page_size: int, capacity: int, out: KvPlan | None = None, stream=None) -> KvPlan:
    """Pages and slots for a step's tokens, from the requests' lengths, on the
    device (see pn_kv_plan).  lens, add, held int32 [batch]; table int32
    [batch][pages per request] (new entries are written), free int32 [pages],
    ring int64 [2].  `out` is an earlier result to write into (its lens, held
    and ring must not be this call's inputs)."""
    return KvPlan(*_call(stream, _step().kv_plan, "pn_kv_plan", lens, add, held, table, free, ring, page_size, capacity,
                         out)[1:])


def kv_append(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, slots: torch.Tensor,
              positions: torch.Tensor | None = None, cos: torch.Tensor | None = None, sin: torch.Tensor | None = None,
              q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
              interleaved: bool = False, q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """Norms and rotation of queries and keys and the write of keys and values
    into the 4-bit cache (see pn_kv_append).  q [tokens][heads][D] (or None), k
    and v [tokens][kv_heads][D], all fp32 or all fp16, tokens at any stride;
    slots int64 [tokens]; positions int32 [tokens] choose the rows of cos and
    sin, fp32 [positions][rotated pairs] (None: no rotation).  Returns the
    queries as fp16 [tokens][heads][D]."""
    return _call(stream, _step().kv_append, "pn_kv_append", q, k, v, cache, slots, positions, cos, sin, q_weight,
                 k_weight, eps, interleaved, q_out)[1]


def kv_read(cache: torch.Tensor, slots: torch.Tensor, out=None, stream=None):
    """The cached keys and values of `slots` (int64), exactly: two fp32
    [tokens][kv_heads][D] tensors (`out`, if given)."""
    return _call(stream, _step().kv_read, "pn_kv_read", cache, slots, *(out if out is not None else (None, None)))[1:]


class AttentionWorkspace:
    """Zeroed device scratch for attention calls on one device (see pn_attention).
    Ready on return, whichever stream the calls run on: the constructor waits for
    its zeros (but not under graph capture, nor with wait=False, where the first
    call has to follow on the current stream)."""

    def __init__(self, device=None, wait: bool = True):
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        with torch.cuda.device(self.device):
            self.nbytes = int(lib().pn_attention_workspace_bytes())
            if self.nbytes == 0:
                raise PnError(4, "pn_attention_workspace_bytes")
            self.buffer = torch.zeros(self.nbytes, dtype=torch.uint8, device=self.device)
            if wait and not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()

    @property
    def ptr(self) -> int:
        return self.buffer.data_ptr()

    def status(self, stream=None) -> int:
        """Synchronise, read and clear the device status word (0 = ok)."""
        return int(lib().pn_workspace_status(self.ptr, self.nbytes, _stream(stream)))


def attention(q: torch.Tensor, cache: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, starts: torch.Tensor,
              max_queries: int, scale: float, window: int = 0, sinks: int = 0, out: torch.Tensor | None = None,
              lse: torch.Tensor | None = None, return_lse: bool = False, workspace: AttentionWorkspace | None = None,
              stream=None):
    """Attention of a step's queries over the 4-bit cache (see pn_attention).
    q fp16 [tokens][heads][D], tokens at any stride; table int32
    [batch][pages per request], lens int32 [batch] (the step's tokens
    included), starts int32 [batch + 1]; no request has more than max_queries
    queries.  window > 0: a query sees the last `window` tokens up to its own
    and the first `sinks`.  Returns out fp16 [tokens][heads][D], with
    return_lse (or a given lse) also fp32 [tokens][heads].  Without a workspace
    the call allocates and zeroes one (about 40 MB): a program keeps its own."""
    if workspace is None:
        with torch.cuda.stream(stream):              # zeroed, used and freed in the order of the stream that runs the call
            workspace = AttentionWorkspace(q.device, wait=False)
    _, out, lse = _call(stream, _step().attention, "pn_attention", q, cache, table, lens, starts, max_queries, scale,
                        window, sinks, out, lse, return_lse, workspace.buffer)
    return out if lse is None else (out, lse)


def verify(tokens: torch.Tensor, target: torch.Tensor, draft: torch.Tensor | None, uniforms: torch.Tensor,
           counts: torch.Tensor | None = None, accepted: torch.Tensor | None = None, out: torch.Tensor | None = None,
           stream=None):
    """Speculative verification (see pn_verify): drafted tokens int32
    [batch][drafts] against target probabilities fp32 [batch][drafts + 1][vocab]
    and the draft model's [batch][drafts][vocab] (None: certain drafts), with
    uniforms fp32 [batch][drafts + 1] in [0, 1).  Returns (accepted int32
    [batch], tokens int32 [batch][drafts + 1]: the accepted ones, one more, -1)."""
    return _call(stream, _step().verify, "pn_verify", tokens, target, draft, uniforms, counts, accepted, out)[1:]


class LogProbs(NamedTuple):
    """What pn.logprobs gives of rows of logits; None where it was not asked for.  The
    four share one allocation, which lasts as long as any of them."""
    logprobs: torch.Tensor      # fp32 [rows] or [rows][count]: log probabilities of the given tokens
    entropy: torch.Tensor       # fp32 [rows]
    top_tokens: torch.Tensor    # int32 [rows][top], -1 where fewer have a probability
    top_logprobs: torch.Tensor  # fp32 [rows][top]


def logprobs(logits: torch.Tensor, tokens: torch.Tensor | None = None, top: int = 0, scale: float = 1.0, entropy: bool = True,
             stream=None) -> LogProbs:
    """Log probabilities of given tokens (int32 [rows] or [rows][count]), the
    entropy and the `top` (at most 32) likeliest tokens of softmax(scale * logits),
    logits fp32 or fp16 [rows][vocab], rows at any stride (see pn_logprobs).  One
    read of the logits; ties go to the lowest token."""
    return LogProbs(*_call(stream, _step().logprobs, "pn_logprobs", logits, tokens, top, scale, entropy)[1:])


def norm(y: torch.Tensor | None, residual: torch.Tensor | None = None, gate: torch.Tensor | None = None, scale: float = 1.0,
         post: int = NORM_NONE, post_weight: torch.Tensor | None = None, post_bias: torch.Tensor | None = None, pre: int = NORM_RMS,
         pre_weight: torch.Tensor | None = None, pre_bias: torch.Tensor | None = None, eps: float = 1e-6,
         residual_out: torch.Tensor | None = None, x: torch.Tensor | None = None, want_residual: bool | None = None, want_x: bool = True,
         stream=None):
    """A block's output into the residual stream and the next GEMV's input, in one
    pass (see pn_norm): r' = residual + scale * gate * post(y), x = pre(r') as fp16.
    y, residual [tokens][hidden] fp32 or fp16 at any row stride (one may be None);
    gate fp32 [hidden] or [tokens][hidden]; post, pre NORM_NONE, NORM_RMS or
    NORM_LAYER with fp32 weights and biases.  Returns (r' in residual's type, x);
    residual_out may be `residual`.  want_residual: None stands for "if there is a y";
    what is not wanted is None (and pre is then left out with x)."""
    if want_residual is None:
        want_residual = y is not None
    if not want_x and x is None:
        pre, pre_weight, pre_bias = NORM_NONE, None, None
    return _call(stream, _step().norm, "pn_norm", y, residual, gate, scale, post, post_weight, post_bias, pre, pre_weight, pre_bias, eps,
                 residual_out, x, want_residual, want_x)[1:]


def kv_weights(cache: torch.Tensor) -> torch.Tensor:
    """Zeroed weights for the tokens of a 4-bit cache: fp32 [pages][kv_heads][page_size]."""
    return torch.zeros(cache.shape[0], cache.shape[1], cache.shape[2] * 16, device=cache.device)


def kv_weigh(q: torch.Tensor, cache: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, starts: torch.Tensor, max_queries: int,
             lse: torch.Tensor, scale: float, weights: torch.Tensor | None = None, decay: float = 1.0, out: torch.Tensor | None = None,
             window: int = 0, sinks: int = 0, stream=None, workspace: AttentionWorkspace | Workspace | None = None) -> torch.Tensor:
    """The attention weight that each cached token gathered from a step's queries
    (see pn_kv_weigh): arguments as of the attention call before it, and the lse
    that it returned.  Added to decay times `weights` (the step's own tokens begin
    at zero; None: all do) and written to `out` (None: into `weights`; both None:
    new zeroed ones).  With a workspace (the attention call's, say) its status()
    tells of a wait on the GPU that gave up, which else shows as NaN alone."""
    if weights is None and out is None:
        with torch.cuda.stream(stream):              # zeroed in the order of the stream that runs the call
            out = kv_weights(cache)
    return _call(stream, _step().kv_weigh, "pn_kv_weigh", q, cache, table, lens, starts, max_queries, lse, scale, weights, decay, out, window, sinks,
                 None if workspace is None else workspace.buffer)[1]


class KvEviction(NamedTuple):
    """The state after pn.kv_evict.  lens, held, ring and refused share one allocation
    (unless given as `out`)."""
    table: torch.Tensor         # int32 [batch][pages per request]: pages of a request cut back, then -1; others as they were
    lens: torch.Tensor          # int32 [batch]
    held: torch.Tensor          # int32 [batch]
    ring: torch.Tensor          # int64 [2]
    kept: torch.Tensor          # int32 [batch][kv_heads][budget]: the positions kept, -1 for a request left alone
    refused: torch.Tensor       # int32 [1]: requests past the limit that found no pages


def kv_evict(cache: torch.Tensor, weights: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, held: torch.Tensor, free: torch.Tensor,
             ring: torch.Tensor, limit: int, budget: int, sinks: int = 0, recent: int = 0, out: KvEviction | None = None,
             stream=None) -> KvEviction:
    """Requests with more than `limit` cached tokens keep `budget` of them, each head
    its first `sinks`, its last `recent` and those of the largest weight between, in
    pages from the free ring; their old pages are given back (see pn_kv_evict).  The
    positions of later tokens go on from the old length: add lens - result.lens to
    those that kv_plan gives from then on.  Layers that share table and ring have a
    call each, all on the state before the first.  `out` is an earlier result to write
    into."""
    return KvEviction(*_call(stream, _step().kv_evict, "pn_kv_evict", cache, weights, table, lens, held, free, ring, limit, budget, sinks, recent,
                             out)[1:])


def read_ranges(tensors, sink: torch.Tensor, stream=None) -> torch.Tensor:
    """Diagnostic read-bandwidth probe (see pn_read_ranges): reads every
    tensor's bytes once and XORs its 32-bit words into sink[i] (int32 device
    tensor with one element per tensor)."""
    tensors = list(tensors)
    n = len(tensors)
    ptrs = (ctypes.c_void_p * n)(*[t.data_ptr() for t in tensors])
    sizes = (ctypes.c_size_t * n)(*[t.numel() * t.element_size() for t in tensors])
    _require(sink, torch.int32, "sink")
    _check(lib().pn_read_ranges(ptrs, sizes, n, sink.data_ptr(), _stream(stream)), "pn_read_ranges")
    return sink


def set_wait_timeout_ns(ns: int) -> None:
    lib().pn_set_wait_timeout_ns(int(ns))


def set_test_stall(on: bool) -> None:
    lib().pn_set_test_stall(1 if on else 0)


def tc_split(shapes, M: int, num_sms: int) -> list[int]:
    """Testing aid (host only, see pn_tc_split): the unit ranges the
    tensor-core GEMV would give its thread blocks for tensors ``shapes`` =
    [(pn_type, N, K), ...] at M tokens on num_sms SMs; returns starts, with
    block c taking units [starts[c], starts[c + 1])."""
    shapes = list(shapes)
    n = len(shapes)
    types = (ctypes.c_int * n)(*[s[0] for s in shapes])
    Ns = (ctypes.c_int64 * n)(*[s[1] for s in shapes])
    Ks = (ctypes.c_int64 * n)(*[s[2] for s in shapes])
    starts = (ctypes.c_uint32 * (max(num_sms, 1) + 1))()
    grid = ctypes.c_int(0)
    _check(lib().pn_tc_split(types, Ns, Ks, n, M, num_sms, starts, ctypes.byref(grid)), "pn_tc_split")
    return list(starts[: grid.value + 1])
