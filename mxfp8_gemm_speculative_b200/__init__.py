"""Python binding of libmxg.so: weight-quantized linear layer on B200, the
adapters beside it and the sampler behind its head.

    Y[M][N] = X[M][K] * dequant(W)^T     bf16 activations, fp32 accumulate, bf16 out

with GPTQ-style symmetric INT4 weights (``w4a16_*``) or MXFP8 weights
(``mxfp8_*``).  Every function here only marshals arguments into the C ABI
declared in ``include/mxg.h`` (same names); all computation runs in the
library's CUDA kernels.  PyTorch provides device memory and the current
stream.  There is no CPU fallback: importing this module raises if the
compiled library is missing.

Workspace: the GEMMs need a caller-owned, zero-initialised workspace that
they leave zeroed.  The functions below keep one per (device, stream) and
grow it on demand; pass ``workspace=`` to manage it yourself.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmxg.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`"
        " (nvcc, sm_100a). There is no fallback implementation.")

_lib = ctypes.CDLL(LIB_PATH)

_p = ctypes.c_void_p
_i = ctypes.c_int
_sz = ctypes.c_size_t
_ll = ctypes.c_longlong

_SIGS = {
    "mxg_status_string": (ctypes.c_char_p, [_i]),
    "w4a16_packed_bytes": (_sz, [_i, _i, _i]),
    "w4a16_repack": (_i, [_p, _p, _i, _i, _i, _p, _p]),
    "w4a16_repack_ct": (_i, [_p, _p, _i, _i, _i, _p, _p]),
    "w4a16_repack_fused": (_i, [_i, _p, _p, _p, _i, _i, _p, _p]),
    "w4a16_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "w4a16_gemm": (_i, [_p, _p, _i, _i, _i, _i, _p, _p, _sz, _p]),
    "w4a16_gemm_ex": (_i, [_p, _p, _i, _i, _i, _i, _p, _p, _sz, _p, _p]),
    "w4a16_static_scratch_status": (_i, [ctypes.POINTER(_i), _i, _p]),
    "w4a16_gemm_static_scratch": (_i, [_p, _p, _i, _i, _i, _i, _p, _p]),
    "mxfp8_workspace_bytes": (_sz, [_i, _i, _i]),
    "mxfp8_gemm": (_i, [_p, _p, _p, _i, _i, _i, _p, _p, _sz, _p]),
    "mxfp8_gemm_ex": (_i, [_p, _p, _p, _i, _i, _i, _p, _p, _sz, _p, _p]),
    "mxfp8_packed_bytes": (_sz, [_i, _i]),
    "mxfp8_repack": (_i, [_p, _p, _i, _i, _p, _p]),
    "mxfp8_packed_workspace_bytes": (_sz, [_i, _i, _i]),
    "mxfp8_gemm_packed": (_i, [_p, _p, _i, _i, _i, _p, _p, _sz, _p]),
    "mxfp8_gemm_packed_ex": (_i, [_p, _p, _i, _i, _i, _p, _p, _sz, _p, _p]),
    "w4a16_unpack": (_i, [_p, _i, _i, _i, _p, _p, _p, _p]),
    "mxfp8_dequant": (_i, [_p, _p, _i, _i, _p, _p]),
    "mxg_workspace_status": (_i, [_p, ctypes.POINTER(_i), _p]),
    "mxg_selftest_wait_timeout": (_i, [_p, _i, _p]),
    "mxg_selftest_stream_ring": (_i, [_i, _i, _i, _i, _i, _i, _i, _p, _p]),
    "w8a16_packed_bytes": (_sz, [_i, _i, _i]),
    "w8a16_repack": (_i, [_p, _p, _i, _i, _i, _p, _p]),
    "w8a16_repack_ct": (_i, [_p, _p, _i, _i, _i, _p, _p]),
    "w8a16_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "w8a16_gemm": (_i, [_p, _p, _i, _i, _i, _i, _p, _p, _sz, _p]),
    "w8a16_gemm_ex": (_i, [_p, _p, _i, _i, _i, _i, _p, _p, _sz, _p, _p]),
    "bf16_gemm_small_workspace_bytes": (_sz, [_i, _i, _i]),
    "bf16_gemm_small": (_i, [_p, _p, _i, _i, _i, _p, _p, _sz, _p]),
    "bf16_gemm_small_ex": (_i, [_p, _p, _i, _i, _i, _p, _p, _sz, _p, _p]),
    "lora_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "lora_add": (_i, [_p, _ll, _p, _p, _p, _p, _p, _ll, _p, _ll, _i, _i, _i, _i, _i, _p, _sz, _p]),
    "lora_status": (_i, [_p, _i, _p]),
    "mxg_selftest_lora_wait_timeout": (_i, [_i, _p]),
    "sample_logits": (_i, [_p, _i, _ll, _i, _i, _p, _p, _p, _p, _p, _p, _p, _p]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_SIGS)

MXG_OK = 0
MXG_ERR_INVALID_ARG = -1
MXG_ERR_UNSUPPORTED_SHAPE = -2
MXG_ERR_WORKSPACE = -3
MXG_ERR_CUDA = -4
MXG_ERR_TIMEOUT = -5
MXG_ERR_CAPTURE = -6

PATH_AUTO, PATH_STREAM, PATH_TENSOR = 0, 1, 2
DTYPE_BF16, DTYPE_FP32 = 0, 1


class GemmOptions(ctypes.Structure):
    """mxg_gemm_options of include/mxg.h: per-call path and weight-load
    timing."""
    _fields_ = [("path", ctypes.c_int), ("late_weights", ctypes.c_int)]


def _options(path: int = PATH_AUTO, late_weights: bool = False):
    """A pointer to the call's options, or None for the defaults.  The
    structure is kept alive by the returned pointer object."""
    if path == PATH_AUTO and not late_weights:
        return None
    return ctypes.pointer(GemmOptions(int(path), 1 if late_weights else 0))


class MxgError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {mxg_status_string(status)} (status {status})")
        self.status = status


def mxg_status_string(status: int) -> str:
    return _lib.mxg_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != MXG_OK:
        raise MxgError(status, what)


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The handle of a device's current stream without a Stream object around it
# (2 us less per call), where this torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)   # the current device's index


def _stream(stream=None, device=None):
    """The CUDA stream handle a call runs on: ``stream``, which must live on
    ``device``, or that device's current stream."""
    if stream is None:
        if _raw_stream is not None and device is not None and device.index is not None:
            return _raw_stream(device.index)
        s = torch.cuda.current_stream(device)
    else:
        s = stream
        sdev = getattr(s, "device", None)
        if device is not None and sdev is not None and torch.device(sdev) != torch.device(device):
            raise ValueError(f"stream is on {sdev}, the call's tensors on {device}")
    return ctypes.c_void_p(s.cuda_stream)


_HERE_ALREADY = contextlib.nullcontext()


def _on_device(device):
    """Makes ``device`` current for a C call: the library plans and launches
    on the current device (its SM count, its kernels, its static scratch)."""
    if torch.cuda.current_device() == device.index:
        return _HERE_ALREADY
    return torch.cuda.device(device)


def _dev_call(device, what: str, fn, *args, stream=None) -> None:
    """fn(*args, stream handle) with ``device`` current; raises on a nonzero
    status."""
    if (stream is None and _raw_device is not None and _raw_stream is not None
            and device.type == "cuda" and device.index == _raw_device()):
        status = fn(*args, _raw_stream(device.index))   # the same, 1 us less
    else:
        with _on_device(device):
            status = fn(*args, _stream(stream, device))
    if status != MXG_OK:
        raise MxgError(status, what)


def _need(t: torch.Tensor, dtype, name: str) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# The C ABI takes plain pointers and cannot see buffer sizes: the binding
# checks every buffer a kernel reads or writes against the call's shape
# (type, then size, then layout and device), so a mismatch raises here
# instead of reaching memory past the end of a tensor.
def _same_device(t: torch.Tensor, device, name: str) -> None:
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _need_out(out: torch.Tensor, M: int, N: int, device) -> None:
    if out.dtype != torch.bfloat16:
        raise ValueError(f"out must be torch.bfloat16, got {out.dtype}")
    if tuple(out.shape) != (M, N):
        raise ValueError(f"out must be [{M}][{N}], got {list(out.shape)}")
    _need(out, torch.bfloat16, "out")
    _same_device(out, device, "out")


def _need_weights(t: torch.Tensor, dtype, nbytes: int, device, name: str) -> None:
    """t holds at least nbytes bytes of weights (nbytes = 0: a shape the
    library rejects itself, with its own status)."""
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if nbytes and t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes, the shape needs "
                         f"{nbytes}")
    _need(t, dtype, name)
    _same_device(t, device, name)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """An uninitialised tensor for a result the library writes on `stream`:
    allocated on that stream, so its memory, once freed, is reused only
    behind the work already queued there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _need_shape(t: torch.Tensor, shape, name: str) -> None:
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _need_ws(ws: torch.Tensor, device) -> None:
    if ws.dtype != torch.uint8:
        raise ValueError(f"workspace_buf must be torch.uint8, got {ws.dtype}")
    _need(ws, torch.uint8, "workspace_buf")
    _same_device(ws, device, "workspace_buf")


def _gemm_buffers(x: torch.Tensor, K: int, N: int, out, workspace_buf, need_ws, stream):
    """(M, out, ws) for a GEMM on x [M][K]: `out` and `workspace_buf` checked,
    or made (a [M][N] bf16 output; the cached workspace of `need_ws()`
    bytes)."""
    _need(x, torch.bfloat16, "x")
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"x must be [M][{K}], got {list(x.shape)}")
    M = x.shape[0]
    if out is None:
        out = _empty((M, N), torch.bfloat16, x.device, stream)
    _need_out(out, M, N, x.device)
    if workspace_buf is None:
        ws = workspace(need_ws(), x.device, stream)
    else:
        ws = workspace_buf
        _need_ws(ws, x.device)
    return M, out, ws


# ------------------------------------------------------------- workspaces
_ws_lock = threading.Lock()
_ws_cache: dict[tuple[int, int], torch.Tensor] = {}


def workspace(nbytes: int, device=None, stream=None) -> torch.Tensor:
    """A zero-filled uint8 workspace of at least ``nbytes`` for (device, stream).
    It is allocated and zeroed on that stream, so the zero fill is ordered
    before the stream's next kernel, and the memory of a workspace it
    replaces goes back to that stream's pool (reused only behind the calls
    already queued there)."""
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else
                       torch.device(device).index)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    key = (dev.index, s.cuda_stream)
    with _ws_lock:
        ws = _ws_cache.get(key)
        if ws is None or ws.numel() < nbytes:
            with torch.cuda.stream(s):
                ws = torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=dev)
            _ws_cache[key] = ws
        return ws


@functools.lru_cache(maxsize=4096)
def _need_bytes(kind: str, device: int, M: int, N: int, K: int, G: int = 0) -> int:
    """Workspace size query, cached per (device, shape); the size depends on
    the device's SM count, so the query runs with that device current."""
    with torch.cuda.device(device):
        if kind == "w4a16":
            return int(_lib.w4a16_workspace_bytes(M, N, K, G))
        return int(_lib.mxfp8_workspace_bytes(M, N, K))


# -------------------------------------------------------------------- INT4
def w4a16_packed_bytes(K: int, N: int, group_size: int = 128) -> int:
    return int(_lib.w4a16_packed_bytes(K, N, group_size))


def _repack_out(words: torch.Tensor, K: int, N: int, group_size: int, out, what: str,
                stream=None):
    nbytes = w4a16_packed_bytes(K, N, group_size)
    if nbytes == 0:
        raise MxgError(MXG_ERR_UNSUPPORTED_SHAPE, what)
    if out is None:
        return _empty(nbytes, torch.uint8, words.device, stream)
    _need(out, torch.uint8, "out")
    if out.numel() != nbytes or out.device != words.device:
        raise ValueError(f"out must hold {nbytes} bytes on {words.device}")
    return out


def _need_scales(scales: torch.Tensor, name: str) -> None:
    if scales.dtype not in (torch.float16, torch.int16):
        raise ValueError(f"{name} must be float16 (or its int16 bit view)")
    _need(scales, scales.dtype, name)


def w4a16_repack(qweight: torch.Tensor, scales: torch.Tensor, group_size: int = 128,
                 stream=None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Re-pack GPTQ words qweight[K/8][N] (int32) and scales[K/G][N] (fp16),
    into `out` (uint8, w4a16_packed_bytes bytes) when given."""
    _need(qweight, torch.int32, "qweight")
    _need_scales(scales, "scales")
    K = qweight.shape[0] * 8
    N = qweight.shape[1]
    packed = _repack_out(qweight, K, N, group_size, out, "w4a16_repack", stream)
    _need_shape(scales, (K // group_size, N), "scales")
    _same_device(scales, qweight.device, "scales")
    _dev_call(qweight.device, "w4a16_repack", _lib.w4a16_repack, _ptr(qweight), _ptr(scales), K, N,
              group_size, _ptr(packed), stream=stream)
    return packed


def w4a16_repack_ct(weight_packed: torch.Tensor, weight_scale: torch.Tensor,
                    group_size: int = 128, stream=None,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """Re-pack compressed-tensors words weight_packed[N][K/8] (int32) and
    weight_scale[N][K/G] (fp16) into the same buffer w4a16_repack makes."""
    _need(weight_packed, torch.int32, "weight_packed")
    _need_scales(weight_scale, "weight_scale")
    N = weight_packed.shape[0]
    K = weight_packed.shape[1] * 8
    packed = _repack_out(weight_packed, K, N, group_size, out, "w4a16_repack_ct", stream)
    _need_shape(weight_scale, (N, K // group_size), "weight_scale")
    _same_device(weight_scale, weight_packed.device, "weight_scale")
    _dev_call(weight_packed.device, "w4a16_repack_ct", _lib.w4a16_repack_ct, _ptr(weight_packed),
              _ptr(weight_scale), K, N, group_size, _ptr(packed), stream=stream)
    return packed


def w4a16_repack_fused(parts, group_size: int = 128, stream=None,
                       out: torch.Tensor | None = None) -> torch.Tensor:
    """One re-packed buffer for projections that share their input: `parts`
    is a sequence of GPTQ (qweight[K/8][Ni], scales[K/G][Ni]) pairs with the
    same K; the fused layer has N = sum Ni columns, part i's in order."""
    parts = list(parts)
    if not parts:
        raise ValueError("parts must not be empty")
    for qw, sc in parts:
        _need(qw, torch.int32, "qweight")
        _need_scales(sc, "scales")
    K = parts[0][0].shape[0] * 8
    if any(qw.shape[0] * 8 != K for qw, _ in parts):
        raise ValueError("every part must have the same K")
    Ns = [int(qw.shape[1]) for qw, _ in parts]
    packed = _repack_out(parts[0][0], K, sum(Ns), group_size, out, "w4a16_repack_fused", stream)
    for i, (qw, sc) in enumerate(parts):
        _need_shape(sc, (K // group_size, Ns[i]), f"scales of part {i}")
        _same_device(qw, packed.device, f"qweight of part {i}")
        _same_device(sc, packed.device, f"scales of part {i}")
    n = len(parts)
    qptrs = (ctypes.c_void_p * n)(*[qw.data_ptr() for qw, _ in parts])
    sptrs = (ctypes.c_void_p * n)(*[sc.data_ptr() for _, sc in parts])
    narr = (ctypes.c_int * n)(*Ns)
    _dev_call(packed.device, "w4a16_repack_fused", _lib.w4a16_repack_fused, n, qptrs, sptrs, narr,
              K, group_size, _ptr(packed), stream=stream)
    return packed


def w4a16_workspace_bytes(M: int, N: int, K: int, group_size: int = 128) -> int:
    return int(_lib.w4a16_workspace_bytes(M, N, K, group_size))


def w4a16_gemm(x: torch.Tensor, packed: torch.Tensor, N: int, K: int, group_size: int = 128,
               out: torch.Tensor | None = None, workspace_buf: torch.Tensor | None = None,
               stream=None, path: int = PATH_AUTO, late_weights: bool = False) -> torch.Tensor:
    """Y = x * dequant(W)^T for x bf16 [M][K] and a re-packed INT4 weight.
    ``path`` forces the weight-streaming (1) or tensor-core (2) path;
    ``late_weights`` makes the kernel load weights only after the previous
    kernel on the stream (for weights that kernel writes)."""
    M, out, ws = _gemm_buffers(
        x, K, N, out, workspace_buf,
        lambda: _need_bytes("w4a16", x.device.index, x.shape[0], N, K, group_size), stream)
    _need_weights(packed, torch.uint8, w4a16_packed_bytes(K, N, group_size), x.device, "packed")
    _dev_call(x.device, "w4a16_gemm", _lib.w4a16_gemm_ex, _ptr(x), _ptr(packed), M, N, K,
              group_size, _ptr(out), _ptr(ws), ws.numel(), _options(path, late_weights),
              stream=stream)
    return out


class PreparedCall:
    """One library call with its arguments marshalled once, for a loop that
    repeats it on the same buffers (a serving step).  The tensors are held
    here so they stay alive; their contents may change between calls, their
    storage must not move."""

    def __init__(self, fn, args, what: str, keep, device):
        self._fn, self._args, self._what, self._keep = fn, tuple(args), what, keep
        self._device = device

    def __call__(self) -> None:
        with _on_device(self._device):
            status = self._fn(*self._args)
        if status != MXG_OK:
            raise MxgError(status, self._what)


def prepare_w4a16_gemm(x: torch.Tensor, packed: torch.Tensor, N: int, K: int,
                       group_size: int = 128, out: torch.Tensor | None = None,
                       workspace_buf: torch.Tensor | None = None, stream=None,
                       path: int = PATH_AUTO, late_weights: bool = False):
    """(call, out): ``call()`` runs w4a16_gemm(x, packed) into ``out``."""
    M, out, ws = _gemm_buffers(
        x, K, N, out, workspace_buf,
        lambda: _need_bytes("w4a16", x.device.index, x.shape[0], N, K, group_size), stream)
    _need_weights(packed, torch.uint8, w4a16_packed_bytes(K, N, group_size), x.device, "packed")
    args = (_ptr(x), _ptr(packed), M, N, K, group_size, _ptr(out), _ptr(ws), ws.numel(),
            _options(path, late_weights), _stream(stream, x.device))
    return PreparedCall(_lib.w4a16_gemm_ex, args, "w4a16_gemm", (x, packed, out, ws, stream),
                        x.device), out


def prepare_mxfp8_gemm(x: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor,
                       out: torch.Tensor | None = None, workspace_buf: torch.Tensor | None = None,
                       stream=None, path: int = PATH_AUTO, late_weights: bool = False):
    """(call, out): ``call()`` runs mxfp8_gemm(x, wq, ws) into ``out``."""
    M, K, N = _mx_shapes(x, wq, ws)
    M, out, wsb = _gemm_buffers(x, K, N, out, workspace_buf,
                                lambda: _need_bytes("mxfp8", x.device.index, M, N, K), stream)
    args = (_ptr(x), _ptr(wq), _ptr(ws), M, N, K, _ptr(out), _ptr(wsb), wsb.numel(),
            _options(path, late_weights), _stream(stream, x.device))
    return PreparedCall(_lib.mxfp8_gemm_ex, args, "mxfp8_gemm", (x, wq, ws, out, wsb, stream),
                        x.device), out


def prepare_bf16_gemm_small(x: torch.Tensor, w: torch.Tensor, out: torch.Tensor | None = None,
                            workspace_buf: torch.Tensor | None = None, stream=None,
                            late_weights: bool = False):
    """(call, out): ``call()`` runs bf16_gemm_small(x, w) into ``out``."""
    M, K, N, need = _small_shapes(x, w)
    M, out, wsb = _gemm_buffers(x, K, N, out, workspace_buf, lambda: need, stream)
    args = (_ptr(x), _ptr(w), M, N, K, _ptr(out), _ptr(wsb), wsb.numel(),
            _options(PATH_AUTO, late_weights), _stream(stream, x.device))
    return PreparedCall(_lib.bf16_gemm_small_ex, args, "bf16_gemm_small",
                        (x, w, out, wsb, stream), x.device), out


def w4a16_gemm_static_scratch(x: torch.Tensor, packed: torch.Tensor, N: int, K: int,
                              group_size: int = 128, out: torch.Tensor | None = None,
                              stream=None) -> torch.Tensor:
    """w4a16_gemm (M <= 32) with the library's fixed device scratch instead of a workspace."""
    _need(x, torch.bfloat16, "x")
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"x must be [M][{K}], got {list(x.shape)}")
    M = x.shape[0]
    if out is None:
        out = _empty((M, N), torch.bfloat16, x.device, stream)
    _need_out(out, M, N, x.device)
    _need_weights(packed, torch.uint8, w4a16_packed_bytes(K, N, group_size), x.device, "packed")
    _dev_call(x.device, "w4a16_gemm_static_scratch", _lib.w4a16_gemm_static_scratch, _ptr(x),
              _ptr(packed), M, N, K, group_size, _ptr(out), stream=stream)
    return out


def w4a16_unpack(packed: torch.Tensor, K: int, N: int, group_size: int = 128, stream=None):
    """(codes uint8 [N][K], w_fp32 float32 [N][K], w_bf16 bfloat16 [N][K])."""
    dev = packed.device
    _need_weights(packed, torch.uint8, w4a16_packed_bytes(K, N, group_size), dev, "packed")
    codes = _empty((N, K), torch.uint8, dev, stream)
    w32 = _empty((N, K), torch.float32, dev, stream)
    w16 = _empty((N, K), torch.bfloat16, dev, stream)
    _dev_call(packed.device, "w4a16_unpack", _lib.w4a16_unpack, _ptr(packed), K, N, group_size,
              _ptr(codes), _ptr(w32), _ptr(w16), stream=stream)
    return codes, w32, w16


# ------------------------------------------------------------------- MXFP8
def _mx_shapes(x: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor):
    """(M, K, N) of x [M][K] against E4M3 wq [N][K] and E8M0 ws [N][K/32]."""
    _need(x, torch.bfloat16, "x")
    if wq.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise ValueError("wq must be uint8 or float8_e4m3fn")
    if ws.dtype not in (torch.uint8, torch.float8_e8m0fnu):
        raise ValueError("ws must be uint8 or float8_e8m0fnu")
    if x.dim() != 2 or wq.dim() != 2 or ws.dim() != 2:
        raise ValueError("x, wq and ws must be 2-D")
    M, K = x.shape
    N = wq.shape[0]
    if wq.shape[1] != K or ws.shape[0] != N or ws.shape[1] * 32 != K:
        raise ValueError("shape mismatch between x, wq and ws")
    _need(wq, wq.dtype, "wq")
    _need(ws, ws.dtype, "ws")
    _same_device(wq, x.device, "wq")
    _same_device(ws, x.device, "ws")
    return M, K, N


def mxfp8_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(_lib.mxfp8_workspace_bytes(M, N, K))


def mxfp8_gemm(x: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor,
               out: torch.Tensor | None = None, workspace_buf: torch.Tensor | None = None,
               stream=None, path: int = PATH_AUTO, late_weights: bool = False) -> torch.Tensor:
    """Y = x * dequant(W)^T for x bf16 [M][K], E4M3 codes wq[N][K], E8M0 ws[N][K/32]."""
    M, K, N = _mx_shapes(x, wq, ws)
    M, out, wsb = _gemm_buffers(x, K, N, out, workspace_buf,
                                lambda: _need_bytes("mxfp8", x.device.index, M, N, K), stream)
    _dev_call(x.device, "mxfp8_gemm", _lib.mxfp8_gemm_ex, _ptr(x), _ptr(wq), _ptr(ws), M, N, K,
              _ptr(out), _ptr(wsb), wsb.numel(), _options(path, late_weights), stream=stream)
    return out


def mxfp8_repack(wq: torch.Tensor, ws: torch.Tensor, stream=None) -> torch.Tensor:
    """Re-pack E4M3 wq[N][K] and E8M0 ws[N][K/32] for mxfp8_gemm_packed."""
    if wq.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise ValueError("wq must be uint8 or float8_e4m3fn")
    if ws.dtype not in (torch.uint8, torch.float8_e8m0fnu):
        raise ValueError("ws must be uint8 or float8_e8m0fnu")
    if wq.dim() != 2:
        raise ValueError("wq must be [N][K]")
    N, K = wq.shape
    nbytes = int(_lib.mxfp8_packed_bytes(N, K))
    if nbytes == 0:
        raise MxgError(MXG_ERR_UNSUPPORTED_SHAPE, "mxfp8_repack")
    _need_shape(ws, (N, K // 32), "ws")
    _need(wq, wq.dtype, "wq")
    _need(ws, ws.dtype, "ws")
    _same_device(ws, wq.device, "ws")
    packed = _empty(nbytes, torch.uint8, wq.device, stream)
    _dev_call(wq.device, "mxfp8_repack", _lib.mxfp8_repack, _ptr(wq), _ptr(ws), N, K,
              _ptr(packed), stream=stream)
    return packed


def _mxp_ws_bytes(M: int, N: int, K: int) -> int:
    need = int(_lib.mxfp8_packed_workspace_bytes(M, N, K))
    if need == 0:
        raise MxgError(MXG_ERR_UNSUPPORTED_SHAPE, "mxfp8_gemm_packed")
    return need


def mxfp8_packed_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(_lib.mxfp8_packed_workspace_bytes(M, N, K))


def mxfp8_gemm_packed(x: torch.Tensor, packed: torch.Tensor, N: int, K: int,
                      out: torch.Tensor | None = None, workspace_buf: torch.Tensor | None = None,
                      stream=None, late_weights: bool = False) -> torch.Tensor:
    """Y = x * dequant(W)^T for x bf16 [M][K] (M <= 16) and mxfp8_repack's buffer."""
    M, out, ws = _gemm_buffers(x, K, N, out, workspace_buf,
                               lambda: _mxp_ws_bytes(x.shape[0], N, K), stream)
    _need_weights(packed, torch.uint8, int(_lib.mxfp8_packed_bytes(N, K)), x.device, "packed")
    _dev_call(x.device, "mxfp8_gemm_packed", _lib.mxfp8_gemm_packed_ex, _ptr(x), _ptr(packed), M,
              N, K, _ptr(out), _ptr(ws), ws.numel(), _options(PATH_AUTO, late_weights),
              stream=stream)
    return out


def prepare_mxfp8_gemm_packed(x: torch.Tensor, packed: torch.Tensor, N: int, K: int,
                              out: torch.Tensor | None = None,
                              workspace_buf: torch.Tensor | None = None, stream=None,
                              late_weights: bool = False):
    """(call, out): ``call()`` runs mxfp8_gemm_packed(x, packed) into ``out``."""
    M, out, ws = _gemm_buffers(x, K, N, out, workspace_buf,
                               lambda: _mxp_ws_bytes(x.shape[0], N, K), stream)
    _need_weights(packed, torch.uint8, int(_lib.mxfp8_packed_bytes(N, K)), x.device, "packed")
    args = (_ptr(x), _ptr(packed), M, N, K, _ptr(out), _ptr(ws), ws.numel(),
            _options(PATH_AUTO, late_weights), _stream(stream, x.device))
    return PreparedCall(_lib.mxfp8_gemm_packed_ex, args, "mxfp8_gemm_packed",
                        (x, packed, out, ws, stream), x.device), out


def mxfp8_dequant(wq: torch.Tensor, ws: torch.Tensor, stream=None) -> torch.Tensor:
    """bf16 [N][K] weights of E4M3 wq[N][K] and E8M0 ws[N][K/32]."""
    if wq.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise ValueError("wq must be uint8 or float8_e4m3fn")
    if ws.dtype not in (torch.uint8, torch.float8_e8m0fnu):
        raise ValueError("ws must be uint8 or float8_e8m0fnu")
    if wq.dim() != 2:
        raise ValueError("wq must be [N][K]")
    N, K = wq.shape
    _need_shape(ws, (N, K // 32), "ws")
    _need(wq, wq.dtype, "wq")
    _need(ws, ws.dtype, "ws")
    _same_device(ws, wq.device, "ws")
    out = _empty((N, K), torch.bfloat16, wq.device, stream)
    _dev_call(wq.device, "mxfp8_dequant", _lib.mxfp8_dequant, _ptr(wq), _ptr(ws), N, K, _ptr(out),
              stream=stream)
    return out


# ------------------------------------------------------------- diagnostics
def _need_header(workspace_buf: torch.Tensor) -> None:
    """A workspace holding at least its 256-byte status header."""
    if workspace_buf.dtype != torch.uint8:
        raise ValueError(f"workspace_buf must be torch.uint8, got {workspace_buf.dtype}")
    if workspace_buf.numel() < 256:
        raise ValueError("workspace_buf must hold at least its 256-byte header")
    _need(workspace_buf, torch.uint8, "workspace_buf")


def mxg_workspace_status(workspace_buf: torch.Tensor, stream=None) -> int:
    _need_header(workspace_buf)
    v = ctypes.c_int(0)
    _dev_call(workspace_buf.device, "mxg_workspace_status", _lib.mxg_workspace_status,
              _ptr(workspace_buf), ctypes.byref(v), stream=stream)
    return v.value


def w8a16_repack(qweight: torch.Tensor, scales: torch.Tensor, group_size: int = 128,
                 stream=None) -> torch.Tensor:
    """Re-pack INT8 words qweight[K/4][N] (int32, 4 codes per word along K,
    zero point 128) and scales[K/G][N] (fp16)."""
    _need(qweight, torch.int32, "qweight")
    _need_scales(scales, "scales")
    K = qweight.shape[0] * 4
    N = qweight.shape[1]
    nbytes = int(_lib.w8a16_packed_bytes(K, N, group_size))
    if nbytes == 0:
        raise MxgError(MXG_ERR_UNSUPPORTED_SHAPE, "w8a16_repack")
    _need_shape(scales, (K // group_size, N), "scales")
    _same_device(scales, qweight.device, "scales")
    packed = _empty(nbytes, torch.uint8, qweight.device, stream)
    _dev_call(qweight.device, "w8a16_repack", _lib.w8a16_repack, _ptr(qweight), _ptr(scales), K, N,
              group_size, _ptr(packed), stream=stream)
    return packed


def w8a16_repack_ct(weight_packed: torch.Tensor, weight_scale: torch.Tensor,
                    group_size: int = 128, stream=None) -> torch.Tensor:
    """Re-pack the compressed-tensors INT8 export weight_packed[N][K/4]
    (int32) and weight_scale[N][K/G] (fp16) into the w8a16_repack buffer."""
    _need(weight_packed, torch.int32, "weight_packed")
    _need_scales(weight_scale, "weight_scale")
    N = weight_packed.shape[0]
    K = weight_packed.shape[1] * 4
    nbytes = int(_lib.w8a16_packed_bytes(K, N, group_size))
    if nbytes == 0:
        raise MxgError(MXG_ERR_UNSUPPORTED_SHAPE, "w8a16_repack_ct")
    _need_shape(weight_scale, (N, K // group_size), "weight_scale")
    _same_device(weight_scale, weight_packed.device, "weight_scale")
    packed = _empty(nbytes, torch.uint8, weight_packed.device, stream)
    _dev_call(weight_packed.device, "w8a16_repack_ct", _lib.w8a16_repack_ct, _ptr(weight_packed),
              _ptr(weight_scale), K, N, group_size, _ptr(packed), stream=stream)
    return packed


def _w8_ws_bytes(M: int, N: int, K: int, group_size: int) -> int:
    need = int(_lib.w8a16_workspace_bytes(M, N, K, group_size))
    if need == 0:
        raise MxgError(MXG_ERR_UNSUPPORTED_SHAPE, "w8a16_gemm")
    return need


def w8a16_gemm(x: torch.Tensor, packed: torch.Tensor, N: int, K: int, group_size: int = 128,
               out: torch.Tensor | None = None, workspace_buf: torch.Tensor | None = None,
               stream=None, late_weights: bool = False) -> torch.Tensor:
    """Y = x * dequant(W)^T for x bf16 [M][K] (M <= 32) and a re-packed INT8 weight."""
    M, out, ws = _gemm_buffers(x, K, N, out, workspace_buf,
                               lambda: _w8_ws_bytes(x.shape[0], N, K, group_size), stream)
    _need_weights(packed, torch.uint8, int(_lib.w8a16_packed_bytes(K, N, group_size)), x.device,
                  "packed")
    _dev_call(x.device, "w8a16_gemm", _lib.w8a16_gemm_ex, _ptr(x), _ptr(packed), M, N, K,
              group_size, _ptr(out), _ptr(ws), ws.numel(), _options(PATH_AUTO, late_weights),
              stream=stream)
    return out


def prepare_w8a16_gemm(x: torch.Tensor, packed: torch.Tensor, N: int, K: int,
                       group_size: int = 128, out: torch.Tensor | None = None,
                       workspace_buf: torch.Tensor | None = None, stream=None,
                       late_weights: bool = False):
    """(call, out): ``call()`` runs w8a16_gemm(x, packed) into ``out``."""
    M, out, ws = _gemm_buffers(x, K, N, out, workspace_buf,
                               lambda: _w8_ws_bytes(x.shape[0], N, K, group_size), stream)
    _need_weights(packed, torch.uint8, int(_lib.w8a16_packed_bytes(K, N, group_size)), x.device,
                  "packed")
    args = (_ptr(x), _ptr(packed), M, N, K, group_size, _ptr(out), _ptr(ws), ws.numel(),
            _options(PATH_AUTO, late_weights), _stream(stream, x.device))
    return PreparedCall(_lib.w8a16_gemm_ex, args, "w8a16_gemm", (x, packed, out, ws, stream),
                        x.device), out


def _small_shapes(x: torch.Tensor, w: torch.Tensor):
    """(M, K, N, workspace bytes) of x [M][K] against dense bf16 w [N][K]."""
    _need(x, torch.bfloat16, "x")
    _need(w, torch.bfloat16, "w")
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError("x must be [M][K] and w [N][K]")
    _same_device(w, x.device, "w")
    M, K = x.shape
    N = w.shape[0]
    need = int(_lib.bf16_gemm_small_workspace_bytes(M, N, K))
    if need == 0:
        raise MxgError(MXG_ERR_UNSUPPORTED_SHAPE, "bf16_gemm_small")
    return M, K, N, need


def bf16_gemm_small(x: torch.Tensor, w: torch.Tensor, out: torch.Tensor | None = None,
                    workspace_buf: torch.Tensor | None = None, stream=None,
                    late_weights: bool = False) -> torch.Tensor:
    """Y = x * w^T with dense bf16 w [N][K] (few columns, e.g. the paired
    48 + 48 GDN A/B projection) and x bf16 [M][K], M <= 8."""
    M, K, N, need = _small_shapes(x, w)
    M, out, ws = _gemm_buffers(x, K, N, out, workspace_buf, lambda: need, stream)
    _dev_call(x.device, "bf16_gemm_small", _lib.bf16_gemm_small_ex, _ptr(x), _ptr(w), M, N, K,
              _ptr(out), _ptr(ws), ws.numel(), _options(PATH_AUTO, late_weights),
              stream=stream)
    return out


# ------------------------------------------------------- low-rank adapters
# Calls of a few microseconds: the checks below take the pointer of an
# argument that is in order at once, and look for what is wrong only otherwise.
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _dense(t: torch.Tensor, dtype, shape, device, name: str) -> int:
    """The pointer of a contiguous tensor of this type and shape."""
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == device.index
            and t.is_contiguous()):
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        _need_shape(t, shape, name)
        _same_device(t, device, name)
        _need(t, dtype, name)
    return t.data_ptr()


def _need_cuda(t: torch.Tensor, name: str) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def _empty_as(t: torch.Tensor, dtype, stream) -> torch.Tensor:
    """_empty of a contiguous tensor's shape (half the host time)."""
    if stream is None:
        return torch.empty_like(t, dtype=dtype)
    with torch.cuda.stream(stream):
        return torch.empty_like(t, dtype=dtype)


def _need_rows(t: torch.Tensor, M: int, N: int, device, name: str) -> int:
    """The row stride of a bf16 [M][N] whose rows are contiguous."""
    if not (t.dtype is _BF16 and t.shape == (M, N) and t.get_device() == device.index):
        if t.dtype != _BF16:
            raise ValueError(f"{name} must be {_BF16}, got {t.dtype}")
        if t.shape != (M, N):
            raise ValueError(f"{name} must be [{M}][{N}], got {list(t.shape)}")
        _same_device(t, device, name)
    ld, one = t.stride()
    if one != 1 and N > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    if M == 1:
        return -(-N // 8) * 8      # one row: its stride says nothing
    return ld


def _overlap(a: torch.Tensor, b: torch.Tensor, lda: int, ldb: int) -> bool:
    """Do the [M][N] of two tensors (2 bytes an element) share memory?  Column
    ranges of one buffer with one row stride do not, when their columns
    differ."""
    M, N = a.shape
    pa, pb = a.data_ptr(), b.data_ptr()
    if pa >= pb + 2 * ((M - 1) * ldb + N) or pb >= pa + 2 * ((M - 1) * lda + N):
        return False
    if lda != ldb:
        return True
    d = (pa - pb) % (2 * lda)
    return d < 2 * N or 2 * lda - d < 2 * N


def _lora_args(x, a, b, index, y, scales, out, workspace_buf, stream):
    """The arguments of the C call, and the tensors behind them."""
    dev = x.device
    _need_cuda(x, "x")
    shape_a, shape_b, shape_x = a.shape, b.shape, x.shape
    if len(shape_a) != 3 or len(shape_b) != 3:
        raise ValueError("a must be [L][R][K] and b [L][N][R]")
    L, R, K = shape_a
    N = shape_b[1]
    if len(shape_x) != 2:
        raise ValueError(f"x must be [M][{K}], got {list(shape_x)}")
    M = shape_x[0]
    pa = _dense(a, _BF16, shape_a, dev, "a")
    pb = _dense(b, _BF16, (L, N, R), dev, "b")
    pi = _dense(index, _I32, (M,), dev, "index")
    ps = None if scales is None else _dense(scales, _F32, (L,), dev, "scales")
    ldx = _need_rows(x, M, K, dev, "x")
    ldy = _need_rows(y, M, N, dev, "y")
    need = _lora_bytes(M, N, K, R)
    if need == 0:
        raise MxgError(MXG_ERR_UNSUPPORTED_SHAPE, "lora_add")
    if out is None:
        if ldy == N and y.is_contiguous():
            out = torch.empty_like(y) if stream is None else _empty_as(y, _BF16, stream)
        else:
            out = _empty((M, N), _BF16, dev, stream)
        ldo = N
    else:
        ldo = _need_rows(out, M, N, dev, "out")
        same = out.data_ptr() == y.data_ptr() and ldo == ldy
        if not same and _overlap(out, y, ldo, ldy):
            raise ValueError("out must be y or not overlap it")
    if workspace_buf is None:
        # this call's own, from the stream's pool: calls captured into
        # different graphs never share it
        if stream is None:
            ws = torch.empty_strided((need,), (1,), dtype=_U8, device=dev)
        else:
            ws = _empty((need,), _U8, dev, stream)
    else:
        ws = workspace_buf
        _need_ws(ws, dev)
        need = ws.numel()
    args = (x.data_ptr(), ldx, pa, pb, ps, pi, y.data_ptr(), ldy, out.data_ptr(), ldo, M, N, K, R,
            L, ws.data_ptr(), need)
    return args, out, (x, a, b, scales, index, y, out, ws, stream)


def lora_workspace_bytes(M: int, N: int, K: int, R: int) -> int:
    return int(_lib.lora_workspace_bytes(M, N, K, R))


_lora_bytes = functools.lru_cache(maxsize=4096)(lora_workspace_bytes)   # of the sizes alone


def lora_add(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, index: torch.Tensor,
             y: torch.Tensor, scales: torch.Tensor | None = None,
             out: torch.Tensor | None = None, workspace_buf: torch.Tensor | None = None,
             stream=None) -> torch.Tensor:
    """Low-rank adapters of many requests on the output ``y`` [M][N] of a
    projection they share: out[m] = y[m] + scales[i] * (x[m] a[i]^T) b[i]^T
    with i = index[m], for x bf16 [M][K], a bf16 [L][R][K], b bf16 [L][N][R],
    scales fp32 [L] (None: 1) and index int32 [M]; a token whose index is
    outside 0 .. L-1 (say -1) keeps its y.  ``out=y`` adds in place.  The rows
    of x, y and out may be strided (a column range of a fused projection).
    A bounded wait that ran out is reported by ``lora_status``."""
    args, out, keep = _lora_args(x, a, b, index, y, scales, out, workspace_buf, stream)
    _dev_call(x.device, "lora_add", _lib.lora_add, *args, stream=stream)
    return out


def prepare_lora_add(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, index: torch.Tensor,
                     y: torch.Tensor, scales: torch.Tensor | None = None,
                     out: torch.Tensor | None = None, workspace_buf: torch.Tensor | None = None,
                     stream=None):
    """(call, out): ``call()`` runs lora_add on these buffers into ``out``."""
    args, out, keep = _lora_args(x, a, b, index, y, scales, out, workspace_buf, stream)
    return PreparedCall(_lib.lora_add, args + (_stream(stream, x.device),), "lora_add", keep,
                        x.device), out


def lora_status(reset: bool = False, stream=None, device=None) -> int:
    """0, or the first error (MXG_ERR_TIMEOUT) that any lora_add has recorded
    on ``device`` (default: the current device) since the last reset, whatever
    workspace it ran in.  Synchronizes the stream."""
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else
                       torch.device(device).index)
    v = ctypes.c_int(0)
    _dev_call(dev, "lora_status", _lib.lora_status, ctypes.byref(v), 1 if reset else 0,
              stream=stream)
    return v.value


# ---------------------------------------------------------------- sampling
def _sample_args(logits, u, temperature, top_k, top_p, min_p, tokens, probs, stream):
    """The arguments of the C call, its outputs, and the tensors behind them."""
    dev = logits.device
    _need_cuda(logits, "logits")
    if logits.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"logits must be torch.bfloat16 or torch.float32, got {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError(f"logits must be [M][V], got {list(logits.shape)}")
    M, V = logits.shape
    ld, one = logits.stride()
    if one != 1 and V > 1:
        raise ValueError("the rows of logits must be contiguous")
    if M == 1:
        ld = V
    if u is None:
        raise ValueError("u must be given: one random number per row")
    shape, f32, i32 = (M,), _F32, _I32
    pu = _dense(u, f32, shape, dev, "u")
    pt = None if temperature is None else _dense(temperature, f32, shape, dev, "temperature")
    pk = None if top_k is None else _dense(top_k, i32, shape, dev, "top_k")
    pp = None if top_p is None else _dense(top_p, f32, shape, dev, "top_p")
    pq = None if min_p is None else _dense(min_p, f32, shape, dev, "min_p")
    if tokens is None:
        tokens = _empty_as(u, i32, stream)
    else:
        _dense(tokens, i32, shape, dev, "tokens")
    if probs is None:
        probs = _empty_as(u, f32, stream)
    else:
        _dense(probs, f32, shape, dev, "probs")
    args = (logits.data_ptr(), DTYPE_BF16 if logits.dtype == torch.bfloat16 else DTYPE_FP32, ld, M,
            V, pu, pt, pk, pp, pq, tokens.data_ptr(), probs.data_ptr())
    return args, (tokens, probs), (logits, u, temperature, top_k, top_p, min_p, tokens, probs,
                                   stream)


def sample_logits(logits: torch.Tensor, u: torch.Tensor, temperature: torch.Tensor | None = None,
                  top_k: torch.Tensor | None = None, top_p: torch.Tensor | None = None,
                  min_p: torch.Tensor | None = None, tokens: torch.Tensor | None = None,
                  probs: torch.Tensor | None = None, stream=None):
    """(tokens int32 [M], probs fp32 [M]): one token per row of logits (bf16
    or fp32 [M][V], rows may be strided) from the random numbers u fp32 [M],
    after each row's temperature (<= 0: greedy), top_p, top_k and min_p ([M]
    each, None: off), and its share of the mass those filters keep.  The
    definition, with its order of filters and ties, is in include/mxg.h."""
    args, outs, keep = _sample_args(logits, u, temperature, top_k, top_p, min_p, tokens, probs,
                                    stream)
    _dev_call(logits.device, "sample_logits", _lib.sample_logits, *args, stream=stream)
    return outs


def prepare_sample_logits(logits: torch.Tensor, u: torch.Tensor,
                          temperature: torch.Tensor | None = None,
                          top_k: torch.Tensor | None = None, top_p: torch.Tensor | None = None,
                          min_p: torch.Tensor | None = None, tokens: torch.Tensor | None = None,
                          probs: torch.Tensor | None = None, stream=None):
    """(call, (tokens, probs)): ``call()`` runs sample_logits on these buffers."""
    args, outs, keep = _sample_args(logits, u, temperature, top_k, top_p, min_p, tokens, probs,
                                    stream)
    return PreparedCall(_lib.sample_logits, args + (_stream(stream, logits.device),),
                        "sample_logits", keep, logits.device), outs


def w8a16_gemm_sample(x: torch.Tensor, packed: torch.Tensor, N: int, K: int, u: torch.Tensor,
                      temperature: torch.Tensor | None = None, top_k: torch.Tensor | None = None,
                      top_p: torch.Tensor | None = None, min_p: torch.Tensor | None = None,
                      group_size: int = 128, vocab: int | None = None,
                      logits: torch.Tensor | None = None,
                      workspace_buf: torch.Tensor | None = None, stream=None):
    """The INT8 vocabulary head and the sampler on its logits: (tokens, probs,
    logits) for x bf16 [M][K] (M <= 32) and w8a16_repack's buffer.  ``vocab``
    (default N) is the number of real columns of a head padded to N; only
    those are sampled."""
    V = N if vocab is None else int(vocab)
    if not 1 <= V <= N:
        raise ValueError(f"vocab must be in 1 .. {N}, got {V}")
    if x.dim() != 2:
        raise ValueError(f"x must be [M][{K}], got {list(x.shape)}")
    if logits is None:
        logits = _empty((x.shape[0], N), torch.bfloat16, x.device, stream)
    _need_out(logits, x.shape[0], N, x.device)
    # the sampler's arguments are looked at before the head runs
    args, outs, keep = _sample_args(logits[:, :V], u, temperature, top_k, top_p, min_p, None,
                                    None, stream)
    w8a16_gemm(x, packed, N, K, group_size, out=logits, workspace_buf=workspace_buf,
               stream=stream)
    _dev_call(x.device, "sample_logits", _lib.sample_logits, *args, stream=stream)
    return *outs, logits


def mxg_selftest_stream_ring(bits: int, M: int, N: int, K: int, group_size: int = 128,
                             sms: int = 148, smem_bytes: int = 227 * 1024):
    """(stages, turns) of the weight-streaming kernel's ring for a shape, from
    the host's plan alone: ``bits`` 4 (INT4), 8 (INT8) or 0 (re-packed
    MXFP8)."""
    stages, turns = ctypes.c_int(0), ctypes.c_int(0)
    _check(_lib.mxg_selftest_stream_ring(bits, M, N, K, group_size, sms, smem_bytes,
                                         ctypes.byref(stages), ctypes.byref(turns)),
           "mxg_selftest_stream_ring")
    return stages.value, turns.value


def mxg_selftest_wait_timeout(workspace_buf: torch.Tensor | None, limit_us: int,
                              stream=None, device=None) -> None:
    """Runs the library's bounded-wait self-test, which records
    MXG_ERR_TIMEOUT in ``workspace_buf``'s status word, or (None) in the
    static scratch array of ``device`` (default: the current device)."""
    if workspace_buf is None:
        dev = torch.device("cuda", torch.cuda.current_device() if device is None else
                           torch.device(device).index)
        _dev_call(dev, "mxg_selftest_wait_timeout", _lib.mxg_selftest_wait_timeout, None,
                  int(limit_us), stream=stream)
        return
    _need_header(workspace_buf)
    _dev_call(workspace_buf.device, "mxg_selftest_wait_timeout", _lib.mxg_selftest_wait_timeout,
              _ptr(workspace_buf), int(limit_us), stream=stream)


def mxg_selftest_lora_wait_timeout(limit_us: int, stream=None, device=None) -> None:
    """The same for what ``lora_status`` reports on ``device``."""
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else
                       torch.device(device).index)
    _dev_call(dev, "mxg_selftest_lora_wait_timeout", _lib.mxg_selftest_lora_wait_timeout,
              int(limit_us), stream=stream)


def w4a16_static_scratch_status(reset: bool = False, stream=None, device=None) -> int:
    """The status word of the static scratch array of ``device`` (default:
    the current device): 0, or the first error a kernel recorded there.
    ``reset`` also zeroes the status word and the arrival counters.
    Synchronizes the stream."""
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else
                       torch.device(device).index)
    v = ctypes.c_int(0)
    _dev_call(dev, "w4a16_static_scratch_status", _lib.w4a16_static_scratch_status,
              ctypes.byref(v), 1 if reset else 0, stream=stream)
    return v.value


def raw_lib() -> ctypes.CDLL:
    """The loaded C library (for callers that pass raw pointers)."""
    return _lib
