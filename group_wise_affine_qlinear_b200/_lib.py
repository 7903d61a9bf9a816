"""ctypes marshalling for libqlinear.so (see include/qlinear.h for the contract)."""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

GROUP = 64
LORA_MAX_RANK = 128
PATH_AUTO, PATH_GEMV, PATH_TC_SKINNY, PATH_TC_FUSED = 0, 1, 2, 3
_F32, _BF16 = 0, 1

STATUS = {
    0: "QL_OK",
    1: "QL_ERR_INVALID_ARG",
    2: "QL_ERR_ALIGNMENT",
    3: "QL_ERR_UNSUPPORTED",
    4: "QL_ERR_WORKSPACE",
    5: "QL_ERR_CUDA",
    6: "QL_ERR_DEVICE_TIMEOUT",
    7: "QL_ERR_BOUNDS",
}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libqlinear.so"
_lock = threading.Lock()
_lib = None


class QLinearError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}")


def library_path() -> str:
    """The in-tree libqlinear.so, or the library QL_LIBRARY names (e.g. the bounds-checked build)."""
    return os.environ.get("QL_LIBRARY") or os.path.join(_HERE, _LIB_NAME)


def lib() -> ctypes.CDLL:
    """Load libqlinear.so (built in-tree by group_wise_affine_qlinear_b200.build)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            _lib = load_library(library_path())
        return _lib


def load_library(path: str) -> ctypes.CDLL:
    """A CDLL of a qlinear library at `path` with every entry point's argument and result types set."""
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m group_wise_affine_qlinear_b200.build`")
    L = ctypes.CDLL(path)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    L.qlinear_workspace_size.argtypes = [i64, i64, i64, i32]
    L.qlinear_workspace_size.restype = sz
    L.qlinear_workspace_size_config.argtypes = [i64, i64, i64, i32, i32, i32]
    L.qlinear_workspace_size_config.restype = sz
    L.qlinear_forward.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, sz, vp]
    L.qlinear_forward.restype = ctypes.c_int
    L.qlinear_forward_config.argtypes = [vp, vp, vp, vp, vp, ctypes.c_int, i64, i64, i64, i32, i32, i32, vp, sz, vp]
    L.qlinear_forward_config.restype = ctypes.c_int
    L.qlinear_dequant.argtypes = [vp, vp, vp, i64, i64, i32, vp, ctypes.c_int, vp]
    L.qlinear_dequant.restype = ctypes.c_int
    L.qlinear_pack.argtypes = [vp, vp, i64, i64, i32, vp, vp, vp, vp]
    L.qlinear_pack.restype = ctypes.c_int
    L.qlinear_get_device_status.argtypes = [vp]
    L.qlinear_get_device_status.restype = ctypes.c_int
    L.qlinear_last_dispatch.argtypes = [ctypes.c_char_p, sz]
    L.qlinear_last_dispatch.restype = ctypes.c_int
    L.qlinear_forward_noalloc.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, vp]
    L.qlinear_forward_noalloc.restype = ctypes.c_int
    L.qlinear_set_profile_events.argtypes = [vp, vp]
    L.qlinear_set_profile_events.restype = ctypes.c_int
    L.qlinear_status_string.argtypes = [ctypes.c_int]
    L.qlinear_status_string.restype = ctypes.c_char_p
    L.qlinear_version.argtypes = []
    L.qlinear_version.restype = ctypes.c_int32
    L.qlinear8_workspace_size.argtypes = [i64, i64, i64, i32]
    L.qlinear8_workspace_size.restype = sz
    L.qlinear8_workspace_size_config.argtypes = [i64, i64, i64, i32, i32, i32]
    L.qlinear8_workspace_size_config.restype = sz
    L.qlinear8_forward.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, sz, vp]
    L.qlinear8_forward.restype = ctypes.c_int
    L.qlinear8_forward_config.argtypes = [vp, vp, vp, vp, vp, ctypes.c_int, i64, i64, i64, i32, i32, i32, vp, sz,
                                          vp]
    L.qlinear8_forward_config.restype = ctypes.c_int
    L.qlinear8_dequant.argtypes = [vp, vp, vp, i64, i64, i32, vp, ctypes.c_int, vp]
    L.qlinear8_dequant.restype = ctypes.c_int
    L.qlinear8_pack.argtypes = [vp, vp, i64, i64, i32, vp, vp, vp, vp]
    L.qlinear8_pack.restype = ctypes.c_int
    L.qlinear_selftest_bounded_wait.argtypes = [vp]
    L.qlinear_selftest_bounded_wait.restype = ctypes.c_int
    L.qlinear_reduce_partials.argtypes = [vp, i32, i64, vp, ctypes.c_int, vp]
    L.qlinear_reduce_partials.restype = ctypes.c_int
    L.qlinear_swiglu_workspace_size.argtypes = [i64, i64, i64, i32]
    L.qlinear_swiglu_workspace_size.restype = sz
    L.qlinear_swiglu_forward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_int, i64, i64, i64, i32, vp, sz, vp]
    L.qlinear_swiglu_forward.restype = ctypes.c_int
    L.qlinear_lora_workspace_size.argtypes = [i64, i64, i64, i32, i32, i32]
    L.qlinear_lora_workspace_size.restype = sz
    L.qlinear8_lora_workspace_size.argtypes = [i64, i64, i64, i32, i32, i32]
    L.qlinear8_lora_workspace_size.restype = sz
    L.qlinear_lora_forward.argtypes = [vp] * 9 + [ctypes.c_int, i64, i64, i64, i32, i32, i32, vp, sz, vp]
    L.qlinear_lora_forward.restype = ctypes.c_int
    L.qlinear8_lora_forward.argtypes = [vp] * 9 + [ctypes.c_int, i64, i64, i64, i32, i32, i32, vp, sz, vp]
    L.qlinear8_lora_forward.restype = ctypes.c_int
    L.qlinear_swiglu_lora_workspace_size.argtypes = [i64, i64, i64, i32, i32, i32]
    L.qlinear_swiglu_lora_workspace_size.restype = sz
    L.qlinear_swiglu_lora_forward.argtypes = [vp] * 14 + [ctypes.c_int, i64, i64, i64, i32, i32, i32, vp, sz, vp]
    L.qlinear_swiglu_lora_forward.restype = ctypes.c_int
    f32 = ctypes.c_float
    L.qlinear_norm_residual.argtypes = [vp, ctypes.c_int, vp, ctypes.c_int, i32, i32, vp, vp, f32, f32, vp, vp, vp,
                                        ctypes.c_int, vp, i32, f32, vp, vp, i64, i64, vp]
    L.qlinear_norm_residual.restype = ctypes.c_int
    L.qlinear_epilogue_workspace_size.argtypes = [i64, i64, i64, i32]
    L.qlinear_epilogue_workspace_size.restype = sz
    L.qlinear8_epilogue_workspace_size.argtypes = [i64, i64, i64, i32]
    L.qlinear8_epilogue_workspace_size.restype = sz
    epilogue = [vp] * 5 + [i32, vp, ctypes.c_int, vp, vp, i32, vp, ctypes.c_int, i64, i64, i64, i32, vp, sz, vp]
    L.qlinear_epilogue_forward.argtypes = epilogue
    L.qlinear_epilogue_forward.restype = ctypes.c_int
    L.qlinear8_epilogue_forward.argtypes = epilogue
    L.qlinear8_epilogue_forward.restype = ctypes.c_int
    rotary = [vp, ctypes.c_int, i32, vp, vp, i32, i32, vp, i64, i64, vp]       # positions .. stream
    L.qlinear_rotary_axes.argtypes = [vp, ctypes.c_int] + rotary          # (a ql_heads: its bytes, or a pointer)
    L.qlinear_rotary_axes.restype = ctypes.c_int
    L.qlinear_qk_norm_rotary.argtypes = [vp, vp] + [ctypes.c_int, ctypes.c_int, f32] + rotary
    L.qlinear_qk_norm_rotary.restype = ctypes.c_int
    L.qlinear_test_stall.argtypes = [i32, ctypes.c_uint64]
    L.qlinear_test_stall.restype = ctypes.c_int
    L.qlinear_test_ring_depth.argtypes = [i32]
    L.qlinear_test_ring_depth.restype = ctypes.c_int
    L.qlinear_test_delay.argtypes = [i32, ctypes.c_uint64]
    L.qlinear_test_delay.restype = ctypes.c_int
    L.qlinear_test_extent.argtypes = [i64]
    L.qlinear_test_extent.restype = ctypes.c_int
    return L


def _stream_handle(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _check(status: int, what: str) -> None:
    if status != 0:
        raise QLinearError(status, what)


def _need_cuda(t: torch.Tensor, name: str, dtype, shape=None) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _weights_shape(codes: torch.Tensor, scales: torch.Tensor, bits: int = 4):
    N, Kw = codes.shape
    K = (32 // bits) * Kw
    return N, K


def workspace_size(M: int, K: int, N: int, path: int = PATH_AUTO, split_k: int = 0, bits: int = 4) -> int:
    fn = lib().qlinear_workspace_size_config if bits == 4 else lib().qlinear8_workspace_size_config
    v = fn(M, K, N, GROUP, path, split_k)
    if v == ctypes.c_size_t(-1).value:
        raise ValueError("shape or path not supported")
    return int(v)


def workspace_size8(M: int, K: int, N: int, path: int = PATH_AUTO, split_k: int = 0) -> int:
    """Workspace bytes of forward8 (qlinear8_workspace_size_config)."""
    return workspace_size(M, K, N, path, split_k, bits=8)


def forward(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor,
            out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
            path: int = PATH_AUTO, split_k: int = 0, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """y = x . W^T for the packed W; see include/qlinear.h (qlinear_forward[_config])."""
    return _forward(x, codes, scales, biases, out, workspace, path, split_k, out_dtype, stream, 4)


def forward8(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor,
             out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
             path: int = PATH_AUTO, split_k: int = 0, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """forward() for 8-bit codes, int32 [N][K/4] (qlinear8_forward[_config])."""
    return _forward(x, codes, scales, biases, out, workspace, path, split_k, out_dtype, stream, 8)


def _forward(x, codes, scales, biases, out, workspace, path, split_k, out_dtype, stream, bits):
    L = lib()
    N, K = _weights_shape(codes, scales, bits)
    M = x.shape[0]
    _need_cuda(x, "x", torch.bfloat16, (M, K))
    _need_cuda(codes, "codes", torch.int32, (N, K * bits // 32))
    _need_cuda(scales, "scales", torch.float16, (N, K // GROUP))
    _need_cuda(biases, "biases", torch.float16, (N, K // GROUP))
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out_dtype must be bfloat16 or float32")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=x.device)
    _need_cuda(out, "out", out_dtype, (M, N))
    need = workspace_size(M, K, N, path, split_k, bits)
    if need > 0 and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = _stream_handle(stream)
    name = "qlinear_forward" if bits == 4 else "qlinear8_forward"
    if path == PATH_AUTO and split_k == 0 and out_dtype == torch.bfloat16:
        s = getattr(L, name)(x.data_ptr(), codes.data_ptr(), scales.data_ptr(), biases.data_ptr(), out.data_ptr(),
                             M, K, N, GROUP, ws_ptr, ws_bytes, st)
    else:
        s = getattr(L, name + "_config")(x.data_ptr(), codes.data_ptr(), scales.data_ptr(), biases.data_ptr(),
                                         out.data_ptr(), _BF16 if out_dtype == torch.bfloat16 else _F32,
                                         M, K, N, GROUP, path, split_k, ws_ptr, ws_bytes, st)
    _check(s, name)
    return out


def forward_noalloc(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor,
                    out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Small-M forward that allocates nothing on the device (qlinear_forward_noalloc in include/qlinear.h)."""
    L = lib()
    N, K = _weights_shape(codes, scales)
    M = x.shape[0]
    _need_cuda(x, "x", torch.bfloat16, (M, K))
    _need_cuda(codes, "codes", torch.int32, (N, K // 8))
    _need_cuda(scales, "scales", torch.float16, (N, K // GROUP))
    _need_cuda(biases, "biases", torch.float16, (N, K // GROUP))
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _need_cuda(out, "out", torch.bfloat16, (M, N))
    _check(L.qlinear_forward_noalloc(x.data_ptr(), codes.data_ptr(), scales.data_ptr(), biases.data_ptr(),
                                     out.data_ptr(), M, K, N, GROUP, _stream_handle(stream)), "qlinear_forward_noalloc")
    return out


def dequant(codes: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor, out_dtype=torch.float32,
            out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """W[n][k] = RN_fp32(scale * q + bias) (optionally rounded again to bf16)."""
    return _dequant(codes, scales, biases, out_dtype, out, stream, 4)


def dequant8(codes: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor, out_dtype=torch.float32,
             out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dequant() for 8-bit codes, int32 [N][K/4] (qlinear8_dequant)."""
    return _dequant(codes, scales, biases, out_dtype, out, stream, 8)


def _dequant(codes, scales, biases, out_dtype, out, stream, bits):
    L = lib()
    N, K = _weights_shape(codes, scales, bits)
    _need_cuda(codes, "codes", torch.int32, (N, K * bits // 32))
    _need_cuda(scales, "scales", torch.float16, (N, K // GROUP))
    _need_cuda(biases, "biases", torch.float16, (N, K // GROUP))
    if out is None:
        out = torch.empty((N, K), dtype=out_dtype, device=codes.device)
    _need_cuda(out, "out", out_dtype, (N, K))
    dt = {torch.float32: _F32, torch.bfloat16: _BF16}[out_dtype]
    name = "qlinear_dequant" if bits == 4 else "qlinear8_dequant"
    _check(getattr(L, name)(codes.data_ptr(), scales.data_ptr(), biases.data_ptr(), K, N, GROUP, out.data_ptr(), dt,
                            _stream_handle(stream)), name)
    return out


def pack(w: torch.Tensor, imatrix: torch.Tensor | None = None, stream=None):
    """Quantize fp32 W [N][K] -> (codes, scales, biases): round-to-nearest, or the imatrix-weighted fit."""
    return _pack(w, imatrix, stream, 4)


def pack8(w: torch.Tensor, stream=None):
    """Round-to-nearest quantization of fp32 W [N][K] to 8-bit codes, int32 [N][K/4] (qlinear8_pack)."""
    return _pack(w, None, stream, 8)


def _pack(w, imatrix, stream, bits):
    L = lib()
    N, K = w.shape
    _need_cuda(w, "w", torch.float32, (N, K))
    codes = torch.empty((N, K * bits // 32), dtype=torch.int32, device=w.device)
    scales = torch.empty((N, K // GROUP), dtype=torch.float16, device=w.device)
    biases = torch.empty((N, K // GROUP), dtype=torch.float16, device=w.device)
    imp = None
    if imatrix is not None:
        _need_cuda(imatrix, "imatrix", torch.float32, (K,))
        imp = imatrix.data_ptr()
    name = "qlinear_pack" if bits == 4 else "qlinear8_pack"
    _check(getattr(L, name)(w.data_ptr(), imp, K, N, GROUP, codes.data_ptr(), scales.data_ptr(), biases.data_ptr(),
                            _stream_handle(stream)), name)
    return codes, scales, biases


def swiglu_workspace_size(M: int, K: int, I: int) -> int:
    """Workspace bytes of swiglu() (qlinear_swiglu_workspace_size)."""
    v = lib().qlinear_swiglu_workspace_size(M, K, I, GROUP)
    if v == ctypes.c_size_t(-1).value:
        raise ValueError("shape not supported")
    return int(v)


def swiglu(x: torch.Tensor, gate, up, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
           out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """h = silu(x . W_gate^T) * (x . W_up^T) for two packed [I][K] weights (qlinear_swiglu_forward).

    gate and up are (codes int32 [I][K/8], scales f16 [I][K/64], biases f16 [I][K/64]) triples.
    """
    L = lib()
    gc, gs, gb = gate
    uc, us, ub = up
    I, K = _weights_shape(gc, gs)
    M = x.shape[0]
    _need_cuda(x, "x", torch.bfloat16, (M, K))
    for name, c, s, b in (("gate", gc, gs, gb), ("up", uc, us, ub)):
        _need_cuda(c, name + " codes", torch.int32, (I, K // 8))
        _need_cuda(s, name + " scales", torch.float16, (I, K // GROUP))
        _need_cuda(b, name + " biases", torch.float16, (I, K // GROUP))
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out_dtype must be bfloat16 or float32")
    if out is None:
        out = torch.empty((M, I), dtype=out_dtype, device=x.device)
    _need_cuda(out, "out", out_dtype, (M, I))
    need = swiglu_workspace_size(M, K, I)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    _check(L.qlinear_swiglu_forward(x.data_ptr(), gc.data_ptr(), gs.data_ptr(), gb.data_ptr(), uc.data_ptr(),
                                    us.data_ptr(), ub.data_ptr(), out.data_ptr(),
                                    _BF16 if out_dtype == torch.bfloat16 else _F32, M, K, I, GROUP,
                                    workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                    _stream_handle(stream)), "qlinear_swiglu_forward")
    return out


def _fit(dev: int, *specs) -> bool:
    """Whether every tensor of the (tensor, dtype, shape) specs is contiguous, of that type and shape, on CUDA device
    `dev`: the one pass of a call whose arguments are right.  Where it fails, the checks by name say what is wrong."""
    try:
        for t, dtype, shape in specs:
            if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
                return False
    except AttributeError:                 # not a tensor
        return False
    return True


def _need_dims(t, dims: int, name: str) -> None:
    if not isinstance(t, torch.Tensor) or t.dim() != dims:
        raise ValueError(f"{name} must be a tensor of {dims} dimensions")


def _same_device(dev: torch.device, tensors) -> None:
    for name, t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"{name} must be on {dev}, got {t.device}")


def _new(x: torch.Tensor, shape, dtype) -> torch.Tensor:
    """An uninitialized tensor on x's device.  (new_empty without a dtype, with sizes of their own, is the cheapest call:
    1 us of a small one's 20, 1.5 with a tuple.)"""
    return x.new_empty(*shape) if dtype is x.dtype else x.new_empty(shape, dtype=dtype)


def _on_stream(dev: int, stream, call):
    """call(raw stream handle) with device `dev` current; a given stream is current too, so that a buffer allocated
    inside belongs to it."""
    if stream is None and torch._C._cuda_getDevice() == dev:        # (a tensor on it: CUDA is initialized)
        return call(torch._C._cuda_getCurrentRawStream(dev))
    if stream is not None and stream.device.index != dev:           # its device would become the current one
        raise ValueError(f"stream must be on cuda:{dev}, got one on {stream.device}")
    with torch.cuda.device(dev):
        if stream is None:
            return call(torch._C._cuda_getCurrentRawStream(dev))
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)


def _need_workspace(workspace: torch.Tensor | None, dev: int) -> None:
    if workspace is None:
        return
    if not isinstance(workspace, torch.Tensor) or workspace.get_device() != dev:
        raise ValueError(f"workspace must be a tensor on cuda:{dev}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")


def _adapter_shape(a: torch.Tensor, b: torch.Tensor, what: str) -> tuple[int, int]:
    """(adapters, rank) of lora_a [L][r][K] and lora_b [L][N][r]."""
    _need_dims(a, 3, what + "_a")
    _need_dims(b, 3, what + "_b")
    n, r, _ = a.shape
    if n < 1 or r < 8 or r % 8 or r > LORA_MAX_RANK:
        raise ValueError(f"{what}_a: at least one adapter, of a rank that is a multiple of 8 up to {LORA_MAX_RANK}")
    return n, r


def _need_rows(ids: torch.Tensor, scale: torch.Tensor | None, M: int, n: int) -> None:
    _need_cuda(ids, "adapter_ids", torch.int32, (M,))
    if scale is not None:
        _need_cuda(scale, "lora_scale", torch.float32, (n,))


@functools.lru_cache(maxsize=1024)
def _lora_workspace(dev: int, M: int, K: int, N: int, adapters: int, rank: int, bits: int) -> int:
    """lora_workspace_size() on device `dev` (which is current), a multiple of 256; it is a function of the shape and the
    SM count."""
    return lora_workspace_size(M, K, N, adapters, rank, bits)


@functools.lru_cache(maxsize=1024)
def _swiglu_lora_workspace(dev: int, M: int, K: int, I: int, adapters: int, rank: int) -> int:
    """swiglu_lora_workspace_size() on device `dev` (which is current)."""
    return swiglu_lora_workspace_size(M, K, I, adapters, rank)


def lora_workspace_size(M: int, K: int, N: int, adapters: int, rank: int, bits: int = 4) -> int:
    """Workspace bytes of forward_lora() (bits=8: forward8_lora())."""
    fn = lib().qlinear_lora_workspace_size if bits == 4 else lib().qlinear8_lora_workspace_size
    v = fn(M, K, N, GROUP, adapters, rank)
    if v == ctypes.c_size_t(-1).value:
        raise ValueError("shape not supported")
    return int(v)


def forward_lora(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor,
                 lora_a: torch.Tensor, lora_b: torch.Tensor, adapter_ids: torch.Tensor,
                 lora_scale: torch.Tensor | None = None, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """y[m] = x[m] . W^T + s_a (x[m] . A_a^T) . B_a^T, a = adapter_ids[m] (qlinear_lora_forward).

    lora_a bf16 [L][r][K], lora_b bf16 [L][N][r], lora_scale fp32 [L] (None: 1), adapter_ids int32 [M] with -1 for
    a row without an adapter.  An id outside [-1, L) counts as -1, a non-finite entry of lora_b as 0, and both set
    the device status word.
    """
    return _forward_lora(x, codes, scales, biases, lora_a, lora_b, adapter_ids, lora_scale, out, workspace, out_dtype,
                         stream, 4)


def forward8_lora(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor,
                  lora_a: torch.Tensor, lora_b: torch.Tensor, adapter_ids: torch.Tensor,
                  lora_scale: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """forward_lora() for 8-bit codes, int32 [N][K/4] (qlinear8_lora_forward)."""
    return _forward_lora(x, codes, scales, biases, lora_a, lora_b, adapter_ids, lora_scale, out, workspace, out_dtype,
                         stream, 8)


def _forward_lora(x, codes, scales, biases, lora_a, lora_b, ids, lora_scale, out, workspace, out_dtype, stream, bits):
    L = lib()
    _need_dims(x, 2, "x")
    _need_dims(codes, 2, "codes")
    N, K = _weights_shape(codes, scales, bits)
    M = x.shape[0]
    n, r = _adapter_shape(lora_a, lora_b, "lora")
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out_dtype must be bfloat16 or float32")
    dev = x.get_device()
    if not (dev >= 0 and _fit(dev, (x, torch.bfloat16, (M, K)), (codes, torch.int32, (N, K * bits // 32)),
                              (scales, torch.float16, (N, K // GROUP)), (biases, torch.float16, (N, K // GROUP)),
                              (lora_a, torch.bfloat16, (n, r, K)), (lora_b, torch.bfloat16, (n, N, r)),
                              (ids, torch.int32, (M,))) and
            (out is None or _fit(dev, (out, out_dtype, (M, N)))) and
            (lora_scale is None or _fit(dev, (lora_scale, torch.float32, (n,))))):
        _need_cuda(x, "x", torch.bfloat16, (M, K))
        _need_cuda(codes, "codes", torch.int32, (N, K * bits // 32))
        _need_cuda(scales, "scales", torch.float16, (N, K // GROUP))
        _need_cuda(biases, "biases", torch.float16, (N, K // GROUP))
        _need_cuda(lora_a, "lora_a", torch.bfloat16, (n, r, K))
        _need_cuda(lora_b, "lora_b", torch.bfloat16, (n, N, r))
        _need_rows(ids, lora_scale, M, n)
        if out is not None:
            _need_cuda(out, "out", out_dtype, (M, N))
        _same_device(x.device, (("codes", codes), ("scales", scales), ("biases", biases), ("lora_a", lora_a),
                                ("lora_b", lora_b), ("adapter_ids", ids), ("lora_scale", lora_scale), ("out", out)))
    _need_workspace(workspace, dev)
    name = "qlinear_lora_forward" if bits == 4 else "qlinear8_lora_forward"

    def call(st):
        y = _new(x, (M, N), out_dtype) if out is None else out
        ws = x.new_empty(_lora_workspace(dev, M, K, N, n, r, bits) // 2) if workspace is None else workspace
        _check(getattr(L, name)(x.data_ptr(), codes.data_ptr(), scales.data_ptr(), biases.data_ptr(),
                                lora_a.data_ptr(), lora_b.data_ptr(), _ptr(lora_scale), ids.data_ptr(), y.data_ptr(),
                                _BF16 if out_dtype == torch.bfloat16 else _F32, M, K, N, GROUP, n, r, ws.data_ptr(),
                                ws.numel() * ws.element_size(), st), name)
        return y
    return _on_stream(dev, stream, call)


def swiglu_lora_workspace_size(M: int, K: int, I: int, adapters: int, rank: int) -> int:
    """Workspace bytes of swiglu_lora() (qlinear_swiglu_lora_workspace_size)."""
    v = lib().qlinear_swiglu_lora_workspace_size(M, K, I, GROUP, adapters, rank)
    if v == ctypes.c_size_t(-1).value:
        raise ValueError("shape not supported")
    return int(v)


def swiglu_lora(x: torch.Tensor, gate, up, gate_lora, up_lora, adapter_ids: torch.Tensor,
                lora_scale: torch.Tensor | None = None, out: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """swiglu() with low-rank adapters on both projections (qlinear_swiglu_lora_forward).

    gate and up as in swiglu(); gate_lora and up_lora are (lora_a bf16 [L][r][K], lora_b bf16 [L][I][r]) pairs of
    the same L and r; adapter_ids and lora_scale as in forward_lora().
    """
    L = lib()
    gc, gs, gb = gate
    uc, us, ub = up
    ga, gbb = gate_lora
    ua, ubb = up_lora
    _need_dims(x, 2, "x")
    _need_dims(gc, 2, "gate codes")
    I, K = _weights_shape(gc, gs)
    M = x.shape[0]
    n, r = _adapter_shape(ga, gbb, "gate_lora")
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out_dtype must be bfloat16 or float32")
    dev = x.get_device()
    wc, wp = (I, K // 8), (I, K // GROUP)
    if not (dev >= 0 and _fit(dev, (x, torch.bfloat16, (M, K)), (gc, torch.int32, wc), (gs, torch.float16, wp),
                              (gb, torch.float16, wp), (uc, torch.int32, wc), (us, torch.float16, wp),
                              (ub, torch.float16, wp), (ga, torch.bfloat16, (n, r, K)), (gbb, torch.bfloat16, (n, I, r)),
                              (ua, torch.bfloat16, (n, r, K)), (ubb, torch.bfloat16, (n, I, r)),
                              (adapter_ids, torch.int32, (M,))) and
            (out is None or _fit(dev, (out, out_dtype, (M, I)))) and
            (lora_scale is None or _fit(dev, (lora_scale, torch.float32, (n,))))):
        _need_cuda(x, "x", torch.bfloat16, (M, K))
        for name, c, s, b in (("gate", gc, gs, gb), ("up", uc, us, ub)):
            _need_cuda(c, name + " codes", torch.int32, wc)
            _need_cuda(s, name + " scales", torch.float16, wp)
            _need_cuda(b, name + " biases", torch.float16, wp)
        for name, a, b in (("gate_lora", ga, gbb), ("up_lora", ua, ubb)):
            _need_cuda(a, name + "_a", torch.bfloat16, (n, r, K))
            _need_cuda(b, name + "_b", torch.bfloat16, (n, I, r))
        _need_rows(adapter_ids, lora_scale, M, n)
        if out is not None:
            _need_cuda(out, "out", out_dtype, (M, I))
        _same_device(x.device, (("gate codes", gc), ("gate scales", gs), ("gate biases", gb), ("up codes", uc),
                                ("up scales", us), ("up biases", ub), ("gate_lora_a", ga), ("gate_lora_b", gbb),
                                ("up_lora_a", ua), ("up_lora_b", ubb), ("adapter_ids", adapter_ids),
                                ("lora_scale", lora_scale), ("out", out)))
    _need_workspace(workspace, dev)

    def call(st):
        h = _new(x, (M, I), out_dtype) if out is None else out
        ws = x.new_empty(_swiglu_lora_workspace(dev, M, K, I, n, r) // 2) if workspace is None else workspace
        _check(L.qlinear_swiglu_lora_forward(x.data_ptr(), gc.data_ptr(), gs.data_ptr(), gb.data_ptr(), uc.data_ptr(),
                                             us.data_ptr(), ub.data_ptr(), ga.data_ptr(), gbb.data_ptr(), ua.data_ptr(),
                                             ubb.data_ptr(), _ptr(lora_scale), adapter_ids.data_ptr(), h.data_ptr(),
                                             _BF16 if out_dtype == torch.bfloat16 else _F32, M, K, I, GROUP, n, r,
                                             ws.data_ptr(), ws.numel() * ws.element_size(), st),
               "qlinear_swiglu_lora_forward")
        return h
    return _on_stream(dev, stream, call)


def _dtype_code(t: torch.Tensor, name: str) -> int:
    if t.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return _BF16 if t.dtype == torch.bfloat16 else _F32


def norm_residual(x: torch.Tensor, y: torch.Tensor | None = None, *, post_norm: bool = True,
                  post_weight: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                  residual_scale: float = 1.0, branch_scale: float = 1.0, pre_norm: bool = True,
                  pre_weight: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                  shift: torch.Tensor | None = None, segment_ids: torch.Tensor | None = None, eps: float = 1e-6,
                  out: torch.Tensor | None = None, h: torch.Tensor | None = None, stream=None):
    """The norms after and before a block with its gate and residual update (qlinear_norm_residual) -> (r, h).

        r = residual_scale * x + branch_scale * gate[seg] * (RMS(y) * post_weight)     (y itself without post_norm)
        h = RMS(r) * pre_weight * (1 + scale[seg]) + shift[seg]                         (None without pre_norm)

    x bf16 or fp32 [M][D]; y bf16 [M][D], fp32 [M][D] or the fp32 partials [S][M][D] of a row-parallel projection;
    post_weight, pre_weight [D] and gate, scale, shift [T][D], all bf16 or all fp32; segment_ids int32 [M] (None:
    segment 0), a negative one for a padding row, which is left alone in out and h.  out may be x (the update in
    place).  Without y, r is x and only h is computed.
    """
    L = lib()
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a tensor [M][D]")
    M, D = x.shape
    xd = x.dtype
    xt = _dtype_code(x, "x")
    S, yt = 0, _BF16                       # S 0: y is [M][D]
    if y is not None:
        if not isinstance(y, torch.Tensor) or y.dim() not in (2, 3):
            raise ValueError("y must be a tensor [M][D] or [S][M][D]")
        yt = _dtype_code(y, "y")
        if y.dim() == 3:
            if yt == _BF16:
                raise ValueError("partials y [S][M][D] must be float32")
            S = y.shape[0]
            if S == 0:
                raise ValueError("y holds no partials")
    elif post_weight is not None or gate is not None or out is not None:
        raise ValueError("post_weight, gate and out need y")
    if not post_norm and post_weight is not None:
        raise ValueError("post_weight needs post_norm")
    if not pre_norm:
        if not (pre_weight is None and scale is None and shift is None and h is None):
            raise ValueError("pre_weight, scale, shift and h need pre_norm")
        if y is None:
            raise ValueError("nothing to compute: no y and no pre_norm")
    # T: segments of gate, scale and shift; P: the vectors' type
    T = P = None
    for t, name in ((gate, "gate"), (scale, "scale"), (shift, "shift")):
        if t is not None:
            _need_dims(t, 2, name)
            T, P = t.shape[0], t.dtype
            break
    else:
        for t, name in ((post_weight, "post_weight"), (pre_weight, "pre_weight")):
            if t is not None:
                _need_dims(t, 1, name)
                P = t.dtype
                break
    if segment_ids is None and T is not None and T != 1:
        raise ValueError("gate, scale and shift of several segments need segment_ids")
    dev = x.get_device()
    rows, vec, mod = (M, D), (D,), (T, D)
    try:
        for t, dtype, shape, name in ((x, xd, rows, "x"), (y, None if y is None else y.dtype, rows if S == 0 else (S, M, D), "y"),
                                      (post_weight, P, vec, "post_weight"), (gate, P, mod, "gate"),
                                      (pre_weight, P, vec, "pre_weight"), (scale, P, mod, "scale"),
                                      (shift, P, mod, "shift"), (segment_ids, torch.int32, rows[:1], "segment_ids"),
                                      (out, xd, rows, "out"), (h, torch.bfloat16, rows, "h")):
            if t is not None and (t.dtype is not dtype or t.shape != shape or t.get_device() != dev or dev < 0 or
                                  not t.is_contiguous()):
                _need_cuda(t, name, dtype, shape)
                _same_device(x.device, ((name, t),))
    except AttributeError:
        raise ValueError(f"{name} must be a CUDA tensor") from None
    pt = _BF16 if P is None or P is torch.bfloat16 else _F32
    if pt == _F32 and P is not torch.float32:
        raise ValueError(f"the weights, gate, scale and shift must be bfloat16 or float32, got {P}")

    def call(st):
        r = x.new_empty(M, D) if y is not None and out is None else out
        n = _new(x, (M, D), torch.bfloat16) if pre_norm and h is None else h
        # without per-segment vectors every segment is as good as any other
        _check(L.qlinear_norm_residual(x.data_ptr(), xt, _ptr(y), yt, S or 1, 1 if post_norm else 0, _ptr(post_weight),
                                       _ptr(gate), residual_scale, branch_scale, _ptr(pre_weight), _ptr(scale),
                                       _ptr(shift), pt, _ptr(segment_ids),
                                       2 ** 31 - 1 if T is None else T, eps, _ptr(r), _ptr(n), M, D, st),
               "qlinear_norm_residual")
        return (x if y is None else r), n
    return _on_stream(dev, stream, call)


def reduce_partials(partials: torch.Tensor, out: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                    stream=None) -> torch.Tensor:
    """Sum fp32 partials [S][...] over S in order, rounded once (qlinear_reduce_partials) -> [...]."""
    L = lib()
    if not isinstance(partials, torch.Tensor) or partials.dim() < 2:
        raise ValueError("partials must be a tensor [S][...]")
    _need_cuda(partials, "partials", torch.float32)
    S = partials.shape[0]
    shape = tuple(partials.shape[1:])
    if out is None:
        out = torch.empty(shape, dtype=out_dtype, device=partials.device)
    _need_cuda(out, "out", out_dtype, shape)
    _check(L.qlinear_reduce_partials(partials.data_ptr(), S, out.numel(), out.data_ptr(),
                                     _BF16 if out_dtype == torch.bfloat16 else _F32, _stream_handle(stream)),
           "qlinear_reduce_partials")
    return out


def selftest_bounded_wait(stream=None) -> None:
    """Enqueue the bounded-wait self-test (qlinear_selftest_bounded_wait); device_status() then reads 6."""
    _check(lib().qlinear_selftest_bounded_wait(_stream_handle(stream)), "qlinear_selftest_bounded_wait")


def device_status(stream=None) -> int:
    """Synchronize the stream, then read and clear the device status word (0 = no kernel error)."""
    return int(lib().qlinear_get_device_status(_stream_handle(stream)))


def last_dispatch() -> str:
    buf = ctypes.create_string_buffer(256)
    _check(lib().qlinear_last_dispatch(buf, 256), "qlinear_last_dispatch")
    return buf.value.decode()


def set_profile_events(start, stop) -> None:
    """Record torch.cuda.Event `start`/`stop` around the main kernel of each later forward call (None, None: off)."""
    if start is None:
        _check(lib().qlinear_set_profile_events(None, None), "qlinear_set_profile_events")
    else:
        _check(lib().qlinear_set_profile_events(start.cuda_event, stop.cuda_event), "qlinear_set_profile_events")


def version() -> int:
    return int(lib().qlinear_version())
