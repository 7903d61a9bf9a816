"""ctypes marshalling for libqlinear.so (see include/qlinear.h for the contract)."""
from __future__ import annotations

import contextlib
import ctypes
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
    with _lock:
        if _lib is not None:
            return _lib
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
    L.qlinear_test_stall.argtypes = [i32, ctypes.c_uint64]
    L.qlinear_test_stall.restype = ctypes.c_int
    L.qlinear_test_ring_depth.argtypes = [i32]
    L.qlinear_test_ring_depth.restype = ctypes.c_int
    L.qlinear_test_delay.argtypes = [i32, ctypes.c_uint64]
    L.qlinear_test_delay.restype = ctypes.c_int
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


def _same_device(dev: torch.device, tensors) -> None:
    for name, t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"{name} must be on {dev}, got {t.device}")


@contextlib.contextmanager
def _call_context(dev: torch.device, stream):
    """The call's device made current, its stream made current too: a buffer allocated inside belongs to it."""
    with torch.cuda.device(dev):
        st = torch.cuda.current_stream() if stream is None else stream
        if stream is None:
            yield st.cuda_stream
        else:
            with torch.cuda.stream(stream):
                yield st.cuda_stream


def _workspace(workspace: torch.Tensor | None, need: int, dev: torch.device) -> torch.Tensor:
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    if not workspace.is_cuda or workspace.device != dev:
        raise ValueError(f"workspace must be on {dev}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace


def _need_adapters(a: torch.Tensor, b: torch.Tensor, K: int, N: int, what: str = "lora") -> tuple[int, int]:
    for name, t in ((what + "_a", a), (what + "_b", b)):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError(f"{name} must be a tensor of three dimensions")
    n, r = a.shape[0], a.shape[1]
    _need_cuda(a, what + "_a", torch.bfloat16, (n, r, K))
    _need_cuda(b, what + "_b", torch.bfloat16, (n, N, r))
    if n < 1 or r < 8 or r % 8 or r > LORA_MAX_RANK:
        raise ValueError(f"{what}_a: at least one adapter, of a rank that is a multiple of 8 up to {LORA_MAX_RANK}")
    return n, r


def _need_rows(ids: torch.Tensor, scale: torch.Tensor | None, M: int, n: int) -> None:
    _need_cuda(ids, "adapter_ids", torch.int32, (M,))
    if scale is not None:
        _need_cuda(scale, "lora_scale", torch.float32, (n,))


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
    N, K = _weights_shape(codes, scales, bits)
    M = x.shape[0]
    _need_cuda(x, "x", torch.bfloat16, (M, K))
    _need_cuda(codes, "codes", torch.int32, (N, K * bits // 32))
    _need_cuda(scales, "scales", torch.float16, (N, K // GROUP))
    _need_cuda(biases, "biases", torch.float16, (N, K // GROUP))
    n, r = _need_adapters(lora_a, lora_b, K, N)
    _need_rows(ids, lora_scale, M, n)
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out_dtype must be bfloat16 or float32")
    if out is not None:
        _need_cuda(out, "out", out_dtype, (M, N))
    dev = x.device
    _same_device(dev, (("codes", codes), ("scales", scales), ("biases", biases), ("lora_a", lora_a),
                       ("lora_b", lora_b), ("adapter_ids", ids), ("lora_scale", lora_scale), ("out", out)))
    name = "qlinear_lora_forward" if bits == 4 else "qlinear8_lora_forward"
    with _call_context(dev, stream) as st:
        if out is None:
            out = torch.empty((M, N), dtype=out_dtype, device=dev)
        ws = _workspace(workspace, lora_workspace_size(M, K, N, n, r, bits) if workspace is None else 0, dev)
        s = getattr(L, name)(x.data_ptr(), codes.data_ptr(), scales.data_ptr(), biases.data_ptr(), lora_a.data_ptr(),
                             lora_b.data_ptr(), _ptr(lora_scale), ids.data_ptr(), out.data_ptr(),
                             _BF16 if out_dtype == torch.bfloat16 else _F32, M, K, N, GROUP, n, r, ws.data_ptr(),
                             ws.numel() * ws.element_size(), st)
    _check(s, name)
    return out


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
    I, K = _weights_shape(gc, gs)
    M = x.shape[0]
    _need_cuda(x, "x", torch.bfloat16, (M, K))
    for name, c, s, b in (("gate", gc, gs, gb), ("up", uc, us, ub)):
        _need_cuda(c, name + " codes", torch.int32, (I, K // 8))
        _need_cuda(s, name + " scales", torch.float16, (I, K // GROUP))
        _need_cuda(b, name + " biases", torch.float16, (I, K // GROUP))
    n, r = _need_adapters(ga, gbb, K, I, "gate_lora")
    if _need_adapters(ua, ubb, K, I, "up_lora") != (n, r):
        raise ValueError("gate_lora and up_lora must hold the same number of adapters of the same rank")
    _need_rows(adapter_ids, lora_scale, M, n)
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out_dtype must be bfloat16 or float32")
    if out is not None:
        _need_cuda(out, "out", out_dtype, (M, I))
    dev = x.device
    _same_device(dev, (("gate codes", gc), ("gate scales", gs), ("gate biases", gb), ("up codes", uc),
                       ("up scales", us), ("up biases", ub), ("gate_lora_a", ga), ("gate_lora_b", gbb),
                       ("up_lora_a", ua), ("up_lora_b", ubb), ("adapter_ids", adapter_ids),
                       ("lora_scale", lora_scale), ("out", out)))
    with _call_context(dev, stream) as st:
        if out is None:
            out = torch.empty((M, I), dtype=out_dtype, device=dev)
        ws = _workspace(workspace, swiglu_lora_workspace_size(M, K, I, n, r) if workspace is None else 0, dev)
        s = L.qlinear_swiglu_lora_forward(x.data_ptr(), gc.data_ptr(), gs.data_ptr(), gb.data_ptr(), uc.data_ptr(),
                                          us.data_ptr(), ub.data_ptr(), ga.data_ptr(), gbb.data_ptr(), ua.data_ptr(),
                                          ubb.data_ptr(), _ptr(lora_scale), adapter_ids.data_ptr(), out.data_ptr(),
                                          _BF16 if out_dtype == torch.bfloat16 else _F32, M, K, I, GROUP, n, r,
                                          ws.data_ptr(), ws.numel() * ws.element_size(), st)
    _check(s, "qlinear_swiglu_lora_forward")
    return out


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
    xt = _dtype_code(x, "x")
    _need_cuda(x, "x", x.dtype, (M, D))
    S, yt = 1, _BF16
    if y is not None:
        if not isinstance(y, torch.Tensor) or y.dim() not in (2, 3):
            raise ValueError("y must be a tensor [M][D] or [S][M][D]")
        yt = _dtype_code(y, "y")
        if y.dim() == 3:
            if yt == _BF16:
                raise ValueError("partials y [S][M][D] must be float32")
            S = y.shape[0]
        _need_cuda(y, "y", y.dtype, (M, D) if y.dim() == 2 else (S, M, D))
    elif post_weight is not None or gate is not None or out is not None:
        raise ValueError("post_weight, gate and out need y")
    if not post_norm and post_weight is not None:
        raise ValueError("post_weight needs post_norm")
    if not pre_norm and not (pre_weight is None and scale is None and shift is None and h is None):
        raise ValueError("pre_weight, scale, shift and h need pre_norm")
    if y is None and not pre_norm:
        raise ValueError("nothing to compute: no y and no pre_norm")
    vectors = [(n, t) for n, t in (("post_weight", post_weight), ("pre_weight", pre_weight), ("gate", gate),
                                   ("scale", scale), ("shift", shift)) if t is not None]
    pt = _dtype_code(vectors[0][1], vectors[0][0]) if vectors else _BF16
    T = None
    for name, t in vectors:
        if name.endswith("weight"):
            _need_cuda(t, name, vectors[0][1].dtype, (D,))
        else:
            T = t.shape[0] if T is None else T
            _need_cuda(t, name, vectors[0][1].dtype, (T, D))
    if segment_ids is not None:
        _need_cuda(segment_ids, "segment_ids", torch.int32, (M,))
    elif T is not None and T != 1:
        raise ValueError("gate, scale and shift of several segments need segment_ids")
    if out is not None:
        _need_cuda(out, "out", x.dtype, (M, D))
    if h is not None:
        _need_cuda(h, "h", torch.bfloat16, (M, D))
    dev = x.device
    _same_device(dev, vectors + [("y", y), ("segment_ids", segment_ids), ("out", out), ("h", h)])
    with _call_context(dev, stream) as st:
        if y is not None and out is None:
            out = torch.empty_like(x)
        if pre_norm and h is None:
            h = torch.empty((M, D), dtype=torch.bfloat16, device=dev)
        # without per-segment vectors every segment is as good as any other
        s = L.qlinear_norm_residual(x.data_ptr(), xt, _ptr(y), yt, S, int(post_norm), _ptr(post_weight), _ptr(gate),
                                    residual_scale, branch_scale, _ptr(pre_weight), _ptr(scale), _ptr(shift), pt,
                                    _ptr(segment_ids), 2 ** 31 - 1 if T is None else T, eps, _ptr(out), _ptr(h), M, D,
                                    st)
    _check(s, "qlinear_norm_residual")
    return (x if y is None else out), h


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
