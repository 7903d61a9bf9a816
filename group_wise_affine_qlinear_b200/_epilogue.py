"""Packed projections with bias, activation, gate and residual in their epilogue (see include/qlinear.h)."""
from __future__ import annotations

import ctypes
import functools

import torch

from ._lib import (GROUP, _BF16, _F32, _check, _fit, _need_cuda, _need_dims, _need_workspace, _new, _on_stream,
                   _same_device, _weights_shape, lib)

ACTIVATIONS = {None: 0, "silu": 1, "gelu": 2, "gelu_tanh": 3}


def epilogue_workspace_size(M: int, K: int, N: int, bits: int = 4) -> int:
    """Workspace bytes of forward_epilogue() (bits=8: forward8_epilogue())."""
    fn = lib().qlinear_epilogue_workspace_size if bits == 4 else lib().qlinear8_epilogue_workspace_size
    v = fn(M, K, N, GROUP)
    if v == ctypes.c_size_t(-1).value:
        raise ValueError("shape not supported")
    return int(v)


@functools.lru_cache(maxsize=1024)
def _workspace(dev: int, M: int, K: int, N: int, bits: int) -> int:
    """epilogue_workspace_size() on device `dev` (which is current)."""
    return epilogue_workspace_size(M, K, N, bits)


def forward_epilogue(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor, *,
                     bias: torch.Tensor | None = None, activation: str | None = None, gate: torch.Tensor | None = None,
                     residual: torch.Tensor | None = None, segment_ids: torch.Tensor | None = None,
                     out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, out_dtype=None,
                     stream=None) -> torch.Tensor:
    """y = residual + gate[seg] * act(x . W^T + bias), rounded once (qlinear_epilogue_forward).

    bias [N] and gate [T][N], both bf16 or both fp32; activation None, "silu", "gelu" or "gelu_tanh"; residual [M][N] of
    y's type; segment_ids int32 [M] (None: segment 0), a negative one for a padding row, whose row of y is left alone.
    out may be residual (the update in place).  out_dtype bfloat16 or float32 (None: residual's or out's, else bfloat16).
    """
    return _forward_epilogue(x, codes, scales, biases, bias, activation, gate, residual, segment_ids, out, workspace,
                             out_dtype, stream, 4)


def forward8_epilogue(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor, *,
                      bias: torch.Tensor | None = None, activation: str | None = None,
                      gate: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                      segment_ids: torch.Tensor | None = None, out: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, out_dtype=None, stream=None) -> torch.Tensor:
    """forward_epilogue() for 8-bit codes, int32 [N][K/4] (qlinear8_epilogue_forward)."""
    return _forward_epilogue(x, codes, scales, biases, bias, activation, gate, residual, segment_ids, out, workspace,
                             out_dtype, stream, 8)


def _forward_epilogue(x, codes, scales, biases, bias, activation, gate, residual, segment_ids, out, workspace, out_dtype,
                      stream, bits):
    L = lib()
    # one pass over arguments that are right; where it fails, the checks by name say what is wrong
    try:
        M, K = x.shape
        N = codes.shape[0]
        dev, act = x.get_device(), ACTIVATIONS[activation]
        like = residual if residual is not None else out
        yt = out_dtype if out_dtype is not None else torch.bfloat16 if like is None else like.dtype
        P = bias.dtype if bias is not None else torch.bfloat16 if gate is None else gate.dtype
        T = 1 if gate is None else gate.shape[0]
        rows, vec = (M, N), (N, K // GROUP)
        specs = [(x, torch.bfloat16, (M, K)), (codes, torch.int32, (N, K * bits // 32)), (scales, torch.float16, vec),
                 (biases, torch.float16, vec)]
        if bias is not None:
            specs.append((bias, P, (N,)))
        if gate is not None:
            specs.append((gate, P, (T, N)))
        if residual is not None:
            specs.append((residual, yt, rows))
        if segment_ids is not None:
            specs.append((segment_ids, torch.int32, (M,)))
        if out is not None:
            specs.append((out, yt, rows))
        fit = (dev >= 0 and (yt is torch.bfloat16 or yt is torch.float32) and (P is torch.bfloat16 or P is torch.float32) and
               (T == 1 or (T > 1 and segment_ids is not None)) and _fit(dev, *specs))
    except (AttributeError, IndexError, KeyError, TypeError, ValueError):
        fit = False
    if not fit:
        _refuse(x, codes, scales, biases, bias, activation, gate, residual, segment_ids, out, out_dtype, bits)
    _need_workspace(workspace, dev)
    run = L.qlinear_epilogue_forward if bits == 4 else L.qlinear8_epilogue_forward

    def call(st):
        y = _new(x, rows, yt) if out is None else out
        ws, n = None, 0
        if workspace is not None:
            ws, n = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        elif need := _workspace(dev, M, K, N, bits):
            scratch = x.new_empty(need // 2)               # held until the call below has been enqueued
            ws, n = scratch.data_ptr(), need
        # without a gate every segment is as good as any other
        status = run(x.data_ptr(), codes.data_ptr(), scales.data_ptr(), biases.data_ptr(),
                     None if bias is None else bias.data_ptr(), act, None if gate is None else gate.data_ptr(),
                     _BF16 if P is torch.bfloat16 else _F32, None if residual is None else residual.data_ptr(),
                     None if segment_ids is None else segment_ids.data_ptr(), 2 ** 31 - 1 if gate is None else T,
                     y.data_ptr(), _BF16 if yt is torch.bfloat16 else _F32, M, K, N, GROUP, ws, n, st)
        if status != 0:
            _check(status, "qlinear_epilogue_forward" if bits == 4 else "qlinear8_epilogue_forward")
        return y
    return _on_stream(dev, stream, call)


def _refuse(x, codes, scales, biases, bias, activation, gate, residual, segment_ids, out, out_dtype, bits):
    """Raises for the first argument of _forward_epilogue() that does not fit, by its name."""
    _need_dims(x, 2, "x")
    _need_dims(codes, 2, "codes")
    N, K = _weights_shape(codes, scales, bits)
    M = x.shape[0]
    if not (activation is None or isinstance(activation, str)) or activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {list(ACTIVATIONS)}, got {activation!r}")
    for t, dims, name in ((bias, 1, "bias"), (gate, 2, "gate"), (residual, 2, "residual"), (out, 2, "out")):
        if t is not None:
            _need_dims(t, dims, name)
    if out_dtype is None:
        out_dtype = residual.dtype if residual is not None else out.dtype if out is not None else torch.bfloat16
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("y, its residual and out_dtype must be bfloat16 or float32")
    P = bias.dtype if bias is not None else gate.dtype if gate is not None else torch.bfloat16
    if P not in (torch.bfloat16, torch.float32):
        raise ValueError(f"bias and gate must be bfloat16 or float32, got {P}")
    T = gate.shape[0] if gate is not None else 1
    if T < 1:
        raise ValueError("gate holds no segments")
    if segment_ids is None and T != 1:
        raise ValueError("a gate of several segments needs segment_ids")
    tensors = [(x, torch.bfloat16, (M, K), "x"), (codes, torch.int32, (N, K * bits // 32), "codes"),
               (scales, torch.float16, (N, K // GROUP), "scales"), (biases, torch.float16, (N, K // GROUP), "biases"),
               (bias, P, (N,), "bias"), (gate, P, (T, N), "gate"), (residual, out_dtype, (M, N), "residual"),
               (segment_ids, torch.int32, (M,), "segment_ids"), (out, out_dtype, (M, N), "out")]
    for i, (t, dtype, shape, name) in enumerate(tensors):
        if t is not None or i < 4:
            _need_cuda(t, name, dtype, shape)
    _same_device(x.device, [(name, t) for t, _, _, name in tensors])
    raise ValueError("the arguments do not fit together")
