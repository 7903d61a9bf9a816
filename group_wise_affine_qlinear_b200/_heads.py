"""Rotation of heads by positions of several axes, with the norms of queries and keys (see include/qlinear.h)."""
from __future__ import annotations

import math
import struct

import torch

from ._lib import _BF16, _F32, _check, _dtype_code, _fit, _need_cuda, _need_dims, _on_stream, _same_device, lib

HEAD_MAX_D = 512
_POSITIONS = {torch.int32: 0, torch.int64: 1, torch.float32: 2}


def rotary_frequencies(sections, theta: float = 10000.0, *, shared: bool = True, cycle: bool = False,
                       device="cuda") -> tuple[torch.Tensor, torch.Tensor]:
    """(turns float64 [P], axes int32 [P]) of a rotation over len(sections) axes, P = sum(sections) pairs.

    sections: pairs per axis, e.g. (24, 20, 20) for time, height and width.  Pair i takes the position of axis axes[i]:
    the axes' sections one behind the other, or with `cycle` by turns, each axis while it has pairs left.  Its angle is
    2 pi turns[i] per unit of position: theta^(-i / P), one series over all pairs, or with shared=False a series of its
    own for every axis, theta^(-j / sections[a]) for the axis's j-th pair.
    """
    sections = [int(n) for n in sections]
    P = sum(sections)
    if not sections or min(sections) < 0 or P < 1 or not theta > 0:
        raise ValueError("sections: pairs per axis, at least one in all; theta > 0")
    if cycle:
        rounds = sorted((j, a) for a, n in enumerate(sections) for j in range(n))
        axes = [a for _, a in rounds]
        index = [j for j, _ in rounds]
    else:
        axes = [a for a, n in enumerate(sections) for _ in range(n)]
        index = [j for n in sections for j in range(n)]
    if shared:
        rates = [theta ** (-i / P) for i in range(P)]
    else:
        rates = [theta ** (-j / sections[a]) for j, a in zip(index, axes)]
    return (torch.tensor([r / (2.0 * math.pi) for r in rates], dtype=torch.float64, device=device),
            torch.tensor(axes, dtype=torch.int32, device=device))


def rotary_axes(x: torch.Tensor, positions: torch.Tensor, rotary, *, adjacent: bool = False,
                segment_ids: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Heads x [M][H][D] turned by positions of several axes (qlinear_rotary_axes).

    positions int32, int64 or fp32 [A][M], a row per axis; rotary = (turns float64 [P], axes int32 [P]), e.g. from
    rotary_frequencies().  Pair i of a head, elements i and i + P (adjacent: 2 i and 2 i + 1), turns by the angle
    2 pi turns[i] positions[axes[i]]; elements from 2 P on stay.  x bf16 or fp32 with any strides of tokens and heads (a
    view of a packed projection's output, or heads kept one behind the other); out alike (None: contiguous), it may be x.
    D is a multiple of 8 up to HEAD_MAX_D, P a multiple of 8; addresses and strides are multiples of 16 bytes.
    segment_ids int32 [M]: a negative one for a padding row, which is left alone in out.
    """
    return _heads("qlinear_rotary_axes", x, None, positions, rotary, False, None, None, 0.0, adjacent, segment_ids, out,
                  None, stream)[0]


def qk_norm_rotary(q: torch.Tensor, k: torch.Tensor | None = None, positions: torch.Tensor | None = None, rotary=None, *,
                   q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                   adjacent: bool = False, segment_ids: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
                   k_out: torch.Tensor | None = None, stream=None):
    """RMS norms of queries and keys head by head and rotary_axes() in the same pass (qlinear_qk_norm_rotary) -> (q, k).

        n = q / sqrt(mean_d q^2 + eps) * q_weight      per token and head (k alike), then the rotation

    q [M][Hq][D] and k [M][Hk][D] (None: queries alone) as x in rotary_axes(), e.g. both views of one QKV projection's
    output; weights [D], bf16 or fp32 (None: 1); positions and rotary None: norms without rotation.  q_out may be q and
    k_out k.
    """
    return _heads("qlinear_qk_norm_rotary", q, k, positions, rotary, True, q_weight, k_weight, eps, adjacent, segment_ids,
                  q_out, k_out, stream)


_ENTRY = struct.Struct("@PPqqqqPi4x")       # ql_heads


def _entry(t: torch.Tensor, o: torch.Tensor, weight) -> bytes:
    """ql_heads of one tensor of heads, as it is read and as it is written."""
    a, b, _ = t.stride()
    c, d, _ = o.stride()
    return _ENTRY.pack(t.data_ptr(), o.data_ptr(), a, b, c, d, 0 if weight is None else weight.data_ptr(), t.shape[1])


def _side_by_side(t: torch.Tensor, dtype, shape, dev: int) -> bool:
    """t is [M][H][D] of that shape, type and device, the elements of a head side by side."""
    return t.dtype is dtype and t.shape == shape and t.get_device() == dev and (t.stride(2) == 1 or shape[2] == 1)


def _heads(name, q, k, positions, rotary, norm, q_weight, k_weight, eps, adjacent, segment_ids, q_out, k_out, stream):
    L = lib()
    turns = axes = None
    A = P = 0
    adjacent = 1 if adjacent else 0
    # one pass over arguments that are right; where it fails, the checks by name say what is wrong
    try:
        dt, shape, dev = q.dtype, q.shape, q.get_device()
        M, _, D = shape
        fit = (dev >= 0 and (dt is torch.bfloat16 or dt is torch.float32) and (q.stride(2) == 1 or D == 1) and
               (q_out is None or _side_by_side(q_out, dt, shape, dev)))
        if k is None:
            fit = fit and k_out is None and k_weight is None
        else:
            kshape = k.shape
            fit = (fit and kshape[0] == M and kshape[2] == D and _side_by_side(k, dt, kshape, dev) and
                   (k_out is None or _side_by_side(k_out, dt, kshape, dev)))
        given = q_weight if q_weight is not None else k_weight
        W = torch.float32 if given is None else given.dtype
        specs = []
        if q_weight is not None:
            specs.append((q_weight, W, (D,)))
        if k_weight is not None:
            specs.append((k_weight, W, (D,)))
        if segment_ids is not None:
            specs.append((segment_ids, torch.int32, (M,)))
        pos_type = 0
        if rotary is not None:
            turns, axes = rotary
            A, P = positions.shape[0], turns.shape[0]
            pos_type = _POSITIONS[positions.dtype]
            specs += ((positions, positions.dtype, (A, M)), (turns, torch.float64, (P,)), (axes, torch.int32, (P,)))
            fit = fit and A >= 1 and 1 <= P and 2 * P <= D
        else:
            fit = fit and norm and positions is None
        fit = fit and (W is torch.bfloat16 or W is torch.float32) and _fit(dev, *specs)
    except (AttributeError, IndexError, KeyError, TypeError, ValueError):
        fit = False
    if not fit:
        _refuse(q, k, positions, rotary, norm, q_weight, k_weight, segment_ids, q_out, k_out)

    def call(st):
        qo = q.new_empty(shape) if q_out is None else q_out
        ko = k_out if k is None or k_out is not None else k.new_empty(k.shape)
        dtype = _BF16 if dt is torch.bfloat16 else _F32
        pos, tu, ax = (None, None, None) if rotary is None else (positions.data_ptr(), turns.data_ptr(), axes.data_ptr())
        seg = None if segment_ids is None else segment_ids.data_ptr()
        if norm:
            status = L.qlinear_qk_norm_rotary(_entry(q, qo, q_weight), None if k is None else _entry(k, ko, k_weight), dtype,
                                              _BF16 if W is torch.bfloat16 else _F32, eps, pos, pos_type, A, tu, ax, P,
                                              adjacent, seg, M, D, st)
        else:
            status = L.qlinear_rotary_axes(_entry(q, qo, None), dtype, pos, pos_type, A, tu, ax, P, adjacent, seg, M, D, st)
        if status != 0:
            _check(status, name)
        return qo, ko
    return _on_stream(dev, stream, call)


def _refuse(q, k, positions, rotary, norm, q_weight, k_weight, segment_ids, q_out, k_out):
    """Raises for the first argument of _heads() that does not fit, by its name."""
    qn, on = ("q", "q_out") if norm else ("x", "out")
    _need_dims(q, 3, qn)
    M, _, D = q.shape
    _dtype_code(q, qn)
    for t, of, what in ((q, q, qn), (q_out, q, on), (k, k, "k"), (k_out, k, "k_out")):
        if t is None:
            continue
        if of is None:
            raise ValueError(f"{what} needs k")
        _need_dims(t, 3, what)
        if not t.is_cuda or t.device != q.device:
            raise ValueError(f"{what} must be a CUDA tensor on the device of the others, got {t.device}")
        if t.dtype is not q.dtype:
            raise ValueError(f"{what} must be {q.dtype}, got {t.dtype}")
        if t.shape[0] != M or t.shape[2] != D:
            raise ValueError(f"{what} must have {M} tokens of heads of {D}, got shape {tuple(t.shape)}")
        if t.shape != of.shape:
            raise ValueError(f"{what} must have its input's shape {tuple(of.shape)}, got {tuple(t.shape)}")
        if t.stride(2) != 1:
            raise ValueError(f"the elements of a head of {what} must lie side by side")
    if k is None and k_weight is not None:
        raise ValueError("k_weight needs k")
    given = q_weight if q_weight is not None else k_weight
    if given is not None:
        _need_dims(given, 1, "q_weight" if q_weight is not None else "k_weight")
        if given.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"the weights must be bfloat16 or float32, got {given.dtype}")
        for t, what in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            if t is not None:
                _need_cuda(t, what, given.dtype, (D,))
                _same_device(q.device, ((what, t),))
    if segment_ids is not None:
        _need_cuda(segment_ids, "segment_ids", torch.int32, (M,))
        _same_device(q.device, (("segment_ids", segment_ids),))
    if (positions is None) != (rotary is None):
        raise ValueError("positions and rotary belong together")
    if rotary is None:
        raise ValueError("positions and rotary must be given")
    if not isinstance(rotary, (tuple, list)) or len(rotary) != 2:
        raise ValueError("rotary must be (turns, axes)")
    turns, axes = rotary
    _need_dims(positions, 2, "positions")
    _need_dims(turns, 1, "rotary's turns")
    if positions.dtype not in _POSITIONS:
        raise ValueError(f"positions must be int32, int64 or float32, got {positions.dtype}")
    A, P = positions.shape[0], turns.shape[0]
    if A < 1 or P < 1 or 2 * P > D:
        raise ValueError(f"rotary turns {P} pairs of heads of {D} by {A} axes")
    for t, dtype, shape, what in ((positions, positions.dtype, (A, M), "positions"), (turns, torch.float64, (P,), "rotary's turns"),
                                  (axes, torch.int32, (P,), "rotary's axes")):
        _need_cuda(t, what, dtype, shape)
        _same_device(q.device, ((what, t),))
    raise ValueError("the arguments do not fit together")
