"""Rotation of heads by positions of several axes, with the norms of queries and keys (see include/qlinear.h)."""
from __future__ import annotations

import math
from ctypes import byref

import torch

from ._lib import Heads, _BF16, _F32, _check, _dtype_code, _need_cuda, _need_dims, _on_stream, _ptr, lib

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


def _check_heads(t, name: str, dtype, M: int, D: int, dev: int) -> None:
    """t is [M][H][D] of that type on device `dev`, its heads' elements side by side."""
    _need_dims(t, 3, name)
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor on the device of the others, got {t.device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape[0] != M or t.shape[2] != D:
        raise ValueError(f"{name} must have {M} tokens of heads of {D}, got shape {tuple(t.shape)}")
    if t.stride(2) != 1 and D > 1:
        raise ValueError(f"the elements of a head of {name} must lie side by side")


def _heads(name, q, k, positions, rotary, norm, q_weight, k_weight, eps, adjacent, segment_ids, q_out, k_out, stream):
    L = lib()
    _need_dims(q, 3, "q" if norm else "x")
    M, _, D = q.shape
    dt, dev = _dtype_code(q, "q" if norm else "x"), q.get_device()
    _check_heads(q, "q" if norm else "x", q.dtype, M, D, dev)
    if q_out is not None:
        _check_heads(q_out, "q_out" if norm else "out", q.dtype, M, D, dev)
        if q_out.shape != q.shape:
            raise ValueError("an output must have its input's shape")
    if k is not None:
        _check_heads(k, "k", q.dtype, M, D, dev)
        if k_out is not None:
            _check_heads(k_out, "k_out", q.dtype, M, D, dev)
            if k_out.shape != k.shape:
                raise ValueError("an output must have its input's shape")
    elif k_weight is not None or k_out is not None:
        raise ValueError("k_weight and k_out need k")
    W = q_weight.dtype if isinstance(q_weight, torch.Tensor) else k_weight.dtype if isinstance(k_weight, torch.Tensor) \
        else torch.float32
    if W not in (torch.bfloat16, torch.float32):
        raise ValueError(f"the weights must be bfloat16 or float32, got {W}")
    turns = axes = None
    A = P = pos_type = 0
    if (positions is None) != (rotary is None):
        raise ValueError("positions and rotary belong together")
    if rotary is not None:
        turns, axes = rotary
        _need_dims(positions, 2, "positions")
        _need_dims(turns, 1, "rotary's turns")
        A, P = positions.shape[0], turns.shape[0]
        if positions.dtype not in _POSITIONS:
            raise ValueError(f"positions must be int32, int64 or float32, got {positions.dtype}")
        pos_type = _POSITIONS[positions.dtype]
        if A < 1 or P < 1 or 2 * P > D:
            raise ValueError(f"rotary turns {P} pairs of heads of {D} by {A} axes")
    elif not norm:
        raise ValueError("positions and rotary must be given")
    for t, dtype, shape, what in ((q_weight, W, (D,), "q_weight"), (k_weight, W, (D,), "k_weight"),
                                  (positions, None if positions is None else positions.dtype, (A, M), "positions"),
                                  (turns, torch.float64, (P,), "rotary's turns"), (axes, torch.int32, (P,), "rotary's axes"),
                                  (segment_ids, torch.int32, (M,), "segment_ids")):
        if t is not None and (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or
                              t.get_device() != dev or not t.is_contiguous()):
            _need_cuda(t, what, dtype, shape)
            raise ValueError(f"{what} must be on {q.device}, got {t.device}")

    def entry(t, o, w):
        st, so = t.stride(), o.stride()
        return Heads(t.data_ptr(), o.data_ptr(), st[0], st[1], so[0], so[1], _ptr(w), t.shape[1])

    def call(st):
        qo = q.new_empty(q.shape) if q_out is None else q_out
        ko = k_out if k is None or k_out is not None else k.new_empty(k.shape)
        hq = entry(q, qo, q_weight)
        tail = (_ptr(positions), pos_type, A, _ptr(turns), _ptr(axes), P, 1 if adjacent else 0, _ptr(segment_ids), M, D, st)
        if norm:
            hk = None if k is None else byref(entry(k, ko, k_weight))
            _check(L.qlinear_qk_norm_rotary(byref(hq), hk, dt, _BF16 if W is torch.bfloat16 else _F32, eps, *tail), name)
        else:
            _check(L.qlinear_rotary_axes(byref(hq), dt, *tail), name)
        return qo, ko
    return _on_stream(dev, stream, call)
