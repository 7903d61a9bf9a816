"""Epilogues of a projection, and norms and rotation of heads, without a GPU: the oracle against loops, the frequencies,
and every refusal of the C entries and of the binding."""
import ctypes
import math

import numpy as np
import pytest
import torch

import group_wise_affine_qlinear_b200 as ql
from group_wise_affine_qlinear_b200 import build as qb
from oracle import qlinear_oracle as O


@pytest.fixture(scope="module")
def L():
    qb.build()
    return ql.lib()


class Heads(ctypes.Structure):
    """ql_heads of include/qlinear.h."""
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("in_token", ctypes.c_int64),
                ("in_head", ctypes.c_int64), ("out_token", ctypes.c_int64), ("out_head", ctypes.c_int64),
                ("weight", ctypes.c_void_p), ("heads", ctypes.c_int32)]


# ------------------------------------------------------------------ the oracle

def test_activations_against_closed_forms():
    z = np.array([-30.0, -3.0, -0.5, 0.0, 0.5, 3.0, 30.0])
    assert np.allclose(O.activation(z, "gelu"), [v * 0.5 * (1 + math.erf(v / math.sqrt(2))) for v in z], atol=1e-12)
    tanh = [0.5 * v * (1 + math.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))) for v in z]
    assert np.allclose(O.activation(z, "gelu_tanh"), tanh, rtol=0, atol=1e-12)
    assert np.allclose(O.activation(z, "silu"), [v / (1 + math.exp(-v)) for v in z], rtol=1e-14)
    assert np.array_equal(O.activation(z, None), z)


def test_slopes_of_the_activations():
    """The GPU tests bound an activation's error by 1.13 times its argument's."""
    z = np.linspace(-12, 12, 48001)
    for kind in ("silu", "gelu", "gelu_tanh"):
        slope = np.diff(O.activation(z, kind)) / np.diff(z)
        assert np.abs(slope).max() < 1.13


def test_epilogue_against_a_loop():
    rng = np.random.default_rng(0)
    lin, bias, gate, res = rng.standard_normal((5, 4)), rng.standard_normal(4), rng.standard_normal((2, 4)), rng.standard_normal((5, 4))
    seg = np.array([0, 1, -1, 1, 0])
    y = O.epilogue_ref(lin, bias, "silu", gate, res, seg)
    for m in range(5):
        for n in range(4):
            if seg[m] < 0:
                assert np.isnan(y[m, n])
                continue
            z = lin[m, n] + bias[n]
            assert math.isclose(y[m, n], res[m, n] + gate[seg[m], n] * z / (1 + math.exp(-z)), rel_tol=1e-13)


@pytest.mark.parametrize("adjacent", [False, True])
def test_rotation_against_complex_numbers(adjacent):
    rng = np.random.default_rng(1)
    M, H, D, P = 3, 2, 12, 4
    x, pos = rng.standard_normal((M, H, D)), rng.integers(0, 50, (2, M))
    turns, axes = rng.uniform(0, 0.2, P), np.array([0, 1, 1, 0])
    y = O.rotary_ref(x, pos, turns, axes, adjacent)
    for m in range(M):
        for h in range(H):
            for i in range(P):
                a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + P)
                w = complex(x[m, h, a], x[m, h, b]) * np.exp(2j * math.pi * turns[i] * pos[axes[i], m])
                assert abs(complex(y[m, h, a], y[m, h, b]) - w) < 1e-12
    assert np.array_equal(y[:, :, 2 * P:], x[:, :, 2 * P:])
    # quarter turns are exact permutations up to the cosine of a right angle
    q = O.rotary_ref(x, np.ones((1, M)), np.full(P, 0.25), np.zeros(P, int), adjacent)
    ia, ib = (np.arange(P) * 2, np.arange(P) * 2 + 1) if adjacent else (np.arange(P), np.arange(P) + P)
    assert np.allclose(q[..., ia], -x[..., ib], atol=1e-15) and np.allclose(q[..., ib], x[..., ia], atol=1e-15)


# ------------------------------------------------------------------ frequencies

def test_frequencies():
    turns, axes = ql.rotary_frequencies((24, 20, 20), 5e6, cycle=True, device="cpu")
    assert turns.dtype == torch.float64 and axes.dtype == torch.int32
    assert axes.tolist() == [0, 1, 2] * 20 + [0] * 4
    assert np.allclose(turns.numpy() * 2 * math.pi, 5e6 ** (-np.arange(64) / 64), rtol=1e-15)
    turns, axes = ql.rotary_frequencies((2, 3), 100.0, shared=False, device="cpu")
    assert axes.tolist() == [0, 0, 1, 1, 1]
    assert np.allclose(turns.numpy() * 2 * math.pi, [1, 0.1, 1, 100 ** (-1 / 3), 100 ** (-2 / 3)], rtol=1e-15)
    turns, axes = ql.rotary_frequencies((2, 3), 100.0, shared=False, cycle=True, device="cpu")
    assert axes.tolist() == [0, 1, 0, 1, 1]
    assert np.allclose(turns.numpy() * 2 * math.pi, [1, 1, 0.1, 100 ** (-1 / 3), 100 ** (-2 / 3)], rtol=1e-15)
    assert ql.rotary_frequencies((0, 8), device="cpu")[1].tolist() == [1] * 8
    for bad in ((), (0, 0), (4, -1)):
        with pytest.raises(ValueError):
            ql.rotary_frequencies(bad, device="cpu")
    with pytest.raises(ValueError):
        ql.rotary_frequencies((8,), 0.0, device="cpu")


# ------------------------------------------------------------------ C ABI refusals (no pointer is dereferenced)

P0 = 0x10000000
STEP = 1 << 26
OK, INVALID, ALIGNMENT, UNSUPPORTED, WORKSPACE, CUDA = 0, 1, 2, 3, 4, 5


def _epilogue(L, fn="qlinear_epilogue_forward", M=16, K=256, N=256, group=64, act=1, pt=1, T=2, dt=1, ws=None, ws_bytes=0,
              **at):
    names = ["x", "c", "s", "b", "bias", "gate", "res", "seg", "y"]
    p = {n: P0 + i * STEP for i, n in enumerate(names)}
    p.update(at)
    return getattr(L, fn)(p["x"], p["c"], p["s"], p["b"], p["bias"], act, p["gate"], pt, p["res"], p["seg"], T, p["y"], dt,
                          M, K, N, group, ws, ws_bytes, None)


@pytest.mark.parametrize("fn", ["qlinear_epilogue_forward", "qlinear8_epilogue_forward"])
def test_epilogue_refusals(L, fn):
    bad = lambda **kw: _epilogue(L, fn, **kw)
    assert bad(group=32) == UNSUPPORTED
    assert bad(K=100) == INVALID and bad(N=12) == INVALID and bad(M=0) == INVALID
    assert bad(act=-1) == INVALID and bad(act=4) == INVALID and bad(T=0) == INVALID
    assert bad(pt=2) == INVALID and bad(dt=7) == INVALID
    for k in ("x", "c", "s", "b", "y"):
        assert bad(**{k: None}) == INVALID, k
    for k in ("x", "c", "s", "b", "bias", "gate", "res", "y"):
        assert bad(**{k: P0 + 100 * STEP + 8}) == ALIGNMENT, k
    assert bad(seg=P0 + 100 * STEP + 2) == ALIGNMENT
    for i, k in enumerate(["x", "c", "s", "b", "bias", "gate", None, "seg"]):
        if k:
            assert bad(y=P0 + i * STEP) == INVALID, k     # the output lies on an input
    assert bad(y=P0 + 6 * STEP + 16) == INVALID           # beside the residual, not on it
    if not torch.cuda.is_available():                     # what is right gets as far as the device
        assert bad() == CUDA and bad(y=P0 + 6 * STEP) == CUDA
        assert bad(bias=None, gate=None, res=None, seg=None) == CUDA


def test_epilogue_workspace_sizes(L):
    big = (1 << 64) - 1
    for fn, plain in ((L.qlinear_epilogue_workspace_size, L.qlinear_workspace_size),
                      (L.qlinear8_epilogue_workspace_size, L.qlinear8_workspace_size)):
        for args in ((0, 256, 256, 64), (16, 100, 256, 64), (16, 256, 12, 64), (16, 256, 256, 32)):
            assert fn(*args) == big, args
        for args in ((33, 256, 256, 64), (300, 512, 256, 64), (8, 53248, 4608, 64)):
            assert plain(*args) <= fn(*args) < big, args
        assert fn(8, 256, 256, 64) == fn(32, 256, 256, 64) == 0    # one launch, no scratch
    assert ql.epilogue_workspace_size(33, 256, 64) > 0 and ql.epilogue_workspace_size(33, 256, 64, bits=8) > 0
    with pytest.raises(ValueError):
        ql.epilogue_workspace_size(0, 256, 64)


def _set(i, heads=2, D=64, w=True, **kw):
    f = dict(in_=P0 + 3 * i * STEP, out=P0 + (3 * i + 1) * STEP, in_token=heads * D, in_head=D, out_token=heads * D,
             out_head=D, weight=P0 + (3 * i + 2) * STEP if w else None, heads=heads)
    f.update(kw)
    return Heads(**f)


def _qk(L, q=None, k=None, one=False, dt=1, wt=1, eps=1e-6, pt=0, A=3, P=32, M=4, D=64, **at):
    names = ["pos", "turns", "axes", "seg"]
    p = {n: P0 + (6 + i) * STEP for i, n in enumerate(names)}
    p.update(at)
    q, k = _set(0) if q is None else q, _set(1) if k is None else k
    return L.qlinear_qk_norm_rotary(ctypes.byref(q), None if one else ctypes.byref(k), dt, wt, eps, p["pos"], pt, A,
                                    p["turns"], p["axes"], P, 0, p["seg"], M, D, None)


def _far(fn):
    """A case that passes every check: without a GPU it ends at the device."""
    if not torch.cuda.is_available():
        assert fn() == CUDA


def test_heads_refusals(L):
    for kw in (dict(M=0), dict(D=0), dict(D=60), dict(P=-8), dict(P=40), dict(A=0), dict(A=513), dict(pt=3), dict(pt=-1),
               dict(dt=2), dict(wt=2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(pos=None),
               dict(turns=None), dict(axes=None), dict(q=_set(0, heads=0)), dict(q=_set(0, in_=None)),
               dict(k=_set(1, out=None)), dict(q=_set(0, in_token=-64)), dict(q=_set(0, in_head=1 << 57)),
               dict(q=_set(0, out_head=0)), dict(k=_set(1, out_token=64)), dict(q=_set(0, out_token=0))):
        assert _qk(L, **kw) == INVALID, kw
    assert _qk(L, P=12) == UNSUPPORTED
    big = dict(D=528, q=_set(0, D=528), k=_set(1, D=528))
    assert _qk(L, **big) == UNSUPPORTED
    for kw in (dict(q=_set(0, in_=P0 + 8)), dict(q=_set(0, out=P0 + 20 * STEP + 8)), dict(k=_set(1, weight=P0 + 20 * STEP + 8)),
               dict(q=_set(0, in_token=132)), dict(k=_set(1, out_head=68, out_token=256)), dict(pos=P0 + 20 * STEP + 2),
               dict(pos=P0 + 20 * STEP + 4, pt=1), dict(turns=P0 + 20 * STEP + 4), dict(axes=P0 + 20 * STEP + 2),
               dict(seg=P0 + 20 * STEP + 2)):
        assert _qk(L, **kw) == ALIGNMENT, kw
    # an output on an input: of the other set, off by a little, or with other strides
    for kw in (dict(q=_set(0, out=P0 + 3 * STEP)), dict(k=_set(1, out=P0)), dict(q=_set(0, out=P0 + 16)),
               dict(q=_set(0, out=P0, out_token=256)), dict(q=_set(0, out=P0 + 4 * STEP)), dict(q=_set(0, out=P0 + 5 * STEP)),
               *[dict(q=_set(0, out=P0 + i * STEP)) for i in (2, 6, 7, 8, 9)]):
        assert _qk(L, **kw) == INVALID, kw
    _far(lambda: _qk(L))
    _far(lambda: _qk(L, one=True))
    _far(lambda: _qk(L, P=0, pos=None, turns=None, axes=None))
    _far(lambda: _qk(L, q=_set(0, out=P0), k=_set(1, out=P0 + 3 * STEP)))                  # both in place


def test_heads_inside_one_projection(L):
    """Queries and keys of one packed buffer: in place, or the keys written over themselves while the queries leave."""
    row = (4 + 2 + 2) * 64
    q = _set(0, heads=4, in_token=row, out=P0, out_token=row)
    k = _set(1, heads=2, in_=P0 + 4 * 128, in_token=row, out=P0 + 4 * 128, out_token=row)
    _far(lambda: _qk(L, q=q, k=k))
    # the last query head would land on the first key head
    over = _set(0, heads=4, in_token=row, in_=P0 + 50 * STEP, out=P0 + 128, out_token=row)
    assert _qk(L, q=over, k=k) == INVALID
    # heads kept one behind the other, in one buffer [6][M][D]
    q = _set(0, heads=4, out_token=64, out_head=4 * 64)
    k = _set(1, heads=2, out=P0 + STEP + 4 * 4 * 64 * 2, out_token=64, out_head=4 * 64)
    _far(lambda: _qk(L, q=q, k=k))
    k = _set(1, heads=2, out=P0 + STEP + 3 * 4 * 64 * 2, out_token=64, out_head=4 * 64)
    assert _qk(L, q=q, k=k) == INVALID


def test_rotary_refusals(L):
    def call(x=None, P=32, D=64, M=4, pos=P0 + 6 * STEP):
        x = _set(0, w=False) if x is None else x
        return L.qlinear_rotary_axes(ctypes.byref(x), 1, pos, 0, 3, P0 + 7 * STEP, P0 + 8 * STEP, P, 1, None, M, D, None)
    assert call(P=0) == INVALID                            # nothing to do
    assert call(x=_set(0)) == INVALID                      # a weight without norms
    assert call(pos=None) == INVALID and call(M=0) == INVALID
    assert L.qlinear_rotary_axes(None, 1, P0, 0, 3, P0, P0, 32, 1, None, 4, 64, None) == INVALID
    _far(call)


# ------------------------------------------------------------------ the Python binding

def test_the_binding_lays_out_a_set_of_heads():
    """The bytes that the binding passes are the C struct's."""
    from group_wise_affine_qlinear_b200 import _heads
    x = torch.zeros((4, 6, 32), dtype=torch.bfloat16)
    t, o, w = x[:, 1:4], torch.zeros((3, 4, 32), dtype=torch.bfloat16).transpose(0, 1), torch.zeros(32)
    raw = _heads._entry(t, o, w)
    assert len(raw) == ctypes.sizeof(Heads)
    h = Heads.from_buffer_copy(raw)
    assert (h.in_, h.out, h.weight, h.heads) == (t.data_ptr(), o.data_ptr(), w.data_ptr(), 3)
    assert (h.in_token, h.in_head, h.out_token, h.out_head) == (192, 32, 32, 128)
    assert Heads.from_buffer_copy(_heads._entry(t, o, None)).weight is None


def test_host_tensors_are_refused():
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    w = (torch.zeros((64, 32), dtype=torch.int32), torch.zeros((64, 4), dtype=torch.float16),
         torch.zeros((64, 4), dtype=torch.float16))
    w8 = (torch.zeros((64, 64), dtype=torch.int32),) + w[1:]
    h = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    pos, rot = torch.zeros((3, 4), dtype=torch.int32), ql.rotary_frequencies((16, 8, 8), device="cpu")
    for call in (lambda: ql.forward_epilogue(x, *w), lambda: ql.forward8_epilogue(x, *w8),
                 lambda: ql.rotary_axes(h, pos, rot), lambda: ql.qk_norm_rotary(h, h, pos, rot)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_what_is_no_tensor_is_refused():
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    w = (torch.zeros((64, 32), dtype=torch.int32), torch.zeros((64, 4), dtype=torch.float16),
         torch.zeros((64, 4), dtype=torch.float16))
    for kw in (dict(bias=1.0), dict(gate=x[0]), dict(residual=[1]), dict(activation="relu"), dict(out_dtype=torch.float16),
               dict(out=3)):
        with pytest.raises(ValueError):
            ql.forward_epilogue(x, *w, **kw)
    h = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    rot = ql.rotary_frequencies((16, 8, 8), device="cpu")
    for call in (lambda: ql.rotary_axes(x, None, rot), lambda: ql.rotary_axes("x", None, rot),
                 lambda: ql.qk_norm_rotary(h, "k"), lambda: ql.qk_norm_rotary(h.half())):
        with pytest.raises(ValueError):
            call()
