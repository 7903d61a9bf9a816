"""Adapters beside the packed layer and the norms around a block, on a host without a GPU: the oracle's formulas
against brute force, the C ABI's refusals (before any launch) and the Python binding's."""
import numpy as np
import pytest
import torch

import group_wise_affine_qlinear_b200 as ql
from group_wise_affine_qlinear_b200 import build as qb
from group_wise_affine_qlinear_b200 import synthetic as S
from oracle import qlinear_oracle as O


@pytest.fixture(scope="module")
def L():
    qb.build()
    return ql.lib()


# ------------------------------------------------------------------ the oracle against brute force

def test_lora_delta_equals_a_triple_loop():
    rng = np.random.default_rng(0)
    M, K, N, n, r = 5, 16, 6, 3, 4
    bits = lambda *shape: S.f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32))
    x, a, b = bits(M, K), bits(n, r, K), bits(n, N, r)
    s, ids = rng.uniform(0.5, 2.0, n), np.array([2, -1, 0, 2, 1])
    got = O.lora_delta(x, a, b, s, ids)
    xv, av, bv = O.decode_bf16(x), O.decode_bf16(a), O.decode_bf16(b)
    for m in range(M):
        for col in range(N):
            want = 0.0
            if ids[m] >= 0:
                i = ids[m]
                for j in range(r):
                    want += sum(xv[m, k] * av[i, j, k] for k in range(K)) * bv[i, col, j] * s[i]
            assert abs(got[m, col] - want) <= 1e-12 * (1.0 + abs(want))
    assert np.array_equal(O.lora_delta(x, a, b, None, ids), O.lora_delta(x, a, b, np.ones(n), ids))


def test_norm_residual_ref_equals_elementwise_loops():
    rng = np.random.default_rng(1)
    M, D, T = 3, 8, 2
    x, y = rng.standard_normal((M, D)), rng.standard_normal((2, M, D))
    pw, qw = rng.standard_normal(D), rng.standard_normal(D)
    gate, sc, sh = (rng.standard_normal((T, D)) for _ in range(3))
    seg = np.array([1, 0, 1])
    r, h = O.norm_residual_ref(x, y, True, pw, gate, 0.5, 2.0, True, qw, sc, sh, seg, 1e-3)
    for m in range(M):
        v = [y[0, m, d] + y[1, m, d] for d in range(D)]
        n1 = (sum(e * e for e in v) / D + 1e-3) ** 0.5
        rr = [0.5 * x[m, d] + 2.0 * gate[seg[m], d] * v[d] / n1 * pw[d] for d in range(D)]
        n2 = (sum(e * e for e in rr) / D + 1e-3) ** 0.5
        for d in range(D):
            assert abs(r[m, d] - rr[d]) <= 1e-12
            assert abs(h[m, d] - (rr[d] / n2 * qw[d] * (1 + sc[seg[m], d]) + sh[seg[m], d])) <= 1e-12
    assert np.array_equal(O.norm_residual_ref(x)[0], x)
    assert O.norm_residual_ref(x, y, pre_norm=False)[1] is None


# ------------------------------------------------------------------ C ABI refusals (no pointer is dereferenced)

P = 0x10000000
STEP = 1 << 26
OK, INVALID, ALIGNMENT, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4


def _ptrs(n):
    return [P + i * STEP for i in range(n)]


def _lora(L, fn="qlinear_lora_forward", M=16, K=256, N=256, group=64, n=2, r=16, dt=1, ws=None, ws_bytes=0, **at):
    names = ["x", "c", "s", "b", "la", "lb", "ls", "ids", "y"]
    p = dict(zip(names, _ptrs(9)))
    p.update(at)
    return getattr(L, fn)(*[p[k] for k in names], dt, M, K, N, group, n, r, ws, ws_bytes, None)


@pytest.mark.parametrize("fn", ["qlinear_lora_forward", "qlinear8_lora_forward"])
def test_lora_forward_refusals(L, fn):
    bad = lambda **kw: _lora(L, fn, **kw)
    assert bad(group=32) == UNSUPPORTED
    assert bad(K=100) == INVALID and bad(N=12) == INVALID and bad(M=0) == INVALID
    assert bad(n=0) == INVALID and bad(r=0) == INVALID and bad(n=-1) == INVALID
    assert bad(r=12) == UNSUPPORTED and bad(r=136) == UNSUPPORTED
    for k in ("x", "c", "s", "b", "la", "lb", "ids", "y"):
        assert bad(**{k: None}) == INVALID, k
    for k in ("x", "c", "s", "b", "la", "lb", "y"):
        assert bad(**{k: P + 100 * STEP + 4}) == ALIGNMENT, k
    for k in ("ls", "ids"):
        assert bad(**{k: P + 100 * STEP + 2}) == ALIGNMENT, k
    assert bad(dt=7) == INVALID
    for i, k in enumerate(["x", "c", "s", "b", "la", "lb", "ls", "ids"]):
        assert bad(y=P + i * STEP) == INVALID, k          # the output lies on an input


def test_lora_workspace_sizes(L):
    for fn in (L.qlinear_lora_workspace_size, L.qlinear8_lora_workspace_size, L.qlinear_swiglu_lora_workspace_size):
        big = (1 << 64) - 1
        assert fn(16, 256, 256, 64, 2, 16) < big
        for args in ((0, 256, 256, 64, 2, 16), (16, 100, 256, 64, 2, 16), (16, 256, 12, 64, 2, 16),
                     (16, 256, 256, 32, 2, 16), (16, 256, 256, 64, 0, 16), (16, 256, 256, 64, 2, 12),
                     (16, 256, 256, 64, 2, 0), (16, 256, 256, 64, 2, 136)):
            assert fn(*args) == big, args
    # at least the layer's own scratch and t, fp32 [M][r]
    assert L.qlinear_lora_workspace_size(300, 512, 256, 64, 3, 24) >= \
        L.qlinear_workspace_size(300, 512, 256, 64) + 300 * 24 * 4


def _swiglu(L, M=16, K=256, I=256, group=64, n=2, r=16, dt=1, ws=None, ws_bytes=0, **at):
    names = ["x", "gc", "gs", "gb", "uc", "us", "ub", "gla", "glb", "ula", "ulb", "ls", "ids", "h"]
    p = dict(zip(names, _ptrs(14)))
    p.update(at)
    return L.qlinear_swiglu_lora_forward(*[p[k] for k in names], dt, M, K, I, group, n, r, ws, ws_bytes, None)


def test_swiglu_lora_refusals(L):
    assert _swiglu(L, group=32) == UNSUPPORTED and _swiglu(L, M=0) == INVALID
    assert _swiglu(L, r=4) == UNSUPPORTED and _swiglu(L, n=0) == INVALID
    for k in ("gla", "glb", "ula", "ulb", "ids", "x", "uc", "h"):
        assert _swiglu(L, **{k: None}) == INVALID, k
        assert _swiglu(L, **{k: P + 100 * STEP + 2}) == ALIGNMENT, k
    for i, k in enumerate(["x", "gc", "gs", "gb", "uc", "us", "ub", "gla", "glb", "ula", "ulb", "ls", "ids"]):
        assert _swiglu(L, h=P + i * STEP) == INVALID, k


def _norm(L, xt=1, yt=1, S_=1, post=1, pt=1, T=2, eps=1e-6, M=4, D=64, **at):
    names = ["x", "y", "pw", "g", "qw", "sc", "sh", "seg", "out", "h"]
    p = dict(zip(names, _ptrs(10)))
    p.update(at)
    return L.qlinear_norm_residual(p["x"], xt, p["y"], yt, S_, post, p["pw"], p["g"], 1.0, 1.0, p["qw"], p["sc"],
                                   p["sh"], pt, p["seg"], T, eps, p["out"], p["h"], M, D, None)


def test_norm_residual_refusals(L):
    for kw in (dict(M=0), dict(D=0), dict(D=12), dict(T=0), dict(S_=0), dict(S_=2), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(xt=3), dict(yt=3), dict(pt=3), dict(x=None),
               dict(out=None), dict(post=0), dict(h=None),
               dict(y=None), dict(y=None, out=None, h=None, qw=None, sc=None, sh=None)):
        assert _norm(L, **kw) == INVALID, kw
    assert _norm(L, D=32768 + 8) == UNSUPPORTED
    for k in ("x", "y", "pw", "g", "qw", "sc", "sh", "out", "h"):
        assert _norm(L, **{k: P + 100 * STEP + 8}) == ALIGNMENT, k
    assert _norm(L, seg=P + 100 * STEP + 2) == ALIGNMENT
    for i, k in enumerate(["x", "y", "pw", "g", "qw", "sc", "sh", "seg"]):
        assert _norm(L, h=P + i * STEP) == INVALID, k
        if k != "x":
            assert _norm(L, out=P + i * STEP) == INVALID, k
    assert _norm(L, out=P + 16) == INVALID                # beside x, not on it
    assert _norm(L, out=P + 9 * STEP) == INVALID          # on h


# ------------------------------------------------------------------ the Python binding

def test_host_tensors_are_refused():
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    w = (torch.zeros((64, 32), dtype=torch.int32), torch.zeros((64, 4), dtype=torch.float16),
         torch.zeros((64, 4), dtype=torch.float16))
    w8 = (torch.zeros((64, 64), dtype=torch.int32),) + w[1:]
    a, b = torch.zeros((2, 8, 256), dtype=torch.bfloat16), torch.zeros((2, 64, 8), dtype=torch.bfloat16)
    ids = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: ql.forward_lora(x, *w, a, b, ids), lambda: ql.forward8_lora(x, *w8, a, b, ids),
                 lambda: ql.swiglu_lora(x, w, w, (a, b), (a, b), ids), lambda: ql.norm_residual(x),
                 lambda: ql.norm_residual(x, x)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_workspace_size_refusals():
    assert ql.lora_workspace_size(4, 256, 64, 2, 8) > 0 and ql.lora_workspace_size(4, 256, 64, 2, 8, bits=8) > 0
    assert ql.swiglu_lora_workspace_size(4, 256, 64, 2, 8) > 0
    for fn in (ql.lora_workspace_size, ql.swiglu_lora_workspace_size):
        for args in ((4, 256, 64, 2, 9), (4, 256, 64, 0, 8), (0, 256, 64, 2, 8), (4, 256, 64, 2, 256)):
            with pytest.raises(ValueError):
                fn(*args)
