"""GPU parity of the norms of queries and keys and their rotation by positions of several axes, against float64.

Bounds, with u = 2^-24 (half an fp32 unit) and b = 2^-8 (half a bf16 unit, relative):
  norm      a sum of at most 512 squares, 16 per lane and then a tree, errs by at most 24 u relative, its root by half
            of that, the hardware's reciprocal root by 4 u, three products by 3 u: |e_n| <= 20 u |n|
  angle     the product with a position errs by 2^-53 of its turns, the rest of a turn by 2^-26 when rounded: 2 pi
            (2^-26 + 2^-52 |turns pos|); its sine and cosine by another 4 u: e_t in all, for either
  pair      a cos - b sin errs by e_t (|a| + |b|) + 3 u (|a| + |b|) beside e_n; + b |out| for bf16 storage
"""
import math

import numpy as np
import pytest
import torch

import group_wise_affine_qlinear_b200 as ql
from oracle import qlinear_oracle as O

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
POS = {"int32": torch.int32, "int64": torch.int64, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required for -m gpu tests")
    ql.lib()
    yield
    assert ql.device_status() == 0


def _f64(t):
    return None if t is None else t.double().cpu().numpy()


def _rand(rng, shape, dt, scale=2.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).cuda().to(dt)


def _rotary(rng, P, A, rate=0.2):
    turns = torch.from_numpy(rng.uniform(0, rate, P)).cuda()
    return turns, torch.from_numpy(rng.integers(0, A, P).astype(np.int32)).cuda()


def _positions(rng, A, M, kind, far=0):
    v = rng.integers(0, 100, (A, M)) + far
    return torch.from_numpy(v * 0.625 if kind == "f32" else v).cuda().to(POS[kind])


def _check(got, x, weight, pos, rot, adjacent, norm, eps=1e-6, rows=None):
    """got [M][H][D] against the definition, on the given rows."""
    if rows is not None:
        ix = torch.from_numpy(np.asarray(rows)).to(x.device)
        got, x, pos = got[ix], x[ix], None if pos is None else pos[:, ix]
    dt = got.dtype
    n = _f64(x)
    if norm:
        n = O.rms_normed(n, eps)
        if weight is not None:
            n = n * _f64(weight)
    want, size = n, np.abs(n)
    bound = 20 * U * np.abs(n) if norm else np.zeros_like(n)
    if rot is not None:
        turns, axes = _f64(rot[0]), rot[1].cpu().numpy()
        want = O.rotary_ref(n, _f64(pos), turns, axes, adjacent)
        P = len(turns)
        t = np.abs(_f64(pos)[axes].T * turns[None, :])
        et = (2 * math.pi * (2.0 ** -26 + 2.0 ** -52 * t) + 4 * U)[:, None, :]
        ia, ib = (np.arange(P) * 2, np.arange(P) * 2 + 1) if adjacent else (np.arange(P), np.arange(P) + P)
        pair = np.abs(n[:, :, ia]) + np.abs(n[:, :, ib])
        extra = (et + 3 * U + (20 * U if norm else 0.0)) * pair
        bound = bound.copy()
        bound[:, :, ia] = extra
        bound[:, :, ib] = extra
    if dt == torch.bfloat16:
        bound = bound + B * (np.abs(want) + bound)
    err = np.abs(_f64(got) - want)
    assert np.all(err <= bound + 1e-38), float((err / (bound + 1e-38)).max())


CASES = [  # M, Hq, Hk, D, P, A
    (1, 1, 1, 16, 8, 1), (1, 18, 18, 256, 128, 3), (3, 5, 1, 64, 32, 3), (7, 4, 4, 80, 40, 2), (19, 3, 1, 96, 16, 3),
    (50, 7, 7, 128, 64, 3), (33, 6, 2, 160, 80, 4), (65, 2, 1, 192, 64, 3), (200, 18, 6, 256, 64, 3), (9, 2, 2, 512, 256, 3),
    (11, 3, 3, 24, 8, 2), (5, 36, 4, 136, 64, 3), (4, 33, 11, 8, 0, 0), (6, 1, 1, 264, 128, 3), (40, 2, 2, 64, 0, 0),
    (6000, 3, 1, 64, 32, 3), (2500, 4, 2, 256, 128, 3),
    (9601, 1, 1, 64, 32, 3), (5003, 5, 1, 96, 48, 3), (4801, 9, 3, 128, 40, 3), (2407, 7, 7, 200, 64, 2)]   # several tokens a warp


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("M,Hq,Hk,D,P,A", CASES)
def test_norms_and_rotation(M, Hq, Hk, D, P, A, adjacent, dt):
    """Queries and keys inside one packed projection, out of place, then head by head, then in place."""
    rng = np.random.default_rng(M + D + P + Hq)
    kind = ["int32", "int64", "f32"][(M + D) % 3]
    qkv = _rand(rng, (M, Hq + 2 * Hk, D), DT[dt])
    kept = qkv.clone()
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    wt = DT["f32" if (M + P) % 2 else "bf16"]
    qw, kw = _rand(rng, D, wt, 1.0), (_rand(rng, D, wt, 1.0) if M != 7 else None)
    rot, pos = (_rotary(rng, P, A), _positions(rng, A, M, kind)) if P else (None, None)
    qo, ko = ql.qk_norm_rotary(q, k, pos, rot, q_weight=qw, k_weight=kw, adjacent=adjacent)
    assert torch.equal(qkv, kept) and qo.is_contiguous() and ko.is_contiguous()
    _check(qo, q, qw, pos, rot, adjacent, True)
    _check(ko, k, kw, pos, rot, adjacent, True)
    by_head = torch.full((Hq + Hk, M, D), 3.0, dtype=DT[dt], device="cuda")
    a, b = by_head[:Hq].transpose(0, 1), by_head[Hq:].transpose(0, 1)
    ql.qk_norm_rotary(q, k, pos, rot, q_weight=qw, k_weight=kw, adjacent=adjacent, q_out=a, k_out=b)
    assert torch.equal(a, qo) and torch.equal(b, ko)
    ql.qk_norm_rotary(q, k, pos, rot, q_weight=qw, k_weight=kw, adjacent=adjacent, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(qkv[:, Hq + Hk:], kept[:, Hq + Hk:])
    one = ql.qk_norm_rotary(kept[:, :Hq], None, pos, rot, q_weight=qw, adjacent=adjacent)
    assert torch.equal(one[0], qo) and one[1] is None


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("M,H,D,P,A", [(1, 18, 256, 128, 3), (4, 1, 64, 32, 1), (130, 3, 80, 24, 3), (999, 24, 128, 64, 3)])
def test_rotation_alone(M, H, D, P, A, adjacent, dt):
    rng = np.random.default_rng(M + D)
    x, rot, pos = _rand(rng, (M, H, D), DT[dt]), _rotary(rng, P, A), _positions(rng, A, M, "f32")
    y = ql.rotary_axes(x, pos, rot, adjacent=adjacent)
    _check(y, x, None, pos, rot, adjacent, False)
    assert torch.equal(y[..., 2 * P:], x[..., 2 * P:])
    strided = torch.zeros((M, H + 2, 2 * D), dtype=DT[dt], device="cuda")[:, 1:H + 1, :D]
    assert ql.rotary_axes(x, pos, rot, adjacent=adjacent, out=strided) is strided
    assert torch.equal(strided, y)
    ql.rotary_axes(x, pos, rot, adjacent=adjacent, out=x)
    assert torch.equal(x, y)


@pytest.mark.parametrize("kind,far", [("int32", 2 ** 31 - 200), ("int64", 2 ** 40), ("f32", 2 ** 22), ("int32", -5000)])
def test_far_positions(kind, far):
    """Angles of millions of turns: in 32 bits their product would be off by whole radians."""
    rng = np.random.default_rng(8)
    x = _rand(rng, (40, 2, 64), torch.float32)
    rot, pos = ql.rotary_frequencies((12, 10, 10), 1e4, cycle=True), _positions(rng, 3, 40, kind, far)
    _check(ql.rotary_axes(x, pos, rot), x, None, pos, rot, False, False)


@pytest.mark.parametrize("M", [12, 3000, 11000])
def test_padding_rows_are_left_alone(M):
    rng = np.random.default_rng(9)
    x, rot, pos = _rand(rng, (M, 5, 64), torch.bfloat16), _rotary(rng, 32, 3), _positions(rng, 3, M, "int32")
    seg = rng.integers(-2, 3, M).astype(np.int32)
    seg[M - 3:] = -1
    pad = torch.from_numpy(seg < 0).cuda()
    x[pad] = float("nan")
    out = torch.full_like(x, 4.0)
    ql.qk_norm_rotary(x, None, pos, rot, segment_ids=torch.from_numpy(seg).cuda(), q_out=out)
    assert (out[pad] == 4.0).all()
    _check(out, x, None, pos, rot, False, True, rows=np.flatnonzero(seg >= 0))


@pytest.mark.parametrize("adjacent", [False, True])
def test_axes_out_of_range(adjacent):
    """A pair whose axis does not exist is not turned, and is reported."""
    rng = np.random.default_rng(10)
    x, (turns, axes), pos = _rand(rng, (9, 2, 64), torch.float32), _rotary(rng, 32, 3), _positions(rng, 3, 9, "int32")
    axes[4], axes[17] = 3, -1
    y = ql.rotary_axes(x, pos, (turns, axes), adjacent=adjacent)
    assert ql.device_status() == 1
    turns, axes = turns.clone(), axes.clone()
    turns[4] = turns[17] = 0.0
    axes[4] = axes[17] = 0
    _check(y, x, None, pos, (turns, axes), adjacent, False)


def test_what_is_not_finite_stays_in_its_head():
    rng = np.random.default_rng(11)
    x, rot, pos = _rand(rng, (30, 4, 96), torch.bfloat16), _rotary(rng, 40, 3), _positions(rng, 3, 30, "int32")
    clean = ql.rotary_axes(x, pos, rot)
    x[7, 2, 90] = float("inf")                              # behind the turned part
    x[8, 1, 3] = float("nan")
    y = ql.rotary_axes(x, pos, rot)
    assert y[7, 2, 90] == float("inf") and torch.isnan(y[8, 1, 3]) and torch.isnan(y[8, 1, 43])
    same = torch.ones_like(y, dtype=torch.bool)
    same[7, 2, 90] = same[8, 1, 3] = same[8, 1, 43] = False
    assert torch.equal(y[same], clean[same])
    n, _ = ql.qk_norm_rotary(x, None, pos, rot)
    assert torch.isnan(n[8, 1]).all() and torch.isfinite(n[8, 0]).all() and torch.isfinite(n[7, 1]).all()


def test_rows_of_zeros_and_magnitudes():
    x = torch.zeros((6, 2, 64), dtype=torch.float32, device="cuda")
    x[1], x[2], x[3] = 1e-30, 1e18, 1e-3
    n, _ = ql.qk_norm_rotary(x, None, eps=1e-6)
    assert (n[0] == 0).all() and torch.isfinite(n).all()
    _check(n, x, None, None, None, False, True)
    z, _ = ql.qk_norm_rotary(x[2:4], None, eps=0.0)
    assert torch.allclose(z, torch.ones_like(z), rtol=1e-6)


def test_broadcast_inputs_and_offsets_past_32_bits():
    rng = np.random.default_rng(12)
    rot = _rotary(rng, 32, 3)
    one = _rand(rng, (1, 1, 64), torch.bfloat16)
    x = one.expand(10, 3, 64)                               # strides of zero: read alike, written apart
    pos = _positions(rng, 3, 10, "int32")
    _check(ql.rotary_axes(x, pos, rot), x, None, pos, rot, False, False)
    M, row = 70_000, 1 << 16
    buf = torch.zeros((M, row), dtype=torch.bfloat16, device="cuda")
    q = buf[:, row - 128:].view(M, 2, 64)
    q.copy_(_rand(rng, (M, 2, 64), torch.bfloat16))
    pos = _positions(rng, 3, M, "int32")
    before = q.clone()
    ql.qk_norm_rotary(q, None, pos, rot, q_out=q)
    _check(q, before, None, pos, rot, False, True, rows=[0, 1, 32767, 32768, 65535, 65536, M - 1])
    assert not buf[:, :row - 128].any()


def test_replays_and_streams():
    rng = np.random.default_rng(13)
    M = 100
    qkv = _rand(rng, (M, 12, 128), torch.bfloat16)
    q, k, rot, pos = qkv[:, :4], qkv[:, 4:8], _rotary(rng, 64, 3), _positions(rng, 3, M, "int32")
    want = ql.qk_norm_rotary(q, k, pos, rot)
    outs = [torch.empty((M, 4, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            ql.qk_norm_rotary(q, k, pos, rot, q_out=outs[0], k_out=outs[1])
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for o in outs:
            o.fill_(0)
        graph.replay()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    torch.cuda.synchronize()
    got = [ql.qk_norm_rotary(q, k, pos, rot, stream=torch.cuda.Stream()) for _ in range(3)]
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_refusals():
    rng = np.random.default_rng(14)
    x, rot, pos = _rand(rng, (8, 4, 64), torch.bfloat16), _rotary(rng, 32, 3), _positions(rng, 3, 8, "int32")
    w = _rand(rng, 64, torch.float32)
    bad = [lambda: ql.qk_norm_rotary(x, x[:-1], pos, rot), lambda: ql.qk_norm_rotary(x, x.float(), pos, rot),
           lambda: ql.qk_norm_rotary(x, None, pos, None), lambda: ql.qk_norm_rotary(x, None, None, rot),
           lambda: ql.qk_norm_rotary(x, None, pos, rot, k_weight=w), lambda: ql.qk_norm_rotary(x, None, pos, rot, q_weight=w[:-1]),
           lambda: ql.qk_norm_rotary(x, x, pos, rot, q_weight=w, k_weight=w.bfloat16()),
           lambda: ql.qk_norm_rotary(x, None, pos.short(), rot), lambda: ql.qk_norm_rotary(x, None, pos[:, :-1], rot),
           lambda: ql.qk_norm_rotary(x, None, pos, (rot[0].float(), rot[1])), lambda: ql.qk_norm_rotary(x, None, pos, (rot[0], rot[1].long())),
           lambda: ql.qk_norm_rotary(x, None, pos, (rot[0], rot[1][:-1])), lambda: ql.rotary_axes(x, None, None),
           lambda: ql.rotary_axes(x[..., ::2], pos, rot), lambda: ql.rotary_axes(x, pos, rot, out=torch.empty_like(x)[:, :3]),
           lambda: ql.rotary_axes(x, pos.cpu(), rot), lambda: ql.rotary_axes(x[:, :, :48], pos, rot),
           lambda: ql.rotary_axes(x, pos, rot, segment_ids=torch.zeros(7, dtype=torch.int32, device="cuda"))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call, status in ((lambda: ql.rotary_axes(x, pos, (rot[0][:12], rot[1][:12])), 3),
                         (lambda: ql.rotary_axes(x[:, 0:3], pos, rot, out=x[:, 1:4]), 1),
                         (lambda: ql.qk_norm_rotary(x[:, :2], x[:, 2:], pos, rot, q_out=x[:, 1:3]), 1),
                         (lambda: ql.rotary_axes(x, pos, rot, out=torch.empty((8, 1, 64), dtype=x.dtype, device="cuda").expand(8, 4, 64)), 1),
                         (lambda: ql.rotary_axes(torch.zeros(8 * 4 * 64 + 4, dtype=x.dtype, device="cuda")[4:].view(8, 4, 64), pos, rot), 2)):
        with pytest.raises(ql.QLinearError) as e:
            call()
        assert e.value.status == status
