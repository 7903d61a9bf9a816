"""GPU parity of the norms around a block (norm_residual) against the oracle in float64.

Bounds, with u = 2^-24 (half an fp32 unit) and b = 2^-8 (half a bf16 unit, relative):
  post norm   a sum of squares errs by at most (32 + 16) u relative (at most 32 terms per thread, then trees), its
              root by half of that; with the division, the products by weight and gate, and the S - 1 additions of the
              partials, v errs by 40 u |v| + S u sum_z |y_z| |v| / |sum_z y_z|
  r           one product, one fused addition: 3 u (|c_x x| + |c_y g v|) more; + b |r| for bf16 storage
  h           r's own error passes through the norm: relative to the row 2 kappa of it, kappa = sum |e_r| |r| / sum r^2;
              then 40 u of the value, the modulation's 4 u (|n| + |shift|), and b |h|
"""
import numpy as np
import pytest
import torch

import group_wise_affine_qlinear_b200 as ql
from oracle import qlinear_oracle as O

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required for -m gpu tests")
    ql.lib()
    yield
    assert ql.device_status() == 0


def _f64(t):
    return None if t is None else t.double().cpu().numpy()


def _make(rng, M, D, T=1, x32=False, y="bf16", S=1, params32=False, full=True):
    def dev(v, f32):
        return torch.from_numpy(np.asarray(v, np.float32)).cuda().to(torch.float32 if f32 else torch.bfloat16)
    x = dev(3 * rng.standard_normal((M, D)), x32)
    yt = None if y is None else dev(rng.standard_normal((S, M, D) if y == "f32" else (M, D)), y == "f32")
    kw = {}
    if full:
        if y is not None:
            kw["post_weight"] = dev(1 + 0.2 * rng.standard_normal(D), params32)
            kw["gate"] = dev(0.5 * rng.standard_normal((T, D)), params32)
        kw["pre_weight"] = dev(1 + 0.2 * rng.standard_normal(D), params32)
        kw["scale"] = dev(0.2 * rng.standard_normal((T, D)), params32)
        kw["shift"] = dev(0.2 * rng.standard_normal((T, D)), params32)
    if T > 1:
        kw["segment_ids"] = torch.from_numpy(rng.integers(0, T, M).astype(np.int32)).cuda()
    return x, yt, kw


def _check(x, y, r, h, kw, rows=None):
    kw = dict(kw)
    seg = kw.pop("segment_ids", None)
    seg = np.zeros(x.shape[0], np.int64) if seg is None else seg.cpu().numpy()
    rows = np.flatnonzero(seg >= 0) if rows is None else rows
    ix = torch.from_numpy(rows).to(x.device)
    xv = _f64(x[ix])
    yv = None if y is None else _f64(y[:, ix] if y.dim() == 3 else y[ix][None])
    seg = seg[rows]
    for k in ("post_weight", "gate", "pre_weight", "scale", "shift"):
        if k in kw:
            kw[k] = _f64(kw[k])
    rr, hr = O.norm_residual_ref(xv, yv, seg=seg, **kw)
    er = np.zeros_like(rr)
    if y is not None:
        v = (rr - kw.get("residual_scale", 1.0) * xv)
        s = yv.sum(0)
        part = len(yv) * U * np.abs(yv).sum(0) * np.abs(v) / np.maximum(np.abs(s), 1e-30)
        er = 43 * U * np.abs(v) + part + 3 * U * np.abs(kw.get("residual_scale", 1.0) * xv)
        stored = er + (B if r.dtype == torch.bfloat16 else U) * np.abs(rr)
        d = np.abs(_f64(r[ix]) - rr)
        assert np.all(d <= stored), (d / stored).max()
    if h is not None:
        eps = kw.get("eps", 1e-6)
        inv = 1.0 / np.sqrt((rr * rr).mean(-1, keepdims=True) + eps)
        kappa = (er * np.abs(rr)).sum(-1, keepdims=True) / np.maximum((rr * rr).sum(-1, keepdims=True), 1e-300)
        gain = np.abs(kw.get("pre_weight", 1.0) * (1.0 + (kw["scale"][seg] if "scale" in kw else 0.0)))
        n = np.abs(rr) * inv * gain
        shift = np.abs(kw["shift"][seg]) if "shift" in kw else 0.0
        bound = er * inv * gain + (2 * kappa + 44 * U) * n + 4 * U * shift + B * np.abs(hr)
        # (1 + scale) is formed inside a fused product: relative to |n| before it when scale nears -1
        bound = bound + 4 * U * np.abs(rr) * inv * np.abs(kw.get("pre_weight", 1.0))
        d = np.abs(_f64(h[ix]) - hr)
        assert np.all(d <= bound * (1 + B)), (d / bound).max()


SHAPES = [(1, 8), (1, 4608), (2, 64), (3, 256), (5, 264), (33, 512), (17, 520), (64, 1024), (9, 1032), (13, 2048),
          (40, 4104), (400, 1544), (300, 4608), (3, 8192), (2, 8200), (310, 8200), (2, 16392), (301, 16392),
          (1, 32768), (2, 32760)]


@pytest.mark.parametrize("M,D", SHAPES)
def test_both_norms(M, D):
    rng = np.random.default_rng(M * 7 + D)
    x, y, kw = _make(rng, M, D, T=min(3, M))
    kw.update(residual_scale=0.75, branch_scale=1.5, eps=1e-5)
    r, h = ql.norm_residual(x, y, **kw)
    _check(x, y, r, h, kw)


@pytest.mark.parametrize("x32", [False, True])
@pytest.mark.parametrize("y,S", [("bf16", 1), ("f32", 1), ("f32", 2), ("f32", 5), (None, 1)])
@pytest.mark.parametrize("params32", [False, True])
@pytest.mark.parametrize("M,D", [(7, 96), (3, 4608), (350, 2056)])
def test_types(x32, y, S, params32, M, D):
    rng = np.random.default_rng(M + D + S)
    x, yt, kw = _make(rng, M, D, T=2, x32=x32, y=y, S=S, params32=params32)
    r, h = ql.norm_residual(x, yt, **kw)
    if yt is None:
        assert r is x
    _check(x, yt, r, h, kw)


def test_every_argument_is_optional():
    rng = np.random.default_rng(3)
    for M, D in ((6, 128), (3, 2056)):
        x, y, full = _make(rng, M, D, T=2)
        for drop in ("post_weight", "gate", "pre_weight", "scale", "shift"):
            kw = {k: v for k, v in full.items() if k != drop}
            r, h = ql.norm_residual(x, y, **kw)
            _check(x, y, r, h, kw)
        r, h = ql.norm_residual(x, y)
        _check(x, y, r, h, {})
        kw = {"post_norm": False, "gate": full["gate"], "segment_ids": full["segment_ids"]}
        r, h = ql.norm_residual(x, y, **kw)
        _check(x, y, r, h, kw)
        kw = {"pre_norm": False, "post_weight": full["post_weight"]}
        r, h = ql.norm_residual(x, y, **kw)
        assert h is None
        _check(x, y, r, h, kw)


def test_update_in_place_and_given_outputs():
    rng = np.random.default_rng(4)
    for M, D, x32 in ((5, 264, False), (4, 4608, True)):
        x, y, kw = _make(rng, M, D, x32=x32)
        r, h = ql.norm_residual(x, y, **kw)
        x2, h2 = x.clone(), torch.full((M, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        r3, h3 = ql.norm_residual(x2, y, out=x2, h=h2, **kw)
        assert r3 is x2 and h3 is h2 and torch.equal(x2, r) and torch.equal(h2, h)


@pytest.mark.parametrize("M,D", [(37, 512), (37, 4608)])
def test_padding_rows_are_left_alone(M, D):
    rng = np.random.default_rng(5)
    x, y, kw = _make(rng, M, D, T=2)
    seg = kw["segment_ids"]
    seg[11], seg[30:] = -1, -1
    live = seg >= 0
    clean, clean_h = ql.norm_residual(x, y, **kw)
    x[~live], y[~live] = float("nan"), float("inf")      # what lies there must not matter
    out = torch.full_like(x, 7.0)
    h = torch.full((M, D), -3.0, dtype=torch.bfloat16, device="cuda")
    ql.norm_residual(x, y, out=out, h=h, **kw)
    assert torch.equal(out[live], clean[live]) and torch.equal(h[live], clean_h[live])
    assert (out[~live] == 7.0).all() and (h[~live] == -3.0).all()
    _check(x, y, out, h, kw)


def test_segment_out_of_range_is_recorded_and_left_alone():
    rng = np.random.default_rng(6)
    for D in (256, 2056):
        x, y, kw = _make(rng, 6, D, T=2)
        kw["segment_ids"][4] = 2
        out, h = torch.full_like(x, 7.0), torch.full((6, D), -3.0, dtype=torch.bfloat16, device="cuda")
        ql.norm_residual(x, y, out=out, h=h, **kw)
        assert ql.device_status() == 1
        assert (out[4] == 7.0).all() and (h[4] == -3.0).all()
        _check(x, y, out, h, kw, rows=np.array([0, 1, 2, 3, 5]))


def test_zero_and_non_finite_rows():
    rng = np.random.default_rng(7)
    for D in (128, 4608):
        x, y, kw = _make(rng, 8, D)
        r0, h0 = ql.norm_residual(x, y, **kw)
        x[1], y[1] = 0, 0                                  # a zero row: r = 0, h = shift
        y[2, 5] = float("nan")
        x[3, 0] = float("inf")
        r, h = ql.norm_residual(x, y, **kw)
        assert (r[1] == 0).all() and torch.equal(h[1], kw["shift"][0])
        assert torch.isnan(r[2]).all() and torch.isnan(h[2]).all()
        assert torch.isinf(r[3, 0]) and torch.isnan(h[3, 0])
        keep = [0, 4, 5, 6, 7]
        assert torch.equal(r[keep], r0[keep]) and torch.equal(h[keep], h0[keep])


def test_partials_are_summed_in_order():
    """S = 3 partials whose fp32 sum depends on the order: the result is that of reduce_partials."""
    big = 2.0 ** 26
    y = torch.zeros((3, 2, 64), device="cuda")
    y[0], y[1], y[2] = big, 1.0, -big
    x = torch.zeros((2, 64), device="cuda")
    r, _ = ql.norm_residual(x, y, post_norm=False, pre_norm=False)
    assert torch.equal(r, ql.reduce_partials(y, out_dtype=torch.float32))
    r, _ = ql.norm_residual(x, y[[0, 2, 1]].contiguous(), post_norm=False, pre_norm=False)
    assert (r == 1.0).all()


def test_streams_repeats_and_graphs():
    rng = np.random.default_rng(8)
    for M, D in ((3, 520), (260, 4608)):
        x, y, kw = _make(rng, M, D, T=2)
        r, h = ql.norm_residual(x, y, **kw)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        r2, h2 = ql.norm_residual(x, y, stream=side, **kw)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(r, r2) and torch.equal(h, h2)
        out, ho = torch.empty_like(r), torch.empty_like(h)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ql.norm_residual(x, y, out=out, h=ho, **kw)
        for _ in range(2):
            out.fill_(0)
            ho.fill_(0)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, r) and torch.equal(ho, h)


@pytest.mark.parametrize("D", [64, 8192, 32768])
def test_row_offsets_beyond_32_bits(D):
    """More than 2^31 elements: the last rows' offsets do not fit 32 bits (short rows, the ring, a CTA per row)."""
    M = 2 ** 31 // D + 3
    x = torch.zeros((M, D), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(9)
    tail = torch.from_numpy(rng.standard_normal((3, D)).astype(np.float32)).cuda().bfloat16()
    x[-3:] = tail
    h = ql.norm_residual(x)[1]
    alone = ql.norm_residual(tail)[1]
    # the tail alone may take another form, whose sums run in another order
    assert torch.allclose(h[-3:].float(), alone.float(), rtol=2 * B, atol=0)
    assert (h[:8] == 0).all()


def test_refusals_of_the_binding():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    v, m = torch.ones(64, device="cuda"), torch.ones((2, 64), device="cuda")
    for kw in (dict(post_weight=v), dict(gate=m), dict(out=x), dict(pre_norm=False), dict(pre_weight=v[:32]),
               dict(scale=m), dict(scale=m[:1], shift=m, segment_ids=torch.zeros(4, dtype=torch.int32, device="cuda")),
               dict(pre_weight=v, scale=m[:1].bfloat16()), dict(segment_ids=torch.zeros(4, device="cuda")),
               dict(h=torch.empty((4, 64), device="cuda")), dict(pre_weight=v.cpu())):
        with pytest.raises(ValueError):
            ql.norm_residual(x, **kw)
    for y in (x[:2], x.half(), x[None].contiguous(), torch.zeros((64, 4), dtype=x.dtype, device="cuda").t()):
        with pytest.raises(ValueError):
            ql.norm_residual(x, y)
    for bad in (dict(x=x[:, :60].contiguous()), dict(x=x, eps=-1.0)):
        with pytest.raises(ql.QLinearError):
            ql.norm_residual(**bad)
