"""The norms' ring (rows of more than 512 elements, more than two per SM) on the forms that the smaller tests run
through the other kernels: padding (also longer than the ring, and at both ends of a CTA's rows), segments out of range,
the update in place, y with one norm or none.  The rows are compared with the float64 formula under the bounds of
test_gpu_z_norm, and what must not be touched with what was there."""
import numpy as np
import pytest
import torch

import group_wise_affine_qlinear_b200 as ql

from .test_gpu_z_norm import _check, _make

pytestmark = pytest.mark.gpu

# each of the ring's four shapes (threads and pieces per thread), with two to four rows in it; the longest rows with
# fp32 partials are too wide for it and take a CTA per row
SHAPES = [(400, 520), (700, 2056), (500, 4608), (450, 5128), (420, 8200), (330, 16384)]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required for -m gpu tests")
    assert min(m for m, _ in SHAPES) > 2 * torch.cuda.get_device_properties(0).multi_processor_count
    ql.lib()
    yield
    assert ql.device_status() == 0


def _segments(rng, M, how):
    seg = rng.integers(0, 2, M).astype(np.int32)
    if how == "scattered":
        seg[rng.random(M) < 0.4] = -1
    elif how == "runs":                                # runs of padding longer than the ring, one at either end
        for a in range(0, M, 29):
            seg[a:a + int(rng.integers(5, 14))] = -1 - int(rng.integers(0, 3))
        seg[-7:] = -1
    elif how == "nothing":                             # every row is padding
        seg[:] = -1
    return seg


@pytest.mark.parametrize("how", ["scattered", "runs", "nothing"])
@pytest.mark.parametrize("M,D", SHAPES)
def test_padding_rows_are_left_alone(M, D, how):
    rng = np.random.default_rng(M + D)
    x, y, kw = _make(rng, M, D, T=2, y="f32" if D == 2056 else "bf16", S=3 if D == 2056 else 1)
    seg = torch.from_numpy(_segments(rng, M, how)).cuda()
    kw["segment_ids"] = seg
    pad = seg < 0
    x[pad] = float("nan")                              # what lies there must not matter
    y[..., pad, :] = float("inf")
    out, h = torch.full_like(x, 7.0), torch.full((M, D), -3.0, dtype=torch.bfloat16, device="cuda")
    ql.norm_residual(x, y, out=out, h=h, **kw)
    assert (out[pad] == 7.0).all() and (h[pad] == -3.0).all()
    if how != "nothing":
        _check(x, y, out, h, kw)


@pytest.mark.parametrize("M,D", SHAPES)
def test_segments_out_of_range_are_recorded_and_left_alone(M, D):
    rng = np.random.default_rng(M)
    x, y, kw = _make(rng, M, D, T=2)
    seg = _segments(rng, M, "scattered")
    bad = np.flatnonzero(rng.random(M) < 0.1)
    bad = np.unique(np.concatenate((bad, [0, M - 1])))
    seg[bad] = rng.integers(2, 9, bad.size)
    kw["segment_ids"] = torch.from_numpy(seg).cuda()
    out, h = torch.full_like(x, 7.0), torch.full((M, D), -3.0, dtype=torch.bfloat16, device="cuda")
    ql.norm_residual(x, y, out=out, h=h, **kw)
    assert ql.device_status() == 1
    left = torch.from_numpy((seg < 0) | (seg >= 2)).cuda()
    assert (out[left] == 7.0).all() and (h[left] == -3.0).all()
    _check(x, y, out, h, kw, rows=np.flatnonzero((seg >= 0) & (seg < 2)))


@pytest.mark.parametrize("x32", [False, True])
@pytest.mark.parametrize("M,D", SHAPES)
def test_update_in_place(M, D, x32):
    rng = np.random.default_rng(M + 1)
    x, y, kw = _make(rng, M, D, T=2, x32=x32)
    kw["segment_ids"] = torch.from_numpy(_segments(rng, M, "scattered")).cuda()
    first = torch.zeros_like(x), torch.zeros((M, D), dtype=torch.bfloat16, device="cuda")
    ql.norm_residual(x, y, out=first[0], h=first[1], **kw)
    for _ in range(3):                                 # rows copied ahead must not be those already updated
        x2, h2 = x.clone(), torch.zeros_like(first[1])
        r, h = ql.norm_residual(x2, y, out=x2, h=h2, **kw)
        live = kw["segment_ids"] >= 0
        assert r is x2 and torch.equal(x2[live], first[0][live]) and torch.equal(x2[~live], x[~live])
        assert torch.equal(h2, first[1])


@pytest.mark.parametrize("y,S", [("bf16", 1), ("f32", 2)])
@pytest.mark.parametrize("M,D", SHAPES)
def test_one_norm_or_none(M, D, y, S):
    rng = np.random.default_rng(M + 2)
    x, yt, full = _make(rng, M, D, T=2, y=y, S=S)
    pick = lambda *names, **more: {**{k: full[k] for k in names}, **more}
    for kw in (pick("post_weight", "gate", "segment_ids", pre_norm=False),
               pick("gate", "pre_weight", "scale", "shift", "segment_ids", post_norm=False),
               pick("gate", "segment_ids", post_norm=False, pre_norm=False), pick(post_norm=False, pre_norm=False)):
        r, h = ql.norm_residual(x, yt, **kw)
        assert (h is None) == (not kw.get("pre_norm", True))
        _check(x, yt, r, h, kw)
    r, h = ql.norm_residual(x, **pick("pre_weight", "scale", "shift", "segment_ids"))
    assert r is x
    _check(x, None, r, h, pick("pre_weight", "scale", "shift", "segment_ids"))
