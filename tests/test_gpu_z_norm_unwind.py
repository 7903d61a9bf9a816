"""The norms' ring of rows (many rows of more than 512 elements) through the checked build with its copies held back
(qlinear_test_stall): the waits must expire within the shortened limit, the call must report it, store nothing and
start no further copy, and the next calls must run normally."""
import ctypes
import time

import pytest
import torch

import group_wise_affine_qlinear_b200 as ql

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Lc():
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required for -m gpu tests")
    from group_wise_affine_qlinear_b200 import build as qb
    return ql.load_library(qb.build(bounds_check=True))


@pytest.mark.parametrize("M,D,S", [(700, 4608, 0), (1500, 520, 2), (400, 16384, 0)])
def test_ring_unwinds_when_its_copies_are_held_back(Lc, M, D, S):
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn((M, D), generator=g, device="cuda").bfloat16()
    y = torch.randn((S, M, D), generator=g, device="cuda") if S else \
        torch.randn((M, D), generator=g, device="cuda").bfloat16()
    seg = (torch.arange(M, device="cuda") % 3 - 1).to(torch.int32)          # every third row is padding
    scale = torch.randn((2, D), generator=g, device="cuda")
    want = ql.norm_residual(x, y, scale=scale, segment_ids=seg)
    out, h = torch.empty_like(x), torch.empty((M, D), dtype=torch.bfloat16, device="cuda")
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)

    def call():
        out.fill_(7.0)
        h.fill_(-3.0)
        return Lc.qlinear_norm_residual(x.data_ptr(), 1, y.data_ptr(), 0 if S else 1, max(S, 1), 1, None, None, 1.0, 1.0,
                                        None, scale.data_ptr(), None, 0, seg.data_ptr(), 2, 1e-6, out.data_ptr(),
                                        h.data_ptr(), M, D, st)

    assert Lc.qlinear_get_device_status(st) == 0
    assert Lc.qlinear_test_stall(4, 20_000_000) == 0
    try:
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        assert call() == 0
        status = Lc.qlinear_get_device_status(st)
        elapsed = time.perf_counter() - t0
    finally:
        assert Lc.qlinear_test_stall(0, 1_000_000_000) == 0
    assert status == 6, status                                # QL_ERR_DEVICE_TIMEOUT
    assert elapsed < 0.9, elapsed                             # the shortened limit, not the default second
    assert (out == 7.0).all() and (h == -3.0).all()
    live = seg >= 0
    for _ in range(2):                                        # the next calls run normally
        assert call() == 0
        assert Lc.qlinear_get_device_status(st) == 0
        assert torch.equal(out[live], want[0][live]) and torch.equal(h[live], want[1][live])
        assert (out[~live] == 7.0).all() and (h[~live] == -3.0).all()
