"""The adapters' first product (more than 64 rows) through the checked build with its copies held back
(qlinear_test_stall): every wait must expire within the shortened limit, also in tiles that meet several adapters one
after the other and in clusters that share a tile's columns, the call must report it, and the next calls must give the
shipped library's bytes."""
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


# a cluster of CTAs per tile and an adapter per CTA; one CTA per tile with all twelve adapters; two blocks of ranks
@pytest.mark.parametrize("M,K,n,r", [(200, 4096, 3, 16), (5000, 256, 12, 8), (700, 1024, 4, 72)])
def test_first_product_unwinds_when_its_copies_are_held_back(Lc, M, K, n, r):
    N = 264
    g = torch.Generator(device="cuda").manual_seed(M)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    x = rand(M, K).bfloat16()
    codes = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    s, b = (0.01 * rand(N, K // 64)).half(), (0.01 * rand(N, K // 64)).half()
    la, lb = (rand(n, r, K) / 64).bfloat16(), (0.05 * rand(n, N, r)).bfloat16()
    ids = torch.randint(-1, n, (M,), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    want = ql.forward_lora(x, codes, s, b, la, lb, ids)
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(Lc.qlinear_lora_workspace_size(M, K, N, 64, n, r), dtype=torch.uint8, device="cuda")
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)

    def call():
        y.fill_(float("nan"))
        return Lc.qlinear_lora_forward(x.data_ptr(), codes.data_ptr(), s.data_ptr(), b.data_ptr(), la.data_ptr(),
                                       lb.data_ptr(), None, ids.data_ptr(), y.data_ptr(), 1, M, K, N, 64, n, r,
                                       ws.data_ptr(), ws.numel(), st)

    assert Lc.qlinear_get_device_status(st) == 0
    assert Lc.qlinear_test_stall(8, 20_000_000) == 0
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
    for _ in range(2):                                        # the next calls run normally
        assert call() == 0
        assert Lc.qlinear_get_device_status(st) == 0
        assert torch.equal(y, want)
