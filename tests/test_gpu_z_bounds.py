"""The index checks of the checked build in the kernels of few tokens, of the epilogues and of the heads.  No index is wrong:
qlinear_test_extent takes the last elements off every extent, and the accesses there are recorded and skipped."""
import ctypes

import pytest
import torch

import group_wise_affine_qlinear_b200 as ql
from group_wise_affine_qlinear_b200 import build as qb

BOUNDS = 7


def test_the_hook_is_inert_in_the_shipped_library():
    qb.build()
    assert ql.lib().qlinear_test_extent(1) == ql.lib().qlinear_test_extent(0) == 3      # QL_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def Lc():
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required for -m gpu tests")
    return ql.load_library(qb.build(bounds_check=True))


def _checked(Lc, call, y, want, last):
    """call() writes want into y; with one element off every extent it records the fact and leaves y's last elements."""
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)

    def run(cut):
        y.fill_(-77.0)
        assert Lc.qlinear_get_device_status(st) == 0
        assert Lc.qlinear_test_extent(cut) == 0
        try:
            assert call(st) == 0
            return Lc.qlinear_get_device_status(st)
        finally:
            assert Lc.qlinear_test_extent(0) == 0
    assert Lc.qlinear_test_extent(-1) == 1                                              # QL_ERR_INVALID_ARG
    assert run(0) == 0 and torch.equal(y, want)
    assert run(1) == BOUNDS and (y.reshape(-1)[-last:] == -77.0).all()
    assert run(0) == 0 and torch.equal(y, want)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,N,path", [(3, 512, 136, "few"), (20, 512, 136, "few"), (40, 1024, 136, "tc_skinny"),
                                        (100, 64, 264, "tc_fused"), (70, 4096, 136, "tc_fused")])
def test_epilogues(Lc, M, K, N, path, out, bits):
    g = torch.Generator(device="cuda").manual_seed(M + N)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    x, res, bias, gate = rand(M, K).bfloat16(), rand(M, N).to(out), rand(N), rand(2, N)
    w = (torch.randint(-2 ** 31, 2 ** 31, (N, K * bits // 32), generator=g, device="cuda", dtype=torch.int64).to(torch.int32),
         (0.01 * rand(N, K // 64)).half(), (0.01 * rand(N, K // 64)).half())
    seg = (torch.arange(M, device="cuda") * 2 // M).to(torch.int32)
    want = (ql.forward_epilogue if bits == 4 else ql.forward8_epilogue)(x, *w, bias=bias, activation="silu", gate=gate, residual=res,
                                                                        segment_ids=seg)
    assert ql.last_dispatch().startswith(f"path={path}_epilogue")
    y = torch.empty_like(want)
    ws = torch.empty(max(16, ql.epilogue_workspace_size(M, K, N, bits)), dtype=torch.uint8, device="cuda")
    fn = Lc.qlinear_epilogue_forward if bits == 4 else Lc.qlinear8_epilogue_forward
    _checked(Lc, lambda st: fn(x.data_ptr(), *[t.data_ptr() for t in w], bias.data_ptr(), ql.ACTIVATIONS["silu"], gate.data_ptr(), 0,
                               res.data_ptr(), seg.data_ptr(), 2, y.data_ptr(), 1 if out is torch.bfloat16 else 0, M, K, N, 64,
                               ws.data_ptr(), ws.numel(), st), y, want, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("adjacent", [0, 1])
@pytest.mark.parametrize("D,P", [(64, 32), (72, 32), (256, 128)])
def test_heads(Lc, D, P, adjacent, out):
    from group_wise_affine_qlinear_b200 import _heads
    M, H = 19, 5
    g = torch.Generator(device="cuda").manual_seed(D)
    x, w = torch.randn((M, H, D), generator=g, device="cuda").to(out), torch.randn(D, generator=g, device="cuda")
    pos = torch.arange(2 * M, device="cuda", dtype=torch.int32).reshape(2, M)
    rot = ql.rotary_frequencies((P // 2, P // 2))
    want = ql.qk_norm_rotary(x, None, pos, rot, q_weight=w, adjacent=adjacent)[0]
    y = torch.empty_like(want)
    _checked(Lc, lambda st: Lc.qlinear_qk_norm_rotary(_heads._entry(x, y, w), None, 1 if out is torch.bfloat16 else 0, 0, 1e-6,
                                                      pos.data_ptr(), 0, 2, rot[0].data_ptr(), rot[1].data_ptr(), P, adjacent, None,
                                                      M, D, st), y, want, 8)
