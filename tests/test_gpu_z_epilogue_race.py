"""The fused kernel's epilogue mode through the checked build: outputs must not depend on the timing of the pipeline's
roles (qlinear_test_delay), and a held-back code producer must end in QL_ERR_DEVICE_TIMEOUT with the next calls right
(qlinear_test_stall: no copy of codes or MMA is ever in flight)."""
import ctypes
import time

import pytest
import torch

import group_wise_affine_qlinear_b200 as ql

pytestmark = pytest.mark.gpu

ROLES = [1, 2, 4, 8, 16, 31]          # activations, codes, dequantizers, MMA, epilogue, all of them


@pytest.fixture(scope="module")
def Lc():
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required for -m gpu tests")
    from group_wise_affine_qlinear_b200 import build as qb
    return ql.load_library(qb.build(bounds_check=True))


def _case(M, K, N, act, out, seed, mixed=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    x, dt = rand(M, K).bfloat16(), torch.bfloat16 if out == "bf16" else torch.float32
    w = (torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), generator=g, device="cuda", dtype=torch.int64).to(torch.int32),
         (0.01 * rand(N, K // 64)).half(), (0.01 * rand(N, K // 64)).half())
    bias, gate, res = rand(N), rand(3, N), rand(M, N).to(dt)
    seg = torch.randint(-1 if mixed else 0, 3, (M,), generator=g, device="cuda", dtype=torch.int64)
    seg = (seg if mixed else seg.sort().values).to(torch.int32)
    want = ql.forward_epilogue(x, *w, bias=bias, activation=act, gate=gate, residual=res, segment_ids=seg, out=res.clone())
    return x, w, bias, gate, res, seg, want


def _call(Lc, st, x, w, bias, act, gate, seg, y, ws):
    """The update in place."""
    M, K = x.shape
    N = w[0].shape[0]
    return Lc.qlinear_epilogue_forward(x.data_ptr(), *[t.data_ptr() for t in w], bias.data_ptr(), ql.ACTIVATIONS[act],
                                       gate.data_ptr(), 0, y.data_ptr(), seg.data_ptr(), 3, y.data_ptr(),
                                       1 if y.dtype == torch.bfloat16 else 0, M, K, N, 64, ws.data_ptr(), ws.numel(), st)


@pytest.mark.parametrize("M,K,N,act,out,mixed", [
    (2000, 512, 8200, None, "bf16", False),        # 363 tiles: three per CTA
    (1500, 1024, 6152, "silu", "bf16", True),      # padding and segments in every chunk
    (1500, 512, 6152, "gelu", "f32", True),
    (200, 4096, 520, "gelu_tanh", "bf16", True),   # its K-steps split
    (40, 2048, 2056, "silu", "bf16", True),        # streaming
])
def test_outputs_do_not_depend_on_role_timing(Lc, M, K, N, act, out, mixed):
    x, w, bias, gate, res, seg, want = _case(M, K, N, act, out, M + N, mixed)
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    ws = torch.empty(Lc.qlinear_epilogue_workspace_size(M, K, N, 64), dtype=torch.uint8, device="cuda")
    y = torch.empty_like(res)

    def same():
        y.copy_(res)
        ws.fill_(0xFF)
        assert _call(Lc, st, x, w, bias, act, gate, seg, y, ws) == 0 and Lc.qlinear_get_device_status(st) == 0
        return torch.equal(y.view(torch.uint8), want.view(torch.uint8))
    assert Lc.qlinear_test_delay(0, 0) == 0
    assert same()
    try:
        for role in ROLES:
            assert Lc.qlinear_test_delay(role, 20_000) == 0        # up to 20 us per role
            for _ in range(2):
                assert same(), role
    finally:
        assert Lc.qlinear_test_delay(0, 0) == 0


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_unwinds_when_the_code_producer_is_held_back(Lc, out):
    M, K, N = 900, 512, 8200
    x, w, bias, gate, res, seg, want = _case(M, K, N, "silu", out, 1)
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    ws = torch.empty(Lc.qlinear_epilogue_workspace_size(M, K, N, 64), dtype=torch.uint8, device="cuda")
    y = res.clone()
    assert Lc.qlinear_get_device_status(st) == 0
    assert Lc.qlinear_test_stall(1, 20_000_000) == 0               # 20 ms
    try:
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        assert _call(Lc, st, x, w, bias, "silu", gate, seg, y, ws) == 0
        status = Lc.qlinear_get_device_status(st)
        elapsed = time.perf_counter() - t0
    finally:
        assert Lc.qlinear_test_stall(0, 1_000_000_000) == 0
    assert status == 6 and elapsed < 0.9, (status, elapsed)
    assert torch.equal(y, res)                                     # nothing was stored
    for _ in range(2):
        y.copy_(res)
        assert _call(Lc, st, x, w, bias, "silu", gate, seg, y, ws) == 0 and Lc.qlinear_get_device_status(st) == 0
        assert torch.equal(y.view(torch.uint8), want.view(torch.uint8))
