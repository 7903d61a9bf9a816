"""The gate/up pair with adapters and the norms' ring through the checked build: outputs must not depend on the timing
of the pipelines' roles (qlinear_test_delay).  The pair by the weight-streaming kernel over several tile segments and by
the fused kernel with several tiles per CTA, behind the adapters' first product with one and with many CTAs per tile;
the ring with a few and with many rows per CTA, padding and in place."""
import ctypes

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


def _shaken(Lc, call, outputs, want):
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)

    def same():
        for o in outputs:
            o.fill_(float("nan"))
        assert call(st) == 0 and Lc.qlinear_get_device_status(st) == 0
        return [torch.equal(o.view(torch.uint8), w.view(torch.uint8)) for o, w in zip(outputs, want)]
    assert Lc.qlinear_test_delay(0, 0) == 0
    assert all(same())
    try:
        for role in ROLES:
            assert Lc.qlinear_test_delay(role, 20_000) == 0        # up to 20 us per role
            for _ in range(2):
                assert all(same()), role
    finally:
        assert Lc.qlinear_test_delay(0, 0) == 0


@pytest.mark.parametrize("M,K,I,n,r", [
    (24, 8192, 2056, 7, 16),        # streaming, 34 tiles of both weights on 148 CTAs
    (64, 512, 12296, 64, 8),        # streaming, several tiles per CTA, an adapter per row
    (300, 1024, 10248, 9, 24),      # fused, 162 tiles; a cluster of CTAs per tile of rows
    (1500, 512, 2056, 5, 72),       # fused, 136 tiles; two blocks of ranks, all adapters one after the other
])
def test_pair_does_not_depend_on_role_timing(Lc, M, K, I, n, r):
    g = torch.Generator(device="cuda").manual_seed(M)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    x = rand(M, K).bfloat16()

    def weight():
        c = torch.randint(-2 ** 31, 2 ** 31, (I, K // 8), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
        return c, (0.01 * rand(I, K // 64)).half(), (0.01 * rand(I, K // 64)).half()
    w = [weight(), weight()]
    ad = [((rand(n, r, K) / K ** 0.5).bfloat16(), (0.1 * rand(n, I, r)).bfloat16()) for _ in range(2)]
    ids = torch.randint(-1, n, (M,), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    scale = 0.5 + torch.rand(n, generator=g, device="cuda")
    want = ql.swiglu_lora(x, *w, *ad, ids, scale)
    h = torch.empty_like(want)
    ws = torch.empty(Lc.qlinear_swiglu_lora_workspace_size(M, K, I, 64, n, r), dtype=torch.uint8, device="cuda")
    tensors = [x, *w[0], *w[1], *ad[0], *ad[1], scale, ids, h]

    def call(st):
        ws.fill_(0xFF)
        return Lc.qlinear_swiglu_lora_forward(*[t.data_ptr() for t in tensors], 1, M, K, I, 64, n, r, ws.data_ptr(),
                                              ws.numel(), st)
    _shaken(Lc, call, [h], [want])


@pytest.mark.parametrize("M,D,S", [(320, 4608, 0), (5000, 1544, 0), (900, 2056, 3), (700, 12288, 0)])
def test_ring_does_not_depend_on_role_timing(Lc, M, D, S):
    g = torch.Generator(device="cuda").manual_seed(D)
    x = torch.randn((M, D), generator=g, device="cuda").bfloat16()
    y = torch.randn((S, M, D), generator=g, device="cuda") if S else \
        torch.randn((M, D), generator=g, device="cuda").bfloat16()
    seg = torch.randint(0, 3, (M,), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    shift = torch.randn((3, D), generator=g, device="cuda").bfloat16()
    want = ql.norm_residual(x, y, shift=shift, segment_ids=seg)
    out, h = torch.empty_like(x), torch.empty_like(x)

    def call(st):
        out.copy_(x)                                        # the update in place
        return Lc.qlinear_norm_residual(out.data_ptr(), 1, y.data_ptr(), 0 if S else 1, max(S, 1), 1, None, None, 1.0, 1.0,
                                        None, None, shift.data_ptr(), 1, seg.data_ptr(), 3, 1e-6, out.data_ptr(),
                                        h.data_ptr(), M, D, st)
    _shaken(Lc, call, [out, h], want)
