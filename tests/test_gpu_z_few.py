"""Projections of up to 32 tokens with an epilogue, in one launch, and the rule that picks it.

Integer layers are exact (whole quarters below 2^24).  Random ones: a group's sum of (128 + q) x or, for 8-bit codes, of
its nibbles' takes 64 products, each addition off by 2 u = 2^-23 at most of sums up to 143 (2288) sum |x|; with the
products by s and b - 128 s (b - 2176 s) and their sum the group errs by 2^-22 (64 + 4) 2^8 (2^12) s sum |x| at the very
most, far above what rounding to nearest makes of it; behind it G fp32 additions.
"""
import numpy as np
import pytest
import torch

import group_wise_affine_qlinear_b200 as ql
from oracle import qlinear_oracle as O
from tests._helpers import random_layer, random_layer8, to_dev_bf16, to_dev_codes, to_dev_f16
from tests.test_gpu_z_epilogue import DT, _check_exact, _exact_case, _f64

pytestmark = pytest.mark.gpu

CALL = {4: ql.forward_epilogue, 8: ql.forward8_epilogue}
U, B = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required for -m gpu tests")
    ql.lib()
    yield
    assert ql.device_status() == 0


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 24, 25, 32])
@pytest.mark.parametrize("K,N", [(64, 8), (64, 136), (448, 24), (512, 1032), (576, 8), (960, 264), (1024, 40), (2048, 72),
                                 (4672, 520)])
def test_exact_integers(M, K, N, bits):
    """One to eight slices of K, whole and partial, rows past N in the last CTA, in place."""
    rng = np.random.default_rng(M * 100 + K + N + bits)
    out, params = ("bf16", "f32") if (M + K // 64) % 2 else ("f32", "bf16")
    x, w, kw, seg, lin = _exact_case(rng, M, K, N, bits, out, params)
    y = O.epilogue_ref(lin, _f64(kw["bias"]), None, _f64(kw["gate"]), _f64(kw["residual"]), seg)
    ids = torch.from_numpy(seg).cuda()
    before = kw["residual"].clone()
    CALL[bits](x, *w, segment_ids=ids, out=kw["residual"], **kw)
    few = K * N * bits // 8 <= (32 if M <= 8 else (16 if M <= 16 else 4) * 4 // bits) << 20
    assert ql.last_dispatch().startswith("path=few_epilogue" if few else "path=tc_skinny_epilogue")
    _check_exact(kw["residual"], y, seg, out, before)


@pytest.mark.parametrize("act", [None, "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M,K,N,bits", [(1, 4608, 264, 4), (8, 512, 1032, 8), (5, 2176, 72, 4), (3, 128, 520, 8),
                                         (13, 1088, 264, 8), (30, 576, 264, 4)])
def test_random_layers(M, K, N, bits, act):
    rng = np.random.default_rng(M + K + N)
    xb, codes, s, b = (random_layer if bits == 4 else random_layer8)(rng, M, K, N)
    xv, w64 = O.decode_bf16(xb), (O.dequant_exact if bits == 4 else O.dequant8_exact)(codes, s, b)
    sx = np.abs(xv).reshape(M, K // 64, 64).sum(-1) @ np.abs(s.astype(np.float64)).T           # sum over groups of s sum |x|
    ez = 2.0 ** -22 * 68 * (2.0 ** 8 if bits == 4 else 2.0 ** 12) * sx + (K / 64) * 2 * U * (np.abs(xv) @ np.abs(w64).T)
    bias = rng.standard_normal(N).astype(np.float32)
    z = xv @ w64.T + bias
    y = O.activation(z, act)
    got = _f64(CALL[bits](to_dev_bf16(xb), to_dev_codes(codes), to_dev_f16(s), to_dev_f16(b), bias=torch.from_numpy(bias).cuda(),
                          activation=act, out_dtype=torch.float32))
    bound = (1.13 if act else 1.0) * (ez + 4 * U * np.abs(z)) + 2.0 ** -20 * np.abs(z)
    assert np.all(np.abs(got - y) <= bound), float((np.abs(got - y) / bound).max())


def test_one_token_does_not_reach_another():
    rng = np.random.default_rng(1)
    for M in (8, 27):
        x, w, kw, seg, lin = _exact_case(rng, M, 512, 136, 4, "bf16", "bf16", padding=False)
        ids = torch.from_numpy(seg).cuda()
        clean = ql.forward_epilogue(x, *w, segment_ids=ids, **kw)
        x[2, 100], x[5, 7] = float("inf"), float("nan")
        kw["residual"][6, 3] = float("nan")
        got = ql.forward_epilogue(x, *w, segment_ids=ids, **kw)
        assert not torch.isfinite(got[2]).any() and torch.isnan(got[5]).all() and torch.isnan(got[6, 3])
        for m in set(range(M)) - {2, 5, 6}:
            assert torch.equal(got[m], clean[m])
        assert torch.equal(got[6, 4:], clean[6, 4:])


def test_magnitudes():
    """Activations from 2^-120 to 2^110 of one row: powers of two scale the sums exactly."""
    rng = np.random.default_rng(2)
    x, w, kw, seg, lin = _exact_case(rng, 4, 256, 72, 4, "f32", "f32")
    scale = 2.0 ** np.array([-118, -20, 60, 109])
    got = _f64(ql.forward_epilogue((x.double() * torch.from_numpy(scale).cuda()[:, None]).bfloat16(), *w,
                                   out_dtype=torch.float32))
    assert np.array_equal(got, lin * scale[:, None])


def test_the_rule():
    """Few tokens of a small weight; more tokens or larger weights are streamed."""
    def path(M, K, N, bits):
        c = torch.zeros((N, K * bits // 32), dtype=torch.int32, device="cuda")
        s = torch.zeros((N, K // 64), dtype=torch.float16, device="cuda")
        CALL[bits](torch.zeros((M, K), dtype=torch.bfloat16, device="cuda"), c, s, s)
        return ql.last_dispatch().split()[0]
    assert path(8, 8192, 8192, 4) == "path=few_epilogue" and path(8, 8192, 8200, 4) == "path=tc_skinny_epilogue"
    assert path(8, 8192, 4096, 8) == "path=few_epilogue" and path(8, 8192, 4104, 8) == "path=tc_skinny_epilogue"
    assert path(16, 8192, 4096, 4) == "path=few_epilogue" and path(16, 8192, 4104, 4) == "path=tc_skinny_epilogue"
    assert path(16, 2048, 4096, 8) == "path=few_epilogue" and path(16, 2048, 4104, 8) == "path=tc_skinny_epilogue"
    assert path(32, 2048, 4096, 4) == "path=few_epilogue" and path(17, 2048, 4104, 4) == "path=tc_skinny_epilogue"
    assert path(32, 2048, 1024, 8) == "path=few_epilogue" and path(17, 2048, 1032, 8) == "path=tc_skinny_epilogue"
    assert path(33, 64, 8, 4) == "path=tc_skinny_epilogue" and path(65, 64, 8, 4) == "path=tc_fused_epilogue"


def test_replays_with_other_values():
    rng = np.random.default_rng(3)
    x, w, kw, seg, lin = _exact_case(rng, 3, 512, 264, 8, "bf16", "f32", padding=False)
    ids = torch.from_numpy(seg).cuda()
    out = torch.empty((3, 264), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            ql.forward8_epilogue(x, *w, segment_ids=ids, out=out, **kw)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        x.copy_(torch.from_numpy(rng.integers(-2, 3, (3, 512)).astype(np.float32)).cuda())
        graph.replay()
        assert torch.equal(out, ql.forward8_epilogue(x, *w, segment_ids=ids, **kw))
