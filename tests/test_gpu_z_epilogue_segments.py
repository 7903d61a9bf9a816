"""Without a gate, segment ids tell padding rows from the others and nothing else: the bits of a call are those of one
without ids, whatever the order of the segments."""
import numpy as np
import pytest
import torch

import group_wise_affine_qlinear_b200 as ql
from tests._helpers import random_layer, to_dev_bf16, to_dev_codes, to_dev_f16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required for -m gpu tests")
    ql.lib()
    yield
    assert ql.device_status() == 0


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,N", [(6, 128, 136), (50, 128, 136), (300, 128, 520), (90, 4096, 136)])
@pytest.mark.parametrize("residual", [False, True])
def test_bits_do_not_depend_on_the_segments(M, K, N, out, residual):
    rng = np.random.default_rng(M + K)
    xb, codes, s, b = random_layer(rng, M, K, N)
    w = to_dev_codes(codes), to_dev_f16(s), to_dev_f16(b)
    # far below, so that half of the outputs of silu are zeros, negative ones
    bias = torch.from_numpy(np.where(rng.random(N) < 0.5, -1e4, 0.0).astype(np.float32)).cuda()
    kw = dict(bias=bias, activation="silu", out_dtype=out)
    if residual:
        kw["residual"] = torch.from_numpy(rng.standard_normal((M, N)).astype(np.float32)).cuda().to(out)
    x = to_dev_bf16(xb)
    want = ql.forward_epilogue(x, *w, **kw)
    for ids in (rng.integers(0, 9, M), np.sort(rng.integers(0, 3, M)), np.full(M, 2 ** 31 - 2), rng.permutation(M)):
        pad = rng.random(M) < 0.1
        ids = np.where(pad, -1 - ids % 3, ids).astype(np.int32)
        got = torch.full((M, N), 7.0, dtype=out, device="cuda")
        ql.forward_epilogue(x, *w, segment_ids=torch.from_numpy(ids).cuda(), out=got, **kw)
        live = torch.from_numpy(~pad).cuda()
        assert torch.equal(got[live].view(torch.uint8), want[live].view(torch.uint8))
        assert (got[~live] == 7.0).all()
