"""Few tokens with an epilogue, to the last bit, with a scale and a bias of its own for every row and group.

Everything is a whole number of quarters: scales of 1 to 15 of them (8-bit codes: 1 to 7), biases up to 1800 (200), so that
a weight takes up to 11 bits: exact in f16, which the other paths multiply, and not in bf16, whatever a kernel makes of the
codes; activations of -2 to 2.  Any order of the sums is exact as long as a group's offset sums and the sums over the groups
stay below 2^24 quarters, which is asserted."""
import numpy as np
import pytest
import torch

import group_wise_affine_qlinear_b200 as ql
from oracle import qlinear_oracle as O
from tests._helpers import to_dev_codes, to_dev_f16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required for -m gpu tests")
    ql.lib()
    yield
    assert ql.device_status() == 0


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M", [1, 8, 13, 32, 40, 100])
@pytest.mark.parametrize("K,N", [(64, 136), (448, 24), (576, 8), (1024, 40), (2048, 72), (4672, 264)])
def test_every_group_has_its_own_scale_and_bias(M, K, N, bits):
    rng = np.random.default_rng(M + K + N + bits)
    G = K // 64
    codes = rng.integers(0, 1 << 32, size=(N, K * bits // 32), dtype=np.uint32)
    q = (O.unpack_codes(codes, K) if bits == 4 else O.unpack_codes8(codes, K)).reshape(N, G, 64).astype(np.float64)
    s, b = rng.integers(1, 16 if bits == 4 else 8, (N, G)), rng.integers(-1, 2, (N, G)) * rng.integers(0, 1801 if bits == 4 else 201, (N, G))
    x = rng.integers(-2, 3, (M, G, 64)).astype(np.float64)
    w = s[..., None] * q + b[..., None]
    assert np.abs(w).max() < 2048                          # 11 bits
    off = 128 if bits == 4 else 17 * 128
    shifted, plain = np.einsum("mgk,ngk->mng", x, off + q), x.sum(-1)[:, None, :]
    ahead = np.abs(s * shifted) + np.abs((b - off * s) * plain)
    lin = np.cumsum(np.einsum("mgk,ngk->mng", x, w), -1)
    assert (ahead + np.abs(lin)).max() < 2 ** 24
    dev = lambda v: to_dev_f16((v / 4).astype(np.float16))
    bias = rng.integers(-64, 65, N)
    call = ql.forward_epilogue if bits == 4 else ql.forward8_epilogue
    got = call(torch.from_numpy(x.reshape(M, K).astype(np.float32)).cuda().bfloat16(), to_dev_codes(codes), dev(s), dev(b),
               bias=torch.from_numpy((bias / 4).astype(np.float32)).cuda(), out_dtype=torch.float32)
    assert ql.last_dispatch().startswith("path=few_epilogue") == (M <= 32)
    assert np.array_equal(got.double().cpu().numpy(), (lin[..., -1] + bias) / 4)
