"""An infinite down projection in one half of a SwiGLU pair: it reaches that half's value alone, as in the formula, so
h is infinite with the other half's sign, not a NaN of both.  Small integers: g and u are exact, and h is silu(g) u with
one of them infinite, so every expected value is an infinity (or a NaN where it meets a zero)."""
import numpy as np
import pytest
import torch

import group_wise_affine_qlinear_b200 as ql
from group_wise_affine_qlinear_b200 import synthetic as S
from oracle import qlinear_oracle as O

from ._helpers import to_dev_bf16, to_dev_codes, to_dev_f16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required for -m gpu tests")
    ql.lib()
    yield
    assert ql.device_status() == 0


def _bits(v):
    return S.f32_to_bf16_bits(np.asarray(v, dtype=np.float32))


def _weight(rng, I, K):
    q = rng.integers(0, 16, size=(I, K))
    s = np.full((I, K // 64), 1.0 / 64, np.float16)
    return (O.pack_codes(q), s, -8 * s), (q - 8) / 64.0


@pytest.mark.parametrize("which", ["gate", "up"])
@pytest.mark.parametrize("M,r", [(30, 16), (250, 8), (250, 24), (400, 40), (200, 128)])
def test_an_infinite_down_projection_stays_in_its_half(M, r, which):
    rng = np.random.default_rng(M + r)
    K, I, n = 128, 136, 3
    x = rng.integers(1, 4, (M, K)).astype(np.float64)             # never zero: x A is infinite, not NaN
    gate, gv = _weight(rng, I, K)
    up, uv = _weight(rng, I, K)
    a = [rng.integers(-1, 2, (n, r, K)) / 64.0 for _ in range(2)]
    b = [rng.integers(1, 3, (n, I, r)).astype(np.float64) for _ in range(2)]
    ids = rng.integers(-1, n, M).astype(np.int32)
    g = x @ gv.T + O.lora_delta(_bits(x), _bits(a[0]), _bits(b[0]), None, ids)
    u = x @ uv.T + O.lora_delta(_bits(x), _bits(a[1]), _bits(b[1]), None, ids)

    def call():
        d = [to_dev_bf16(_bits(v)) for v in (a[0], b[0], a[1], b[1])]
        w = [(to_dev_codes(c), to_dev_f16(s), to_dev_f16(z)) for c, s, z in (gate, up)]
        return ql.swiglu_lora(to_dev_bf16(_bits(x)), *w, (d[0], d[1]), (d[2], d[3]), torch.from_numpy(ids).cuda(),
                              out_dtype=torch.float32).double().cpu().numpy()
    clean = call()
    hit, half = ids == 1, 0 if which == "gate" else 1
    a[half][1, r - 1, 5] = np.inf                                 # B is positive: that half is +inf in every column
    h = call()
    assert np.array_equal(h[~hit], clean[~hit])
    other = (u if which == "gate" else O.silu(g))[hit]
    assert np.all(np.isfinite(other)) and (other > 0).any() and (other < 0).any()
    with np.errstate(invalid="ignore"):
        assert np.array_equal(h[hit], np.inf * other, equal_nan=True)
