"""The activations' relative accuracy, far in their tails too, on each path of a projection with an epilogue.

The activations are zero, so that the argument z is the bias.  Bounds, with u = 2^-24 (half an fp32 unit): the hardware's
exponential errs by 4 u relative, its reciprocal by 2 u, and rounding the exponential's argument by its magnitude times
  silu       1.5 u (the constant and one product): 4 u + 1.5 |z| u, then three roundings and the reciprocal: (9 + 1.5 |z|) u
  gelu_tanh  7 u (two constants, a square, two products): (9 + 7 E) u, E = 2 sqrt(2 / pi) |z + 0.044715 z^3|
  gelu       of the tail 1 - Phi(|z|): the fit 4 u (1 + z^2 / 2), its evaluation in fp32 4 u and t's error 6 u (a slope of 2.3
             at most), the exponential 4 u and its argument 1.5 z^2 u, two products 2 u: (20 + 4 z^2) u; and u of the result
of the value, beside what is under 2^-120."""
import math

import numpy as np
import pytest
import torch

import group_wise_affine_qlinear_b200 as ql

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
RANGE = {"silu": 80.0, "gelu": 12.5, "gelu_tanh": 8.5}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required for -m gpu tests")
    ql.lib()
    yield
    assert ql.device_status() == 0


def _definition(z, act):
    """(value, bound of its error) in float64, without cancellation in the tails."""
    a = np.abs(z)
    if act == "gelu":
        upper = np.vectorize(lambda v: 0.5 * math.erfc(v / math.sqrt(2.0)))(a)          # 1 - Phi(|z|)
        y = np.where(z < 0, z * upper, z - z * upper)
        return y, (20 + 4 * z * z) * U * a * upper + U * np.abs(y)
    e = a if act == "silu" else 2.0 * math.sqrt(2.0 / math.pi) * (a + 0.044715 * a ** 3)
    y = z * np.where(z < 0, np.exp(-e), 1.0) / (1.0 + np.exp(-e))
    return y, (9 + (1.5 if act == "silu" else 7.0) * e) * U * np.abs(y)


@pytest.mark.parametrize("M,K,path", [(3, 64, "few_epilogue"), (20, 64, "few_epilogue"), (40, 64, "tc_skinny_epilogue"),
                                      (100, 64, "tc_fused_epilogue"), (70, 4096, "tc_fused_epilogue")])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_relative_error(act, M, K, path):
    N = 2048
    z = np.linspace(-RANGE[act], RANGE[act], N).astype(np.float32)
    codes = torch.zeros((N, K // 8), dtype=torch.int32, device="cuda")
    s = torch.ones((N, K // 64), dtype=torch.float16, device="cuda")
    got = ql.forward_epilogue(torch.zeros((M, K), dtype=torch.bfloat16, device="cuda"), codes, s, s,
                              bias=torch.from_numpy(z).cuda(), activation=act, out_dtype=torch.float32)
    assert ql.last_dispatch().split()[0] == "path=" + path
    assert torch.equal(got, got[:1].expand_as(got))
    y, bound = _definition(z.astype(np.float64), act)
    err = np.abs(got[0].double().cpu().numpy() - y)
    bound = bound + 2.0 ** -120
    assert np.all(err <= bound), (float((err / bound).max()), float(z[np.argmax(err / bound)]))
