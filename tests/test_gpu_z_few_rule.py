"""Which path a few tokens with an epilogue take: wide weights near the one-launch kernel's limit are streamed (measured
12 to 36 % faster), and a call without that path's workspace is one launch as before."""
import ctypes

import numpy as np
import pytest
import torch

import group_wise_affine_qlinear_b200 as ql
from group_wise_affine_qlinear_b200 import build as qb
from tests._helpers import to_dev_codes, to_dev_f16

STREAMED = [(1, 4608, 13824), (8, 4608, 13824), (8, 4608, 12288), (4, 2304, 24576), (8, 4608, 10240), (16, 5120, 5120),
            (9, 4096, 8192), (32, 512, 16384), (17, 1024, 6656)]
ONE_LAUNCH = [(1, 4608, 4608), (8, 4608, 9216), (8, 12288, 4608), (16, 4608, 4608), (16, 2304, 9216), (32, 2048, 4096), (8, 512, 32768)]


def test_workspace_sizes():
    qb.build()
    L = ql.lib()
    for M, K, N in STREAMED:
        assert L.qlinear_epilogue_workspace_size(M, K, N, 64) == L.qlinear_workspace_size(M, K, N, 64) > 0, (M, K, N)
    for M, K, N in ONE_LAUNCH:
        assert L.qlinear_epilogue_workspace_size(M, K, N, 64) == 0, (M, K, N)
    for M, K, N in ((8, 2304, 11520), (8, 4608, 6912), (16, 1024, 8192), (32, 512, 4096)):
        assert L.qlinear8_epilogue_workspace_size(M, K, N, 64) == 0, (M, K, N)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N,path", [(*c, "tc_skinny") for c in STREAMED] + [(*c, "few") for c in ONE_LAUNCH])
def test_paths(M, K, N, path):
    """Integer layers, so that both paths give the same bytes."""
    rng = np.random.default_rng(M + K + N)
    codes = to_dev_codes(rng.integers(0, 1 << 32, size=(N, K // 8), dtype=np.uint32))
    s, b = (to_dev_f16(np.full((N, K // 64), v, np.float16)) for v in (1.0, -8.0))
    x = torch.from_numpy(rng.integers(-2, 3, (M, K)).astype(np.float32)).cuda().bfloat16()
    bias = torch.from_numpy((rng.integers(-8, 9, N) / 4).astype(np.float32)).cuda()
    got = ql.forward_epilogue(x, codes, s, b, bias=bias, out_dtype=torch.float32)
    assert ql.last_dispatch().startswith(f"path={path}_epilogue")
    # without a workspace, through the C entry
    y = torch.full_like(got, float("nan"))
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert ql.lib().qlinear_epilogue_forward(x.data_ptr(), codes.data_ptr(), s.data_ptr(), b.data_ptr(), bias.data_ptr(), 0,
                                             None, 0, None, None, 1, y.data_ptr(), 0, M, K, N, 64, None, 0, st) == 0
    assert ql.last_dispatch().startswith("path=few_epilogue")
    shifts = torch.arange(8, device="cuda", dtype=torch.int32) * 4
    w = (((codes[:, :, None] >> shifts) & 15) - 8).reshape(N, K).double()
    want = x.double() @ w.T + bias.double()
    assert torch.equal(got.double(), want) and torch.equal(y, got)
    assert ql.device_status() == 0
