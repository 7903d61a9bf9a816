"""Adapters through the checked build: outputs must not depend on the timing of the pipelines' roles
(qlinear_test_delay), and a call whose code producer is held back must report the expired wait and leave the next
calls right (qlinear_test_stall).  Shapes reach several tiles per CTA, tiles with one and with many adapters, split-K
slices that share the extra K-steps, and the weight-streaming kernel over two tile segments."""
import ctypes
import time

import numpy as np
import pytest
import torch

import group_wise_affine_qlinear_b200 as ql
from oracle import qlinear_oracle as O

from ._helpers import FUSED_TILE_TOKENS, bf16_bits, random_layer, sample_rows, to_dev_bf16, to_dev_codes, to_dev_f16
from group_wise_affine_qlinear_b200 import synthetic as S

pytestmark = pytest.mark.gpu

ROLES = [1, 2, 4, 8, 16, 31]          # activations, codes, dequantizers, MMA, epilogue, all of them


@pytest.fixture(scope="module")
def Lc():
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required for -m gpu tests")
    from group_wise_affine_qlinear_b200 import build as qb
    return ql.load_library(qb.build(bounds_check=True))


class _Case:
    def __init__(self, Lc, M, K, N, n, r, mixed):
        rng = np.random.default_rng(M + K)
        bits = lambda v: S.f32_to_bf16_bits(v.astype(np.float32))
        self.Lc, self.M, self.N = Lc, M, N
        self.x, self.codes, self.s, self.b = random_layer(rng, M, K, N)
        self.a = bits(rng.standard_normal((n, r, K)) / np.sqrt(K))
        self.up = bits(0.05 * rng.standard_normal((n, N, r)))
        self.scale = rng.uniform(0.5, 2.0, n).astype(np.float32)
        cuts = np.sort(rng.integers(0, M + 1, n))
        self.ids = (rng.integers(-1, n, M) if mixed else np.searchsorted(cuts, np.arange(M), side="right") - 1).astype(np.int32)
        self.dev = [to_dev_bf16(self.x), to_dev_codes(self.codes), to_dev_f16(self.s), to_dev_f16(self.b),
                    to_dev_bf16(self.a), to_dev_bf16(self.up), torch.from_numpy(self.scale).cuda(),
                    torch.from_numpy(self.ids).cuda()]
        self.y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        self.ws = torch.empty(Lc.qlinear_lora_workspace_size(M, K, N, 64, n, r), dtype=torch.uint8, device="cuda")
        self.tail = (1, M, K, N, 64, n, r, self.ws.data_ptr(), self.ws.numel())
        self.st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)

    def launch(self):
        self.y.fill_(float("nan"))
        return self.Lc.qlinear_lora_forward(*[t.data_ptr() for t in self.dev], self.y.data_ptr(), *self.tail, self.st)

    def status(self):
        return self.Lc.qlinear_get_device_status(self.st)

    def run(self):
        assert self.launch() == 0 and self.status() == 0
        return bf16_bits(self.y)

    def check(self, got):
        rows = sample_rows(self.M, n_random=16, seed=self.M, tile=FUSED_TILE_TOKENS)
        ref = O.forward_rows(self.x, self.codes, self.s, self.b, rows) + \
            O.lora_delta(self.x[rows], self.a, self.up, self.scale, self.ids[rows])
        t = O.tolerance(O.decode_bf16(got[rows]), ref)
        assert t["ok"], t


@pytest.mark.parametrize("M,K,N,n,r,mixed", [
    (1152, 1024, 9216, 5, 24, False),     # 216 tiles on 148 CTAs, one to three adapters in a tile
    (400, 512, 9216, 12, 16, True),       # twelve adapters in every tile: six extra K-steps
    (200, 8192, 1032, 6, 40, True),       # split-K: the slices share the extra K-steps
    (24, 16384, 4608, 7, 16, True),       # stream-K runs over two tile segments
])
def test_outputs_do_not_depend_on_role_timing(Lc, M, K, N, n, r, mixed):
    c = _Case(Lc, M, K, N, n, r, mixed)
    assert Lc.qlinear_test_delay(0, 0) == 0
    ref = c.run()
    c.check(ref)
    try:
        for role in ROLES:
            assert Lc.qlinear_test_delay(role, 20_000) == 0        # up to 20 us per role
            for _ in range(2):
                diff = np.flatnonzero(c.run() != ref)
                assert diff.size == 0, (role, diff.size, diff[:8])
    finally:
        assert Lc.qlinear_test_delay(0, 0) == 0


@pytest.mark.parametrize("M,bit", [(200, 1), (16, 2)])
def test_pipeline_unwinds_when_its_code_producer_is_held_back(Lc, M, bit):
    c = _Case(Lc, M, 1024, 264, 3, 16, True)
    assert c.status() == 0
    assert Lc.qlinear_test_stall(bit, 20_000_000) == 0
    try:
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        assert c.launch() == 0
        status = c.status()
        elapsed = time.perf_counter() - t0
    finally:
        assert Lc.qlinear_test_stall(0, 1_000_000_000) == 0
    assert status == 6, status                                # QL_ERR_DEVICE_TIMEOUT
    assert elapsed < 0.9, elapsed                             # the shortened limit, not the default second
    assert c.status() == 0
    for _ in range(2):                                        # the next calls run normally
        c.check(c.run())
