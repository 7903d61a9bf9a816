"""The epilogues, norms of heads and rotation together, as a block uses them: QKV projection with bias -> norms of queries
and keys and their rotation, in place inside the projection's output -> (an attention in elementary operations) -> output
projection with gate and residual, in place -> norm -> MLP of two projections, GELU in the first, gate and residual in
the second.  For one token, a few and a ragged batch with padding; every step against the oracle on the values that the
step before produced; the chain captured in a CUDA graph replays to the same bytes with other inputs, on two streams too."""
import numpy as np
import pytest
import torch

import group_wise_affine_qlinear_b200 as ql
from oracle import qlinear_oracle as O
from tests._helpers import random_layer, to_dev_codes, to_dev_f16

pytestmark = pytest.mark.gpu

H, KV, DH = 6, 2, 64
D, I = H * DH, 768
B = 2.0 ** -8                         # half a bf16 unit, relative


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required for -m gpu tests")
    ql.lib()
    yield
    assert ql.device_status() == 0


def _f64(t):
    return t.double().cpu().numpy()


class _Block:
    def __init__(self, seed, T=2):
        rng = np.random.default_rng(seed)
        self.rng, self.T = rng, T
        raw = {"qkv": (D, (H + 2 * KV) * DH), "o": (D, D), "up": (D, I), "down": (I, D)}
        raw = {k: random_layer(rng, 1, *v)[1:] for k, v in raw.items()}
        self.w64 = {k: O.dequant_exact(*v) for k, v in raw.items()}
        self.w = {k: (to_dev_codes(c), to_dev_f16(s), to_dev_f16(b)) for k, (c, s, b) in raw.items()}
        vec = lambda *shape: torch.from_numpy((0.5 * rng.standard_normal(shape)).astype(np.float32)).cuda()
        self.b_qkv, self.b_up, self.b_down = vec((H + 2 * KV) * DH), vec(I), vec(D)
        self.g_o, self.g_down = vec(T, D), vec(T, D)
        self.qw, self.kw, self.nw = 1 + vec(DH), 1 + vec(DH), 1 + vec(D)
        self.rot = ql.rotary_frequencies((12, 10, 10), 5e6, cycle=True)

    def inputs(self, M, padding):
        x = torch.from_numpy(self.rng.standard_normal((M, D)).astype(np.float32)).cuda().bfloat16()
        seg = np.sort(self.rng.integers(0, self.T, M)).astype(np.int32)
        seg[M - padding:] = -1
        pos = np.stack([np.arange(M), np.arange(M) // 7, np.arange(M) % 7]) + 1000
        return x, torch.from_numpy(seg).cuda(), torch.from_numpy(pos.astype(np.int32)).cuda()

    def run(self, x, seg, pos):
        """Every intermediate, in order; padding rows stay zero or what they were."""
        M = x.shape[0]
        zeros = lambda n: torch.zeros((M, n), dtype=torch.bfloat16, device="cuda")
        qkv = ql.forward_epilogue(x, *self.w["qkv"], bias=self.b_qkv, segment_ids=seg, out=zeros((H + 2 * KV) * DH))
        raw = qkv.clone()
        heads = qkv.view(M, H + 2 * KV, DH)
        q, k, v = heads[:, :H], heads[:, H:H + KV], heads[:, H + KV:]
        ql.qk_norm_rotary(q, k, pos, self.rot, q_weight=self.qw, k_weight=self.kw, segment_ids=seg, q_out=q, k_out=k)
        own = (seg[:, None] == seg[None, :]) & (seg >= 0)[:, None]
        kk, vv = (t.float().repeat_interleave(H // KV, 1) for t in (k, v))
        a = torch.einsum("mhd,nhd->hmn", q.float(), kk) / DH ** 0.5
        a = torch.softmax(a.masked_fill(~own[None], -1e30), -1)
        mix = torch.einsum("hmn,nhd->mhd", a, vv).reshape(M, D).bfloat16()
        x1 = x.clone()
        ql.forward_epilogue(mix, *self.w["o"], gate=self.g_o, residual=x1, segment_ids=seg, out=x1)
        _, h = ql.norm_residual(x1, pre_weight=self.nw, segment_ids=seg, h=zeros(D))
        u = ql.forward_epilogue(h, *self.w["up"], bias=self.b_up, activation="gelu_tanh", segment_ids=seg, out=zeros(I))
        x2 = x1.clone()
        ql.forward_epilogue(u, *self.w["down"], bias=self.b_down, gate=self.g_down, residual=x2, segment_ids=seg, out=x2)
        return raw, qkv, mix, x1, h, u, x2

    def check(self, x, seg, pos, steps):
        raw, qkv, mix, x1, h, u, x2 = (_f64(t) for t in steps)
        s, p, M = seg.cpu().numpy(), _f64(pos), x.shape[0]
        live = s >= 0

        def projected(name, inp, got, bias=None, act=None, gate=None, res=None):
            w = self.w64[name]
            lin, ez = inp @ w.T, (2.0 ** -11 + 2.0 ** -15) * (np.abs(inp) @ np.abs(w).T)
            b, g = None if bias is None else _f64(bias), None if gate is None else _f64(gate)
            y = O.epilogue_ref(lin, b, act, g, res, s)
            bound = 1.13 * (1.0 if g is None else np.abs(g)[np.maximum(s, 0)]) * (ez + 2.0 ** -18 * np.abs(lin + (0 if b is None else b)))
            assert np.all((np.abs(got - y) <= bound + B * (np.abs(y) + bound) + (0 if res is None else 2.0 ** -22 * np.abs(res)))[live]), name
        projected("qkv", _f64(x), raw, bias=self.b_qkv)
        heads, before = (t.reshape(M, H + 2 * KV, DH) for t in (qkv, raw))
        turns, axes = _f64(self.rot[0]), self.rot[1].cpu().numpy()
        for lo, hi, w in ((0, H, self.qw), (H, H + KV, self.kw)):
            n = O.rms_normed(before[:, lo:hi], 1e-6) * _f64(w)
            want = O.rotary_ref(n, p, turns, axes)
            size = np.abs(n) + np.abs(np.roll(n, 32, axis=-1))
            assert np.all((np.abs(heads[:, lo:hi] - want) <= 2.0 ** -18 * size + B * (np.abs(want) + size * 2.0 ** -18))[live])
        assert np.array_equal(heads[:, H + KV:], before[:, H + KV:]) and not qkv[~live].any()
        projected("o", mix, x1, gate=self.g_o, res=_f64(x))
        projected("up", h, u, bias=self.b_up, act="gelu_tanh")
        projected("down", u, x2, bias=self.b_down, gate=self.g_down, res=x1)
        for a in (x1, x2):
            assert np.array_equal(a[~live], _f64(x)[~live])
        assert not u[~live].any()


@pytest.mark.parametrize("M,padding", [(1, 0), (7, 2), (50, 0), (300, 23), (1500, 100)])
def test_a_block_step_by_step(M, padding):
    blk = _Block(M)
    args = blk.inputs(M, padding)
    blk.check(*args, blk.run(*args))


@pytest.mark.parametrize("M,padding", [(3, 0), (40, 3), (250, 20)])
def test_a_captured_block_and_two_streams(M, padding):
    blk = _Block(100 + M)
    args = blk.inputs(M, padding)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        blk.run(*args)                                      # (library loading and allocations outside the capture)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            steps = blk.run(*args)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        x, seg, pos = blk.inputs(M, padding)
        for to, new in zip(args, (x, seg, pos)):
            to.copy_(new)
        graph.replay()
        want = blk.run(x, seg, pos)
        for a, b in zip(steps, want):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    torch.cuda.synchronize()
    outs = []
    for st in (torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(st):
            outs.append(blk.run(*args))
    torch.cuda.synchronize()
    for o in outs:
        for a, b in zip(o, steps):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
