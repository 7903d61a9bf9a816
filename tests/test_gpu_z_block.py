"""The operators together, as a transformer block uses them: norm -> QKV with adapters ... -> output projection with
adapters -> gate, residual and norm -> SwiGLU pair with adapters -> row-parallel down projection -> the next block's
norm from its partials.  Every step is checked against the oracle on the values the step before it produced, for a
single token, a few tokens of many requests and a batch of ragged requests with padding; and the whole chain, captured
once in a CUDA graph, replays to the same bytes with other inputs copied in."""
import numpy as np
import pytest
import torch

import group_wise_affine_qlinear_b200 as ql
from group_wise_affine_qlinear_b200 import synthetic as S
from group_wise_affine_qlinear_b200 import tp
from oracle import qlinear_oracle as O

from ._helpers import bf16_bits, random_layer, to_dev_bf16, to_dev_codes, to_dev_f16

pytestmark = pytest.mark.gpu

D, I, N_QKV, LAYERS, RANK = 512, 768, 1536, 4, 16
B = 2.0 ** -8                         # half a bf16 unit, relative


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required for -m gpu tests")
    ql.lib()
    yield
    assert ql.device_status() == 0


class _Block:
    def __init__(self, M, T, seed):
        rng = np.random.default_rng(seed)
        f32 = lambda v: np.asarray(v, np.float32)
        bits = lambda v: S.f32_to_bf16_bits(f32(v))
        w = lambda n, k: random_layer(rng, 1, k, n)[1:]
        self.w = {"qkv": w(N_QKV, D), "o": w(D, D), "gate": w(I, D), "up": w(I, D), "down": w(D, I)}
        self.lora = {k: (bits(rng.standard_normal((LAYERS, RANK, v[0].shape[1] * 8)) / 20),
                         bits(rng.standard_normal((LAYERS, v[0].shape[0], RANK)) / 20)) for k, v in self.w.items()}
        self.wd = {k: (to_dev_codes(c), to_dev_f16(s), to_dev_f16(b)) for k, (c, s, b) in self.w.items()}
        self.ld = {k: tuple(to_dev_bf16(t) for t in v) for k, v in self.lora.items()}
        self.scale = rng.uniform(0.5, 2.0, LAYERS).astype(np.float32)
        self.sd = torch.from_numpy(self.scale).cuda()
        vec = lambda rows: torch.from_numpy(f32(1 + 0.2 * rng.standard_normal((rows, D)))).cuda().bfloat16()
        self.norm = [dict(post_weight=vec(1)[0], pre_weight=vec(1)[0], gate=vec(T), scale=0.2 * vec(T),
                          shift=0.2 * vec(T)) for _ in range(3)]
        self.M, self.T, self.rng = M, T, rng

    def inputs(self, padding):
        rng, M = self.rng, self.M
        x = torch.from_numpy(rng.standard_normal((M, D)).astype(np.float32)).cuda().bfloat16()
        seg = np.sort(rng.integers(0, self.T, M)).astype(np.int32)
        ids = rng.integers(-1, LAYERS, M).astype(np.int32)
        seg[M - padding:] = ids[M - padding:] = -1
        return x, torch.from_numpy(seg).cuda(), torch.from_numpy(ids).cuda()

    def run(self, x, seg, ids):
        """Every intermediate, in order."""
        n0, n1, n2 = self.norm
        pre = {k: n0[k] for k in ("pre_weight", "scale", "shift")}
        h0 = torch.zeros_like(x)
        ql.norm_residual(x, segment_ids=seg, h=h0, **pre)
        qkv = ql.forward_lora(h0, *self.wd["qkv"], *self.ld["qkv"], ids, self.sd)
        mix = qkv[:, :D].contiguous()                      # stands for the attention's output
        o = ql.forward_lora(mix, *self.wd["o"], *self.ld["o"], ids, self.sd)
        x1, h1 = x.clone(), torch.zeros_like(x)
        ql.norm_residual(x1, o, segment_ids=seg, out=x1, h=h1, residual_scale=0.9, branch_scale=0.5, **n1)
        g = ql.swiglu_lora(h1, self.wd["gate"], self.wd["up"], self.ld["gate"], self.ld["up"], ids, self.sd)
        parts = torch.stack([ql.forward(tp.input_shard(g, r, 2), *tp.row_shard(*self.wd["down"], r, 2),
                                        out_dtype=torch.float32) for r in range(2)])
        x2, h2 = x1.clone(), torch.zeros_like(x)
        ql.norm_residual(x2, parts, segment_ids=seg, out=x2, h=h2, branch_scale=0.5, **n2)
        return h0, qkv, o, x1, h1, g, parts, x2, h2


def _f64(t):
    return t.double().cpu().numpy()


def _close(got, ref, bf16=True):
    """fp32 arithmetic of a few hundred terms (2^-14 of the row's largest value is far above its error and far below
    any mistake), and half a unit of bf16 storage."""
    row = np.abs(ref).max(axis=-1, keepdims=True)
    assert np.all(np.abs(got - ref) <= 2.0 ** -14 * row + (B * np.abs(ref) if bf16 else 0.0))


def _check_norm(x, y, out, h, seg, kw):
    kw = {k: (_f64(v) if isinstance(v, torch.Tensor) else v) for k, v in kw.items()}
    live = seg.cpu().numpy() >= 0
    yv = None if y is None else (_f64(y) if y.dim() == 3 else _f64(y)[None])
    r, hr = O.norm_residual_ref(_f64(x), yv, seg=seg.cpu().numpy(), **kw)
    if out is not None:
        _close(_f64(out)[live], r[live])
        assert torch.equal(out[~live], x[~live])           # rows behind the last sequence: left as they were
    _close(_f64(h)[live], hr[live])
    assert (h[~live] == 0).all()


@pytest.mark.parametrize("M,T,padding", [(1, 1, 0), (24, 5, 3), (333, 7, 20)])
def test_block(M, T, padding):
    blk = _Block(M, T, M)
    x, seg, ids = blk.inputs(padding)
    h0, qkv, o, x1, h1, g, parts, x2, h2 = blk.run(x, seg, ids)
    idn = ids.cpu().numpy()
    n0, n1, n2 = blk.norm
    _check_norm(x, None, None, h0, seg, {k: n0[k] for k in ("pre_weight", "scale", "shift")})
    for name, inp, out in (("qkv", h0, qkv), ("o", qkv[:, :D].contiguous(), o)):
        xb = bf16_bits(inp)
        ref = O.forward_ref(xb, *blk.w[name]) + O.lora_delta(xb, *blk.lora[name], blk.scale, idn)
        t = O.tolerance(O.decode_bf16(bf16_bits(out)), ref)
        assert t["ok"], (name, t)
    _check_norm(x, o, x1, h1, seg, dict(n1, residual_scale=0.9, branch_scale=0.5))
    hb = bf16_bits(h1)
    gl, ul = O.swiglu_linears(hb, blk.w["gate"], blk.w["up"])
    t = O.swiglu_tolerance(O.decode_bf16(bf16_bits(g)), gl + O.lora_delta(hb, *blk.lora["gate"], blk.scale, idn),
                           ul + O.lora_delta(hb, *blk.lora["up"], blk.scale, idn))
    assert t["ok"], t
    t = O.tolerance(_f64(parts.sum(0)), O.forward_ref(bf16_bits(g), *blk.w["down"]), bf16_output=False)
    assert t["ok"], t
    _check_norm(x1, parts, x2, h2, seg, dict(n2, branch_scale=0.5))


@pytest.mark.parametrize("M,T,padding", [(1, 1, 0), (200, 3, 9)])
def test_block_in_a_graph(M, T, padding):
    blk = _Block(M, T, 100 + M)
    first, second = blk.inputs(padding), blk.inputs(padding)
    want = [[t.clone() for t in blk.run(*inp)] for inp in (first, second)]
    static = [t.clone() for t in first]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = blk.run(*static)
    for inp, ref in ((first, want[0]), (second, want[1]), (first, want[0])):
        for s, t in zip(static, inp):
            s.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            assert torch.equal(a, b)
    del graph


def test_two_streams_at_once():
    """Two calls in flight on two streams, each with buffers of its own stream, give what they give alone."""
    blk = _Block(96, 3, 7)
    inp = [blk.inputs(0) for _ in range(2)]
    want = [[t.clone() for t in blk.run(*i)] for i in inp]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(3):
        outs = []
        for i, s in zip(inp, streams):
            with torch.cuda.stream(s):
                outs.append(blk.run(*i))
        torch.cuda.synchronize()
        for got, ref in zip(outs, want):
            for a, b in zip(got, ref):
                assert torch.equal(a, b)
