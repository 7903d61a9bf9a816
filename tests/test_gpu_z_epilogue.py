"""GPU parity of projections with bias, activation, gate and residual in their epilogue against float64.

Bounds, with u = 2^-24 (half an fp32 unit) and b = 2^-8 (half a bf16 unit, relative):
  z   every weight is rounded once to f16 (2^-11 relative) and the products accumulate in fp32, each of at most K / 16
      additions in the tensor core and a few tens behind it off by 2 u at most (it may cut instead of round):
      e_z = (2^-11 + (K / 16 + 64) 2 u) sum_k |x w|; the activations are exact above 2^-28 of their row's largest.
  a   1.13 e_z (the steepest slope of the activations) + 2^-20 |z|: the hardware exponential errs by (2 + 1.2 |v|) 2^-23
      relative at an argument v, times e^-v |v| <= 0.37 of |z| where v is large; its division by 2^-22; Abramowitz and
      Stegun's 1 - erf by 1.5e-7, half of it times |z|
  y   |gate| e_a + 4 u (|gate a| + |residual|), + b |y| for bf16 storage
The one-launch kernel of few tokens multiplies exact codes, offset by 128: five additions per group off by 2 u of at most
143 sum |x|, times the group's scale s, 2^-13 s sum |x|; below the 2^-11 sum |x w| above wherever the weights are a
quarter of s on average (those here are 3.7 s).
Integer layers are exact instead: every product and sum is a whole number of quarters below 2^24.
"""
import numpy as np
import pytest
import torch

import group_wise_affine_qlinear_b200 as ql
from group_wise_affine_qlinear_b200 import synthetic as S
from oracle import qlinear_oracle as O
from tests._helpers import random_layer, random_layer8, to_dev_bf16, to_dev_codes, to_dev_f16

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8
CALL = {4: ql.forward_epilogue, 8: ql.forward8_epilogue}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required for -m gpu tests")
    ql.lib()
    yield
    assert ql.device_status() == 0


def _dev(v, dt):
    return torch.from_numpy(np.asarray(v, np.float32)).cuda().to(dt)


def _f64(t):
    return None if t is None else t.double().cpu().numpy()


def _weights(rng, K, N, bits):
    """An integer weight: codes of either width with scale 1 and a bias of half their range."""
    codes = rng.integers(0, 1 << 32, size=(N, K * bits // 32), dtype=np.uint32)
    s, b = np.ones((N, K // 64), np.float16), np.full((N, K // 64), -float(2 ** (bits - 1)), np.float16)
    q = O.unpack_codes(codes, K) if bits == 4 else O.unpack_codes8(codes, K)
    return (to_dev_codes(codes), to_dev_f16(s), to_dev_f16(b)), q.astype(np.float64) - 2 ** (bits - 1)


def _exact_case(rng, M, K, N, bits, out, params, T=3, padding=True):
    w, wv = _weights(rng, K, N, bits)
    xv = rng.integers(-2, 3, (M, K)).astype(np.float64)
    kw = {"bias": _dev(rng.integers(-8, 9, N) / 4, DT[params]),
          "gate": _dev(2.0 ** rng.integers(-2, 3, (T, N)) * rng.choice([-1, 1], (T, N)), DT[params]),
          "residual": _dev(rng.integers(-64, 65, (M, N)) / 4, DT[out])}
    seg = rng.integers(-1 if padding else 0, T, M).astype(np.int32)
    return _dev(xv, torch.bfloat16), w, kw, seg, xv @ wv.T


def _rounded(y, out):
    return torch.from_numpy(y).to(DT[out])                 # one rounding from float64's exact value


def _check_exact(got, y, seg, out, sentinel):
    got = got.cpu()
    want = _rounded(np.nan_to_num(y), out)
    live = torch.from_numpy(seg >= 0)
    assert torch.equal(got[live], want[live])
    assert torch.equal(got[~live], sentinel.cpu()[~live])


SHAPES = [(1, 64, 8), (1, 1024, 256), (3, 320, 72), (17, 576, 520), (20, 4096, 2056), (33, 128, 136), (64, 1024, 1288), (65, 64, 8),
          (97, 320, 264), (192, 1024, 256), (193, 4096, 72), (400, 192, 520), (1200, 128, 2056), (777, 1024, 4608)]


@pytest.mark.parametrize("out,params", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_exact_integers(M, K, N, bits, out, params):
    """Bias, gate of mixed segments, residual and padding rows, to the last bit, out of place and in place."""
    rng = np.random.default_rng(M * 7 + K + N + bits)
    x, w, kw, seg, lin = _exact_case(rng, M, K, N, bits, out, params)
    y = O.epilogue_ref(lin, _f64(kw["bias"]), None, _f64(kw["gate"]), _f64(kw["residual"]), seg)
    ids = torch.from_numpy(seg).cuda()
    sentinel = torch.full((M, N), -77.0, dtype=DT[out], device="cuda")
    got = sentinel.clone()
    assert CALL[bits](x, *w, segment_ids=ids, out=got, **kw) is got
    _check_exact(got, y, seg, out, sentinel)
    before = kw["residual"].clone()
    CALL[bits](x, *w, segment_ids=ids, out=kw["residual"], **kw)
    _check_exact(kw["residual"], y, seg, out, before)
    assert ql.device_status() == 0


@pytest.mark.parametrize("M,K,N", [(5, 128, 136), (200, 128, 136), (130, 2048, 72), (2000, 64, 264)])
@pytest.mark.parametrize("use", ["bias", "gate", "residual", ""])
def test_each_part_alone(M, K, N, use):
    """One argument at a time: with none of them the result is forward()'s."""
    rng = np.random.default_rng(M + len(use))
    x, w, kw, seg, lin = _exact_case(rng, M, K, N, 4, "bf16", "bf16", T=1)
    kw = {use: kw[use]} if use else {}
    y = O.epilogue_ref(lin, _f64(kw.get("bias")), None, _f64(kw.get("gate")), _f64(kw.get("residual")))
    got = ql.forward_epilogue(x, *w, **kw)
    assert torch.equal(got.cpu(), _rounded(y, "bf16"))
    if not use:
        assert torch.equal(got, ql.forward(x, *w))


def _layer(rng, M, K, N, bits):
    xb, codes, s, b = (random_layer if bits == 4 else random_layer8)(rng, M, K, N)
    w64 = (O.dequant_exact if bits == 4 else O.dequant8_exact)(codes, s, b)
    xv = O.decode_bf16(xb)
    lin = xv @ w64.T
    ez = (2.0 ** -11 + (K / 16 + 64) * 2 * U) * (np.abs(xv) @ np.abs(w64).T)
    return to_dev_bf16(xb), (to_dev_codes(codes), to_dev_f16(s), to_dev_f16(b)), lin, ez


def _bounded(got, lin, ez, kw, act, seg, out):
    bias, gate, res = _f64(kw.get("bias")), _f64(kw.get("gate")), _f64(kw.get("residual"))
    z = lin + (0.0 if bias is None else bias)
    a = O.activation(z, act)
    g = np.ones_like(z) if gate is None else np.abs(gate[np.maximum(seg, 0)])
    ea = (1.13 if act else 1.0) * (ez + 2 * U * np.abs(z)) + 2.0 ** -20 * np.abs(z)
    y = O.epilogue_ref(lin, bias, act, gate, res, seg)
    bound = g * ea + 4 * U * (np.abs(g * a) + (0.0 if res is None else np.abs(res)))
    if out == "bf16":
        bound = bound + B * (np.abs(y) + bound)
    live = seg >= 0
    err = np.abs(_f64(got) - y)[live]
    assert np.all(err <= bound[live]), float((err / bound[live]).max())


@pytest.mark.parametrize("act", [None, "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M,K,N,bits,out", [(1, 512, 136, 4, "bf16"), (40, 128, 264, 8, "f32"), (64, 1024, 72, 4, "f32"),
                                            (70, 1024, 264, 8, "bf16"), (300, 64, 520, 4, "bf16"), (500, 192, 1032, 4, "f32"),
                                            (260, 2048, 128, 8, "f32"), (1000, 128, 3080, 8, "bf16")])
def test_random_layers(M, K, N, bits, out, act):
    rng = np.random.default_rng(M + K + N)
    x, w, lin, ez = _layer(rng, M, K, N, bits)
    T = min(4, M)
    seg = np.sort(rng.integers(0, T, M)).astype(np.int32)
    seg[M - M // 7:] = -1
    kw = {"bias": _dev(rng.standard_normal(N), DT["f32"]), "gate": _dev(0.5 * rng.standard_normal((T, N)), DT["f32"]),
          "residual": _dev(3 * rng.standard_normal((M, N)), DT[out])}
    got = CALL[bits](x, *w, activation=act, segment_ids=torch.from_numpy(seg).cuda(), out_dtype=DT[out], **kw)
    _bounded(got, lin, ez, kw, act, seg, out)


@pytest.mark.parametrize("M", [4, 150])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activations_at_their_ends(M, act):
    """x = 0, so z is the bias: from far below to far above, and what is not finite."""
    N = 256
    z = np.concatenate([np.linspace(-12, 12, 120), [v * s for v in (20.0, 88.0, 89.0, 300.0, 1e4, 1e13, 1e30) for s in (1, -1)],
                        np.zeros(N)])[:N].astype(np.float32)
    z[200], z[201] = np.inf, np.nan
    w, _ = _weights(np.random.default_rng(0), 64, N, 4)
    x = torch.zeros((M, 64), dtype=torch.bfloat16, device="cuda")
    got = _f64(ql.forward_epilogue(x, *w, bias=_dev(z, DT["f32"]), activation=act, out_dtype=torch.float32))
    assert np.all(got == got[0:1], where=~np.isnan(got)) and np.isnan(got[:, 201]).all() and np.isposinf(got[:, 200]).all()
    ok = np.isfinite(z)
    with np.errstate(over="ignore"):
        want = O.activation(z[ok].astype(np.float64), act)
    assert np.all(np.abs(got[0, ok] - want) <= 2.0 ** -20 * np.abs(z[ok]))


def test_what_is_not_finite_stays_in_its_place():
    """A NaN or infinity of the residual reaches its own element, one of x its own row, one of a padding row nothing."""
    rng = np.random.default_rng(3)
    for M in (20, 300):
        x, w, kw, seg, lin = _exact_case(rng, M, 128, 136, 4, "bf16", "bf16", padding=False)
        seg[5:9] = -1
        ids = torch.from_numpy(seg).cuda()
        clean = ql.forward_epilogue(x, *w, segment_ids=ids, out=torch.zeros((M, 136), dtype=torch.bfloat16, device="cuda"), **kw)
        x[6, 3], kw["residual"][7, 5] = float("nan"), float("inf")             # both in padding rows
        x[2, 100] = float("inf")
        kw["residual"][11, 70], kw["residual"][12, 135] = float("nan"), float("-inf")
        got = ql.forward_epilogue(x, *w, segment_ids=ids, out=torch.zeros((M, 136), dtype=torch.bfloat16, device="cuda"), **kw)
        assert torch.isnan(got[11, 70]) and got[12, 135] == float("-inf") and not torch.isfinite(got[2]).any()
        same = torch.ones((M, 136), dtype=torch.bool, device="cuda")
        same[2] = False
        same[11, 70] = same[12, 135] = False
        assert torch.equal(got[same], clean[same])


@pytest.mark.parametrize("M", [10, 250])
def test_segments_out_of_range(M):
    rng = np.random.default_rng(4)
    x, w, kw, seg, lin = _exact_case(rng, M, 128, 72, 4, "bf16", "bf16", T=2)
    seg[3], seg[9] = 2, 2 ** 31 - 1
    sentinel = torch.full((M, 72), 5.0, dtype=torch.bfloat16, device="cuda")
    got = ql.forward_epilogue(x, *w, segment_ids=torch.from_numpy(seg).cuda(), out=sentinel.clone(), **kw)
    assert ql.device_status() == 1
    seg[3] = seg[9] = -1
    y = O.epilogue_ref(lin, _f64(kw["bias"]), None, _f64(kw["gate"]), _f64(kw["residual"]), seg)
    _check_exact(got, y, seg, "bf16", sentinel)
    # every row padding: nothing is written
    got = ql.forward_epilogue(x, *w, segment_ids=torch.full((M,), -1, dtype=torch.int32, device="cuda"), out=sentinel.clone(), **kw)
    assert torch.equal(got, sentinel) and ql.device_status() == 0


@pytest.mark.parametrize("M,K,N", [(8, 512, 264), (130, 2048, 72), (600, 128, 2056)])
def test_poisoned_workspace_replays_and_streams(M, K, N):
    rng = np.random.default_rng(5)
    x, w, kw, seg, lin = _exact_case(rng, M, K, N, 4, "bf16", "f32")
    ids = torch.from_numpy(seg).cuda()
    y = O.epilogue_ref(lin, _f64(kw["bias"]), None, _f64(kw["gate"]), _f64(kw["residual"]), seg)
    sentinel = torch.full((M, N), 9.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((ql.epilogue_workspace_size(M, K, N),), 0xFF, dtype=torch.uint8, device="cuda")
    out = sentinel.clone()
    _check_exact(ql.forward_epilogue(x, *w, segment_ids=ids, out=out, workspace=ws, **kw), y, seg, "bf16", sentinel)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            ql.forward_epilogue(x, *w, segment_ids=ids, out=out, workspace=ws, **kw)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        out.copy_(sentinel)
        ws.fill_(0xFF)
        graph.replay()
        _check_exact(out, y, seg, "bf16", sentinel)
    # two streams at once, each with its own workspace
    torch.cuda.synchronize()
    outs = [sentinel.clone() for _ in range(2)]
    torch.cuda.synchronize()
    for o, st in zip(outs, (torch.cuda.Stream(), torch.cuda.Stream())):
        ql.forward_epilogue(x, *w, segment_ids=ids, out=o, stream=st, **kw)
    torch.cuda.synchronize()
    for o in outs:
        _check_exact(o, y, seg, "bf16", sentinel)


def test_offsets_past_32_bits():
    """Outputs and residual of more than 2^31 elements: the first rows, the last ones and those where 2^31 falls."""
    M, K, N = 300_007, 64, 7208
    rng = np.random.default_rng(6)
    w, wv = _weights(rng, K, N, 4)
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randint(-2, 3, (M, K), generator=g, device="cuda").to(torch.bfloat16)
    res = torch.randint(-64, 65, (M, N), generator=g, device="cuda", dtype=torch.int8).to(torch.bfloat16)
    at = (1 << 31) // N
    rows = torch.tensor([0, 1, at - 1, at, at + 1, M - 2, M - 1], device="cuda")
    want = _f64(res[rows]) + _f64(x[rows]) @ wv.T
    seg = torch.zeros(M, dtype=torch.int32, device="cuda")
    seg[at + 2] = -1                                        # a block with a padding row is stored row by row
    kept = res[at + 2].clone()
    ql.forward_epilogue(x, *w, residual=res, segment_ids=seg, out=res)
    assert torch.equal(res[rows].cpu(), _rounded(want, "bf16"))
    assert torch.equal(res[at + 2], kept)


def test_refusals():
    rng = np.random.default_rng(7)
    x, w, kw, seg, _ = _exact_case(rng, 16, 128, 72, 4, "bf16", "bf16")
    ids = torch.from_numpy(seg).cuda()
    call = lambda **over: ql.forward_epilogue(x, *w, **{**kw, "segment_ids": ids, **over})
    for over in (dict(segment_ids=None), dict(bias=kw["bias"][:-1]), dict(bias=kw["bias"].float()), dict(gate=kw["gate"].t()),
                 dict(residual=kw["residual"].float(), out_dtype=torch.bfloat16), dict(residual=kw["residual"][:-1]),
                 dict(segment_ids=ids.long()), dict(activation="tanh"), dict(out_dtype=torch.float16), dict(bias=kw["bias"].cpu()),
                 dict(out=torch.empty((16, 72), device="cuda")), dict(workspace=torch.empty(8)), dict(gate=kw["gate"][:0])):
        with pytest.raises(ValueError):
            call(**over)
    assert ql.epilogue_workspace_size(16, 128, 72) == 0     # (one launch: whatever it is given is not looked at)
    x, w, kw, seg, _ = _exact_case(rng, 40, 128, 72, 4, "bf16", "bf16")
    ids = torch.from_numpy(seg).cuda()
    with pytest.raises(ql.QLinearError) as e:
        call(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 4
    with pytest.raises(ql.QLinearError) as e:
        call(out=kw["residual"], residual=kw["residual"], workspace=kw["residual"])
    assert e.value.status in (1, 4)
