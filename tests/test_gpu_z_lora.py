"""GPU parity of the low-rank adapters beside a packed projection, and of the SwiGLU pair with them.

Two kinds of check:
  * Integers: x in [-4, 4], W = q - 8 (or q - 128), A and B in {-1, 0, 1}, factors powers of two.  Every product
    and sum is an integer multiple of 1/2 below 2^24, exact in fp32 in any order; t is below 2^16 in those units,
    so its two bf16 parts hold it exactly.  The fp32 output must equal the integer result bit for bit, whatever the
    path, the tile, the rank or the order of the ids.
  * Random layers against the oracle's float64 result within reading R5 (R11 for the pair).  The adapters add to
    R5's errors the rounding of t's two parts, 2^-16 relative, and fp32 sums, both far below its 4e-3.
"""
import numpy as np
import pytest
import torch

import group_wise_affine_qlinear_b200 as ql
from group_wise_affine_qlinear_b200 import synthetic as S
from oracle import qlinear_oracle as O

from ._helpers import (FUSED_TILE_TOKENS, bf16_bits, random_layer, random_layer8, sample_rows, to_dev_bf16,
                       to_dev_codes, to_dev_f16)

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


def _ids(rng, M, n, how):
    if how == "none":
        return np.full(M, -1, np.int32)
    if how == "one":
        return np.full(M, n - 1, np.int32)
    if how == "mixed":                                    # any order, some rows without an adapter
        return rng.integers(-1, n, M).astype(np.int32)
    if how == "distinct":                                 # as many adapters as there are, then again
        return (rng.permutation(M) % n).astype(np.int32)
    cuts = np.sort(rng.integers(0, M + 1, n))             # "runs": ragged runs, the rows before the first without
    return (np.searchsorted(cuts, np.arange(M), side="right") - 1).astype(np.int32)


def _int_layer(rng, N, K, bits):
    q = rng.integers(0, 1 << bits, size=(N, K))
    codes = O.pack_codes(q) if bits == 4 else O.pack_codes8(q)
    one = np.ones((N, K // 64), np.float16)
    return (codes, one, -one * (1 << (bits - 1))), q.astype(np.float64) - (1 << (bits - 1))


def _dev_w(w):
    return to_dev_codes(w[0]), to_dev_f16(w[1]), to_dev_f16(w[2])


def _int_adapters(rng, n, r, K, N):
    return rng.integers(-1, 2, (n, r, K)).astype(np.float64), rng.integers(-1, 2, (n, N, r)).astype(np.float64)


def _dev_ids(ids):
    return torch.from_numpy(ids).cuda()


def _call(bits):
    return ql.forward_lora if bits == 4 else ql.forward8_lora


CASES = [
    # M, K, N, bits, adapters, rank, ids              weight streaming (M <= 64)
    (1, 64, 8, 4, 1, 8, "one"), (1, 4608, 264, 4, 3, 16, "one"), (2, 128, 136, 8, 2, 8, "mixed"),
    (16, 512, 264, 4, 16, 16, "distinct"), (17, 576, 136, 8, 4, 24, "runs"), (33, 1024, 520, 4, 40, 40, "distinct"),
    (64, 2048, 264, 4, 5, 64, "mixed"), (64, 320, 8, 8, 64, 128, "distinct"), (48, 4160, 136, 4, 2, 128, "runs"),
    (7, 256, 64, 4, 3, 8, "none"),
    # fused kernel
    (65, 64, 8, 4, 1, 8, "one"), (65, 4096, 264, 4, 3, 16, "mixed"), (100, 8192, 136, 8, 9, 24, "distinct"),
    (191, 512, 264, 4, 5, 40, "runs"), (192, 576, 520, 4, 48, 8, "distinct"), (193, 320, 136, 8, 2, 64, "mixed"),
    (400, 1024, 264, 4, 33, 16, "mixed"), (400, 256, 776, 8, 200, 8, "distinct"), (577, 128, 264, 4, 1, 128, "one"),
    (300, 640, 136, 4, 6, 48, "none"), (1000, 192, 2056, 4, 7, 16, "runs"), (700, 512, 264, 4, 30, 128, "mixed"),
]


@pytest.mark.parametrize("M,K,N,bits,n,r,how", CASES)
def test_integers_exact(M, K, N, bits, n, r, how):
    rng = np.random.default_rng(M * 1000003 + K * 101 + N + r)
    w, wv = _int_layer(rng, N, K, bits)
    x = rng.integers(-4, 5, (M, K)).astype(np.float64)
    a, b = _int_adapters(rng, n, r, K, N)
    scale = np.array([0.5, 1.0, 2.0], np.float32)[rng.integers(0, 3, n)]
    ids = _ids(rng, M, n, how)
    ref = x @ wv.T + O.lora_delta(_bits(x), _bits(a), _bits(b), scale, ids)
    dev = (to_dev_bf16(_bits(x)), *_dev_w(w), to_dev_bf16(_bits(a)), to_dev_bf16(_bits(b)), _dev_ids(ids),
           torch.from_numpy(scale).cuda())
    y = _call(bits)(*dev, out_dtype=torch.float32)
    assert ("lora" in ql.last_dispatch()) and (("skinny" in ql.last_dispatch()) == (M <= 64))
    got = y.double().cpu().numpy()
    assert np.array_equal(got, ref), np.argwhere(got != ref)[:5]
    # bf16 output: the same value rounded once
    yb = _call(bits)(*dev)
    assert torch.equal(yb, y.bfloat16())


@pytest.mark.parametrize("M", [40, 300])
def test_no_scale_is_one_and_no_adapter_is_the_plain_layer(M):
    rng = np.random.default_rng(5)
    K, N, n, r = 512, 264, 3, 16
    x, codes, s, b = random_layer(rng, M, K, N)
    la, lb = (to_dev_bf16(_bits(v)) for v in (rng.standard_normal((n, r, K)) / 20, rng.standard_normal((n, N, r)) / 50))
    ids = _dev_ids(_ids(rng, M, n, "mixed"))
    dev = (to_dev_bf16(x), to_dev_codes(codes), to_dev_f16(s), to_dev_f16(b), la, lb)
    ones = torch.ones(n, device="cuda")
    assert torch.equal(ql.forward_lora(*dev, ids), ql.forward_lora(*dev, ids, ones))
    none = torch.full_like(ids, -1)
    assert torch.equal(ql.forward_lora(*dev, none), ql.forward(*dev[:4]))
    # rows without an adapter are the plain layer's, bit for bit, among rows with one
    y, plain = ql.forward_lora(*dev, ids), ql.forward(*dev[:4])
    assert torch.equal(y[ids < 0], plain[ids < 0])
    assert not torch.equal(y[ids >= 0], plain[ids >= 0])


@pytest.mark.parametrize("M,K,N,bits,n,r,how", [
    (1, 4608, 4608, 4, 4, 16, "one"), (32, 4608, 1032, 4, 30, 16, "distinct"), (8, 53248, 520, 8, 3, 32, "mixed"),
    (333, 4608, 1032, 4, 5, 24, "runs"), (1021, 4608, 776, 8, 12, 64, "runs"), (130, 8192, 264, 4, 3, 8, "mixed"),
])
def test_random_layers(M, K, N, bits, n, r, how):
    rng = np.random.default_rng(M + K + N)
    x, codes, s, b = (random_layer if bits == 4 else random_layer8)(rng, M, K, N)
    a, up = _bits(rng.standard_normal((n, r, K)) / np.sqrt(K)), _bits(0.05 * rng.standard_normal((n, N, r)))
    scale = rng.uniform(0.5, 2.0, n).astype(np.float32)
    ids = _ids(rng, M, n, how)
    y = _call(bits)(to_dev_bf16(x), to_dev_codes(codes), to_dev_f16(s), to_dev_f16(b), to_dev_bf16(a), to_dev_bf16(up),
                    _dev_ids(ids), torch.from_numpy(scale).cuda())
    rows = sample_rows(M, n_random=40, seed=M, tile=FUSED_TILE_TOKENS)
    base = (O.forward_rows if bits == 4 else O.forward8_rows)(x, codes, s, b, rows)
    ref = base + O.lora_delta(x[rows], a, up, scale, ids[rows])
    t = O.tolerance(O.decode_bf16(bf16_bits(y)[rows]), ref)
    assert t["ok"], t


@pytest.mark.parametrize("M", [20, 400])
def test_large_and_small_adapters(M):
    """Adapters far above and far below the layer's own magnitude: t's parts have fp32's exponents, so neither
    overflows.  With W = 0 the output is the adapters' alone: relative error 2^-16 of t's parts, 2^-9 of the output's
    rounding and fp32 sums of K and r terms."""
    rng = np.random.default_rng(6)
    K, N, n, r = 512, 136, 3, 16
    codes = np.zeros((N, K // 8), np.uint32)
    zero = np.zeros((N, K // 64), np.float16)
    x = rng.standard_normal((M, K))
    x[1] *= 2.0 ** 40
    x[2] *= 2.0 ** -40
    a = rng.standard_normal((n, r, K)) * np.array([1.0, 2.0 ** 30, 2.0 ** -30])[:, None, None]
    b = rng.standard_normal((n, N, r)) * np.array([1.0, 2.0 ** 20, 2.0 ** -40])[:, None, None]
    ids = (np.arange(M) % n).astype(np.int32)
    xb, ab, bb = _bits(x), _bits(a), _bits(b)
    y = ql.forward_lora(to_dev_bf16(xb), to_dev_codes(codes), to_dev_f16(zero), to_dev_f16(zero), to_dev_bf16(ab),
                        to_dev_bf16(bb), _dev_ids(ids), out_dtype=torch.float32).double().cpu().numpy()
    xv, av, bv = O.decode_bf16(xb), O.decode_bf16(ab), O.decode_bf16(bb)
    ref = O.lora_delta(xb, ab, bb, None, ids)
    # |t| <= sum |x||A| =: u; each t errs by 2^-16 |t| and K roundings of 2^-24 of u; then r more terms
    u = np.einsum("mk,mjk->mj", np.abs(xv), np.abs(av[ids]))
    bound = np.einsum("mj,mnj->mn", u, np.abs(bv[ids])) * (2.0 ** -16 + (K + 2 * r) * 2.0 ** -23)
    assert np.all(np.abs(y - ref) <= bound)


@pytest.mark.parametrize("M", [20, 400])
def test_factors_far_from_one_on_rows_far_from_one(M):
    """A row near the bottom of bf16's range with a large factor, and one near its top with a small one: the product of
    the factor and the row's own power of two would leave fp32's range, t itself and t over that power do not.  Bound as
    in test_large_and_small_adapters."""
    rng = np.random.default_rng(16)
    K, N, n, r = 512, 136, 3, 16
    codes = np.zeros((N, K // 8), np.uint32)
    zero = np.zeros((N, K // 64), np.float16)
    x = rng.standard_normal((M, K))
    x[1::3] *= 2.0 ** -101
    x[2::3] *= 2.0 ** 112
    scale = np.array([1.0, 2.0 ** 20, 2.0 ** -50], np.float32)
    ids = (np.arange(M) % n).astype(np.int32)
    xb, ab, bb = _bits(x), _bits(rng.standard_normal((n, r, K))), _bits(rng.standard_normal((n, N, r)))
    y = ql.forward_lora(to_dev_bf16(xb), to_dev_codes(codes), to_dev_f16(zero), to_dev_f16(zero), to_dev_bf16(ab),
                        to_dev_bf16(bb), _dev_ids(ids), torch.from_numpy(scale).cuda(),
                        out_dtype=torch.float32).double().cpu().numpy()
    xv, av, bv = O.decode_bf16(xb), O.decode_bf16(ab), O.decode_bf16(bb)
    ref = O.lora_delta(xb, ab, bb, scale, ids)
    u = np.einsum("mk,mjk->mj", np.abs(xv), np.abs(av[ids])) * scale[ids].astype(np.float64)[:, None]
    bound = np.einsum("mj,mnj->mn", u, np.abs(bv[ids])) * (2.0 ** -16 + (K + 2 * r) * 2.0 ** -23)
    assert np.all(np.abs(y - ref) <= bound)


@pytest.mark.parametrize("M", [24, 300])
def test_non_finite_rows_and_adapters_stay_in_their_rows(M):
    rng = np.random.default_rng(7)
    K, N, n, r = 256, 136, 4, 16
    x, codes, s, b = random_layer(rng, M, K, N)
    a, up = _bits(rng.standard_normal((n, r, K))), _bits(rng.standard_normal((n, N, r)))
    ids = (np.arange(M) % n).astype(np.int32)
    dev = lambda x_, a_, up_: ql.forward_lora(to_dev_bf16(x_), to_dev_codes(codes), to_dev_f16(s), to_dev_f16(b),
                                              to_dev_bf16(a_), to_dev_bf16(up_), _dev_ids(ids))
    clean = dev(x, a, up)
    xn = x.copy()
    xn[5, 17] = 0x7FC0                                    # a NaN activation
    y = dev(xn, a, up)
    assert torch.isnan(y[5]).all()
    keep = torch.arange(M) != 5
    assert torch.equal(y[keep.cuda()], clean[keep.cuda()])
    an = a.copy()
    an[2, 3, 9] = 0x7F80                                  # an infinite entry of one adapter's A
    y = dev(x, an, up)
    own = torch.from_numpy(ids == 2).cuda()
    assert not torch.isfinite(y[own]).all()
    assert torch.equal(y[~own], clean[~own])
    assert ql.device_status() == 0
    un = up.copy()
    un[1, 7, 2] = 0x7FC0                                  # a NaN entry of one adapter's B: counts as zero, recorded
    y = dev(x, a, un)
    assert ql.device_status() == 1
    un[1, 7, 2] = 0
    assert torch.equal(y, dev(x, a, un))
    assert ql.device_status() == 0


@pytest.mark.parametrize("M", [9, 210])
def test_id_out_of_range_is_recorded_and_counts_as_none(M):
    rng = np.random.default_rng(8)
    K, N, n, r = 128, 72, 2, 8
    x, codes, s, b = random_layer(rng, M, K, N)
    args = (to_dev_bf16(x), to_dev_codes(codes), to_dev_f16(s), to_dev_f16(b),
            to_dev_bf16(_bits(rng.standard_normal((n, r, K)))), to_dev_bf16(_bits(rng.standard_normal((n, N, r)))))
    ids = _ids(rng, M, n, "mixed")
    bad = ids.copy()
    bad[3], bad[M - 1] = n, -7
    good = ids.copy()
    good[3] = good[M - 1] = -1
    y = ql.forward_lora(*args, _dev_ids(bad))
    assert ql.device_status() == 1
    assert torch.equal(y, ql.forward_lora(*args, _dev_ids(good)))
    assert ql.device_status() == 0


@pytest.mark.parametrize("M", [24, 300])
def test_views_at_16_byte_offsets_and_ids_at_4(M):
    """Tensors that start inside larger ones: 16-byte offsets everywhere, 4-byte ones for ids and factors."""
    rng = np.random.default_rng(9)
    K, N, n, r = 192, 72, 3, 8
    w, wv = _int_layer(rng, N, K, 4)
    x = rng.integers(-4, 5, (M, K)).astype(np.float64)
    a, b = _int_adapters(rng, n, r, K, N)
    ids = _ids(rng, M, n, "mixed")

    def shifted(t, elems):
        buf = torch.empty(t.numel() + elems, dtype=t.dtype, device="cuda")
        v = buf[elems:].view(t.shape)
        v.copy_(t)
        return v
    c, s, bi = _dev_w(w)
    y = ql.forward_lora(shifted(to_dev_bf16(_bits(x)), 8), shifted(c, 4), shifted(s, 8), shifted(bi, 8),
                        shifted(to_dev_bf16(_bits(a)), 8), shifted(to_dev_bf16(_bits(b)), 8), shifted(_dev_ids(ids), 1),
                        shifted(torch.full((n,), 2.0, device="cuda"), 1), out_dtype=torch.float32)
    ref = x @ wv.T + O.lora_delta(_bits(x), _bits(a), _bits(b), np.full(n, 2.0), ids)
    assert np.array_equal(y.double().cpu().numpy(), ref)


def _one(rng, M, K, N, n, r):
    x, codes, s, b = random_layer(rng, M, K, N)
    return (to_dev_bf16(x), to_dev_codes(codes), to_dev_f16(s), to_dev_f16(b),
            to_dev_bf16(_bits(rng.standard_normal((n, r, K)) / 10)), to_dev_bf16(_bits(rng.standard_normal((n, N, r)) / 10)),
            _dev_ids(_ids(rng, M, n, "mixed")), torch.rand(n, device="cuda"))


@pytest.mark.parametrize("M,K,N", [(5, 1024, 264), (64, 4160, 136), (130, 8192, 264), (900, 512, 776)])
def test_repeats_with_a_poisoned_workspace_and_replays(M, K, N):
    """Same bytes on every call, whatever the workspace held; on another stream; and from two captured graphs that
    share a workspace, replayed one after the other."""
    rng = np.random.default_rng(M)
    args, other = _one(rng, M, K, N, 5, 24), _one(rng, M, K, N, 5, 24)
    ref, ref2 = ql.forward_lora(*args), ql.forward_lora(*other)
    ws = torch.empty(ql.lora_workspace_size(M, K, N, 5, 24), dtype=torch.uint8, device="cuda")
    for fill in (0xFF, 0x00, 0x7F):
        ws.fill_(fill)
        assert torch.equal(ql.forward_lora(*args, workspace=ws), ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = ql.forward_lora(*args, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, ref)
    outs, graphs = [torch.empty_like(ref) for _ in range(2)], []
    with torch.cuda.stream(side):
        ql.forward_lora(*args, out=outs[0], workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    for inp, o in ((args, outs[0]), (other, outs[1])):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ql.forward_lora(*inp, out=o, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.fill_(float("nan"))
        ws.fill_(0xFF)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref2)
    del graphs


def test_refusals_of_the_binding():
    rng = np.random.default_rng(10)
    x, c, s, b, la, lb, ids, sc = _one(rng, 8, 128, 72, 2, 8)
    for bad in ((x, c, s, b, la[:, :4], lb, ids, sc), (x, c, s, b, la, lb[:1], ids, sc),
                (x, c, s, b, la.float(), lb, ids, sc), (x, c, s, b, la, lb, ids.long(), sc),
                (x, c, s, b, la, lb, ids[:4], sc), (x, c, s, b, la, lb, ids, sc[:1]),
                (x, c, s, b, la, lb.transpose(1, 2), ids, sc), (x, c, s, b, la, lb, ids.cpu(), sc)):
        with pytest.raises(ValueError):
            ql.forward_lora(*bad)
    with pytest.raises(ValueError):
        ql.forward_lora(x, c, s, b, la, lb, ids, sc, out=torch.empty((8, 72), device="cuda"))
    with pytest.raises(ql.QLinearError) as e:
        ql.forward_lora(x, c, s, b, la, lb, ids, sc, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 4
    with pytest.raises(ql.QLinearError):
        ql.forward_lora(x, c, s, b, la, lb, ids, sc, out=x.view(-1)[:8 * 72].view(8, 72))


# ------------------------------------------------------------------ the SwiGLU pair

def _pair(rng, M, K, I, n, r):
    x, gc, gs, gb = random_layer(rng, M, K, I)
    _, uc, us, ub = random_layer(rng, 1, K, I)
    ad = [_bits(v) for v in (rng.standard_normal((n, r, K)) / np.sqrt(K), 0.05 * rng.standard_normal((n, I, r)),
                             rng.standard_normal((n, r, K)) / np.sqrt(K), 0.05 * rng.standard_normal((n, I, r)))]
    return x, (gc, gs, gb), (uc, us, ub), ad, rng.uniform(0.5, 2.0, n).astype(np.float32)


def _pair_call(x, gate, up, ad, ids, scale, **kw):
    d = [to_dev_bf16(v) for v in ad]
    return ql.swiglu_lora(to_dev_bf16(x), _dev_w(gate), _dev_w(up), (d[0], d[1]), (d[2], d[3]), _dev_ids(ids),
                          torch.from_numpy(scale).cuda(), **kw)


@pytest.mark.parametrize("M,K,I,n,r,how", [
    (1, 64, 8, 1, 8, "one"), (24, 1024, 264, 6, 16, "mixed"), (191, 320, 136, 3, 24, "runs"),
    (193, 512, 264, 40, 8, "distinct"), (400, 1024, 520, 5, 64, "mixed"), (300, 256, 136, 2, 128, "runs"),
    (33, 4608, 264, 12, 32, "distinct"), (20, 320, 136, 3, 24, "mixed"), (64, 2048, 520, 9, 40, "runs"),
    (64, 576, 8, 64, 128, "distinct"),
])
def test_swiglu_lora(M, K, I, n, r, how):
    rng = np.random.default_rng(M + K + I + r)
    x, gate, up, ad, scale = _pair(rng, M, K, I, n, r)
    ids = _ids(rng, M, n, how)
    g, u = O.swiglu_linears(x, gate, up)
    g = g + O.lora_delta(x, ad[0], ad[1], scale, ids)
    u = u + O.lora_delta(x, ad[2], ad[3], scale, ids)
    h = _pair_call(x, gate, up, ad, ids, scale)
    t = O.swiglu_tolerance(O.decode_bf16(bf16_bits(h)), g, u)
    assert t["ok"], t
    h32 = _pair_call(x, gate, up, ad, ids, scale, out_dtype=torch.float32)
    t = O.swiglu_tolerance(h32.double().cpu().numpy(), g, u, bf16_output=False)
    assert t["ok"], t
    assert "swiglu_lora" in ql.last_dispatch()
    assert torch.equal(h, _pair_call(x, gate, up, ad, ids, scale))


def test_swiglu_lora_without_adapters_is_the_plain_pair():
    rng = np.random.default_rng(11)
    for M in (24, 300):
        x, gate, up, ad, scale = _pair(rng, M, 512, 264, 3, 16)
        plain = ql.swiglu(to_dev_bf16(x), _dev_w(gate), _dev_w(up), out_dtype=torch.float32)
        none = _pair_call(x, gate, up, ad, np.full(M, -1, np.int32), scale, out_dtype=torch.float32)
        # the same weights and activations through the same or another tile shape: fp32 sums in another order
        assert torch.allclose(plain, none, rtol=1e-4, atol=1e-4 * plain.abs().max().item())
        ids = _ids(rng, M, 3, "mixed")
        mixed = _pair_call(x, gate, up, ad, ids, scale, out_dtype=torch.float32)
        bare = torch.from_numpy(ids < 0).cuda()
        assert torch.equal(mixed[bare], none[bare])


@pytest.mark.parametrize("M,K,I", [(3, 4608, 264), (48, 320, 136), (260, 1024, 264)])
def test_swiglu_lora_repeats_and_replays(M, K, I):
    rng = np.random.default_rng(M + K)
    x, gate, up, ad, scale = _pair(rng, M, K, I, 4, 16)
    ids = _ids(rng, M, 4, "mixed")
    d = [to_dev_bf16(v) for v in ad]
    args = (to_dev_bf16(x), _dev_w(gate), _dev_w(up), (d[0], d[1]), (d[2], d[3]), _dev_ids(ids),
            torch.from_numpy(scale).cuda())
    ref = ql.swiglu_lora(*args)
    ws = torch.empty(ql.swiglu_lora_workspace_size(M, K, I, 4, 16), dtype=torch.uint8, device="cuda")
    for fill in (0xFF, 0x00):
        ws.fill_(fill)
        assert torch.equal(ql.swiglu_lora(*args, workspace=ws), ref)
    out = torch.empty_like(ref)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ql.swiglu_lora(*args, out=out, workspace=ws)
    for _ in range(2):
        out.fill_(float("nan"))
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    # a non-finite entry of either up projection counts as zero and is recorded
    bad = d[3].clone()
    bad[1, 5, 3] = float("inf")
    ql.swiglu_lora(*args[:4], (d[2], bad), *args[5:])
    assert ql.device_status() == (1 if (ids == 1).any() else 0)
    del g


def test_swiglu_lora_keeps_gate_and_up_apart():
    """One projection's adapter at a time, exact integers under an identity-like other half: with W_up = 0 and an up
    adapter alone, h = silu(g) * delta_u; with W_gate = 0 and a gate adapter alone, g = delta_g."""
    rng = np.random.default_rng(12)
    K, I, n, r = 128, 136, 2, 8
    for M in (30, 250):
        x = rng.integers(-2, 3, (M, K)).astype(np.float64)
        w, wv = _int_layer(rng, I, K, 4)
        zero = (np.zeros_like(w[0]), np.zeros_like(w[1]), np.zeros_like(w[2]))
        a, b = _int_adapters(rng, n, r, K, I)
        nil_a, nil_b = np.zeros_like(a), np.zeros_like(b)
        ids = _ids(rng, M, n, "mixed")
        one = np.ones(n, np.float32)
        delta = O.lora_delta(_bits(x), _bits(a), _bits(b), None, ids)
        lin = x @ wv.T / 64.0
        w64 = (w[0], w[1] / 64, w[2] / 64)
        for gate, up, ad, g, u in ((w64, zero, (nil_a, nil_b, a, b), lin, delta),
                                   (zero, w64, (a, b, nil_a, nil_b), delta, lin)):
            h = _pair_call(_bits(x), gate, up, [_bits(v) for v in ad], ids, one, out_dtype=torch.float32)
            ref = O.silu(g) * u
            # g and u are exact; silu and the product in fp32 with the hardware exponential and reciprocal: the
            # exponential's relative error is (2 + |1.16 g|) 2^-23 at most, the rest a few roundings
            bound = np.abs(ref) * (np.abs(g) * 1.2 + 16) * 2.0 ** -23 + 1e-30
            assert np.all(np.abs(h.double().cpu().numpy() - ref) <= bound)
