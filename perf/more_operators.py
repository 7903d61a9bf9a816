"""Cases of further operators beside the packed projection, for timing and comparison.

Three operators, each in its plain form (elementary torch operations in 32 bits) and as the library's call:

  product  y = residual + gate[seg] * act(x . W^T + bias)     a packed projection with bias, activation, gate and
           residual in its epilogue
  rotary   x's heads turned by positions of several axes (time, height, width): pair i of a head by
           2 pi turns[i] pos[axes[i]][m], with pairs of halves (i, i + P) or of neighbours (2i, 2i + 1)
  qk       q and k = RMS(q) w_q, RMS(k) w_k head by head, then the same rotation

`own` chooses between the two forms.  A case is a dict of plain values; prepare() makes its tensors on the GPU
from a seed, run() makes one pass, exact() gives the same outputs from the definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

GROUP = 64


# ------------------------------------------------------------------------------------------------ cases

def _product(name, M, K, N, bits=4, act=None, bias=True, gate=False, residual=False, params="bf16", segments=1,
             padding=0):
    return {"name": name, "op": "product", "M": M, "K": K, "N": N, "bits": bits, "act": act, "bias": bias, "gate": gate,
            "residual": residual, "params": params, "segments": segments, "padding": padding}


def _rotary(name, M, heads, D, sections, series="shared", turn="blocks", adjacent=False, x="bf16", layout="tokens",
            positions="int32", start=0, padding=0):
    return {"name": name, "op": "rotary", "M": M, "heads": heads, "D": D, "sections": sections, "series": series,
            "turn": turn, "adjacent": adjacent, "x": x, "layout": layout, "positions": positions, "start": start,
            "padding": padding}


def _qk(name, M, heads, kv, D, sections, params="bf16", **kw):
    case = _rotary(name, M, heads, D, sections, **kw)
    case.update({"op": "qk", "kv": kv, "params": params})
    return case


def listed():
    """The cases that are always measured; what each stands for is said beside it."""
    return [
        # one timestep's embedding through its MLP: the smallest product, latency counts
        _product("time_mlp", 1, 4608, 4608, act="silu", params="f32"),
        # the adaLN modulation vectors of a conditional and an unconditional pass of two requests, 8-bit codes
        _product("modulation_w8", 4, 512, 18432, bits=8, params="f32"),
        # the text-conditioning projection of a short prompt
        _product("text_tokens", 32, 53248, 4608),
        # patches of one 1024^2 canvas into the model: almost nothing but the output
        _product("patches_in", 4608, 128, 4608),
        # a ragged few prompts through a GELU MLP's first projection, 8-bit codes
        _product("prompts_gelu_w8", 333, 4608, 12288, bits=8, act="gelu_tanh"),
        # the attention's output projection of one canvas, gate and residual, two segments and padding behind them
        _product("attention_out", 4608, 4608, 4608, bias=False, gate=True, residual=True, segments=2, padding=37),
        # the MLP's down projection of an odd number of tokens, bias, gate and residual
        _product("mlp_down", 4609, 12288, 4608, gate=True, residual=True, params="f32", segments=3),
        # queries of one token (cross attention's, say), neighbours paired, far along the sequence
        _rotary("rotary_token", 1, 18, 256, "44-42-42", series="per_axis", adjacent=True, start=1 << 20),
        # a clip of 21 frames of 30 x 52 patches, a rotation of its own per axis, fractional positions
        _rotary("rotary_video", 32760, 24, 128, "22-21-21", series="per_axis", adjacent=True, positions="f32"),
        # queries and keys of one token out of the fused QKV projection
        _qk("qk_token", 1, 18, 18, 256, "44-42-42", turn="cycle"),
        # of one 1024^2 canvas and its prompt, half of each head turned, padding behind them
        _qk("qk_canvas", 4608, 18, 18, 256, "24-20-20", turn="cycle", padding=37),
        # two packed 2048^2 canvases, fewer key heads, written head by head for the attention
        _qk("qk_canvases", 33792, 18, 6, 256, "44-42-42", turn="cycle", layout="heads", params="f32"),
    ]


def _sections(case):
    """Pairs of each axis."""
    return [int(n) for n in case["sections"].split("-")]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["product", "product", "rotary", "qk"])
    if op == "product":
        K = GROUP * _log_int(rng, 1, 192)
        N = 8 * _log_int(rng, 8, 2304)
        M = _log_int(rng, 1, max(1, min(8192, 4609 * 12288 * 4608 // (K * N))))
        return {"op": op, "M": M, "K": K, "N": N, "bits": rng.choice([4, 4, 8]),
                "act": rng.choice([None, None, "silu", "gelu", "gelu_tanh"]), "bias": rng.random() < 0.7,
                "gate": rng.random() < 0.5, "residual": rng.random() < 0.6, "params": rng.choice(["bf16", "f32"]),
                "segments": rng.randint(1, min(6, M)), "padding": rng.choice([0, rng.randint(0, M // 16)])}
    D = rng.choice([64, 80, 96, 128, 160, 192, 256])
    pairs = D // 2 if rng.random() < 0.6 else 8 * rng.randint(1, D // 16)
    axes = rng.randint(1, min(4, pairs))
    cuts = sorted(rng.sample(range(1, pairs), axes - 1)) + [pairs]
    sections = "-".join(str(b - a) for a, b in zip([0] + cuts, cuts))
    heads = _log_int(rng, 1, 36)
    kv = rng.choice([h for h in range(1, heads + 1) if heads % h == 0])
    M = _log_int(rng, 1, min(33792, 33792 * 18 * 256 // (heads * D)))
    case = {"op": op, "M": M, "heads": heads, "D": D, "sections": sections,
            "series": rng.choice(["shared", "per_axis"]), "turn": rng.choice(["blocks", "cycle"]),
            "adjacent": rng.random() < 0.4, "x": rng.choice(["bf16", "bf16", "f32"]),
            "layout": rng.choice(["tokens", "heads"]), "positions": rng.choice(["int32", "int64", "f32"]),
            "start": rng.choice([0, _log_int(rng, 1, 1 << 20)]), "padding": rng.choice([0, rng.randint(0, M // 16)])}
    if op == "qk":
        case.update({"kv": kv, "params": rng.choice(["bf16", "f32"])})
    return case


# ------------------------------------------------------------------------------------------------ inputs

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "int32": torch.int32, "int64": torch.int64}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _packed(g, N, K, bits):
    """Uniform codes, scales spread over a factor of twenty, each bias near the middle of its group's range."""
    codes = torch.randint(-2 ** 31, 2 ** 31, (N, K * bits // 32), generator=g, device="cuda", dtype=torch.int64)
    top = 2 ** bits - 1
    s = torch.exp(torch.empty((N, K // GROUP), device="cuda").uniform_(math.log(1e-3), math.log(2e-2), generator=g))
    s = s * (15.0 / top)
    b = -0.5 * top * s + 0.1 * s * torch.randn(s.shape, generator=g, device="cuda")
    return codes.to(torch.int32), s.half(), b.half()


def _segments(M, T, padding):
    """Segment of every row in equal runs; the last `padding` rows lie behind the last sequence."""
    ids = (torch.arange(M, device="cuda") * T) // M
    ids[M - padding:] = -1
    return ids.to(torch.int32)


def _positions(case):
    """[3 or so axes][M]: a prompt along all axes at once, then the patches of a grid (fractions of it in 32 bits)."""
    M, axes = case["M"], len(_sections(case))
    prompt = M // 9
    side = max(1, math.isqrt(max(1, (M - prompt) // 2)))
    i = torch.arange(M, device="cuda")
    j = (i - prompt).clamp(min=0)
    grid = [j // (side * side), (j // side) % side, j % side, j % 7]
    pos = torch.stack([torch.where(i < prompt, i, prompt + grid[a]) for a in range(axes)]) + case["start"]
    if case["positions"] == "f32":
        return pos.float() * 0.625                     # a canvas of another size than the trained one
    return pos.to(_TYPES[case["positions"]])


def _turns(case):
    """(turns, axes): each pair's turns per unit of position and the axis whose position it takes."""
    s = _sections(case)
    P, theta = sum(s), 5e6 if case["series"] == "shared" else 1e4
    if case["turn"] == "blocks":
        axes = [a for a, n in enumerate(s) for _ in range(n)]
    else:                                              # the axes take turns, each while it has pairs left
        left, axes = list(s), []
        while len(axes) < P:
            for a in range(len(s)):
                if left[a]:
                    left[a] -= 1
                    axes.append(a)
    if case["series"] == "shared":
        rates = [theta ** (-i / P) for i in range(P)]
    else:
        seen, rates = [0] * len(s), []
        for a in axes:
            rates.append(theta ** (-seen[a] / s[a]))
            seen[a] += 1
    turns = torch.tensor([r / (2 * math.pi) for r in rates], dtype=torch.float64, device="cuda")
    return turns, torch.tensor(axes, dtype=torch.int32, device="cuda")


def _heads_out(case, heads):
    """The program's own output buffer [M][heads][D], or one kept head by head; zeros, so that rows behind the last
    sequence have a known value."""
    M, D, t = case["M"], case["D"], _TYPES[case["x"]]
    if case["layout"] == "heads":
        return torch.zeros((heads, M, D), dtype=t, device="cuda").transpose(0, 1)
    return torch.zeros((M, heads, D), dtype=t, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    op, M = case["op"], case["M"]
    if op == "product":
        K, N, T = case["K"], case["N"], case["segments"]
        pt = _TYPES[case["params"]]
        sigma = torch.exp(torch.randn(K, generator=g, device="cuda"))
        st = {"op": op, "bits": case["bits"], "act": case["act"], "w": _packed(g, N, K, case["bits"]),
              "x": (torch.randn((M, K), generator=g, device="cuda") * sigma).bfloat16()}
        st["bias"] = torch.randn(N, generator=g, device="cuda").to(pt) if case["bias"] else None
        st["gate"] = (0.5 * torch.randn((T, N), generator=g, device="cuda")).to(pt) if case["gate"] else None
        r = 3.0 * torch.randn((M, N), generator=g, device="cuda") if case["residual"] else None
        st["residual"] = r.bfloat16() if case["residual"] else None
        st["segment_ids"] = _segments(M, T, case["padding"]) if T > 1 or case["padding"] else None
        st["out"] = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
        return st
    D, heads, kv = case["D"], case["heads"], case.get("kv", 0)
    st = {"op": op, "adjacent": case["adjacent"], "rotary": _turns(case), "positions": _positions(case)}
    st["segment_ids"] = _segments(M, 1, case["padding"]) if case["padding"] else None
    packed = heads + 2 * kv                            # queries, keys and values side by side, as projected
    sigma = torch.exp(0.5 * torch.randn((packed, D), generator=g, device="cuda"))
    qkv = (2.0 * torch.randn((M, packed, D), generator=g, device="cuda") * sigma).to(_TYPES[case["x"]])
    st["x"], st["x_out"] = qkv[:, :heads], _heads_out(case, heads)
    if op == "qk":
        pt = _TYPES[case["params"]]
        st["k"], st["k_out"] = qkv[:, heads:heads + kv], _heads_out(case, kv)
        st["q_weight"] = (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(pt)
        st["k_weight"] = (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(pt)
        st["eps"] = 1e-6
    return st


# ------------------------------------------------------------------------------------------------ one pass

def _dequant32(codes, scales, biases, bits):
    per = 32 // bits
    shifts = torch.arange(per, device=codes.device, dtype=torch.int32) * bits
    q = (codes[:, :, None] >> shifts) & (2 ** bits - 1)
    q = q.reshape(codes.shape[0], -1, GROUP).float()
    w = q * scales.float()[:, :, None] + biases.float()[:, :, None]
    return w.reshape(codes.shape[0], -1)


def _act32(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 2.0 ** -0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _rotate32(v, rotary, positions, adjacent):
    """v fp32 [M][H][D]; the angles in 64 bits (positions may be far), their sines and cosines rounded to 32."""
    turns, axes = rotary
    P = turns.shape[0]
    angle = 2.0 * math.pi * (positions[axes.long()].double().t() * turns)
    c, s = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    if adjacent:
        a, b = v[..., 0:2 * P:2], v[..., 1:2 * P:2]
        turned = torch.stack((a * c - b * s, b * c + a * s), dim=-1).flatten(-2)
    else:
        a, b = v[..., :P], v[..., P:2 * P]
        turned = torch.cat((a * c - b * s, b * c + a * s), dim=-1)
    return torch.cat((turned, v[..., 2 * P:]), dim=-1)


def _live(st, v, out):
    """v where a row belongs to a sequence, what `out` held where it does not."""
    ids = st["segment_ids"]
    if ids is not None:
        v = torch.where((ids >= 0).reshape([-1] + [1] * (v.dim() - 1)), v, out.float())
    return v.to(out.dtype)


def _run_plain(st):
    if st["op"] == "product":
        z = st["x"].float() @ _dequant32(*st["w"], st["bits"]).t()
        if st["bias"] is not None:
            z = z + st["bias"].float()
        y = _act32(z, st["act"])
        if st["gate"] is not None:
            seg = st["segment_ids"]
            y = y * (st["gate"].float() if seg is None else st["gate"].float()[seg.clamp(min=0).long()])
        if st["residual"] is not None:
            y = st["residual"].float() + y
        return _live(st, y, st["out"])
    if st["op"] == "rotary":
        return _live(st, _rotate32(st["x"].float(), st["rotary"], st["positions"], st["adjacent"]), st["x_out"])
    out = []
    for v, weight, o in ((st["x"], st["q_weight"], st["x_out"]), (st["k"], st["k_weight"], st["k_out"])):
        v = v.float()
        v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + st["eps"]) * weight.float()
        out.append(_live(st, _rotate32(v, st["rotary"], st["positions"], st["adjacent"]), o))
    return out


def _run_own(st):
    import group_wise_affine_qlinear_b200 as ql
    if st["op"] == "product":
        call = ql.forward_epilogue if st["bits"] == 4 else ql.forward8_epilogue
        return call(st["x"], *st["w"], bias=st["bias"], activation=st["act"], gate=st["gate"], residual=st["residual"],
                    segment_ids=st["segment_ids"], out=st["out"])
    if st["op"] == "rotary":
        return ql.rotary_axes(st["x"], st["positions"], st["rotary"], adjacent=st["adjacent"],
                              segment_ids=st["segment_ids"], out=st["x_out"])
    return list(ql.qk_norm_rotary(st["x"], st["k"], st["positions"], st["rotary"], q_weight=st["q_weight"],
                                  k_weight=st["k_weight"], eps=st["eps"], adjacent=st["adjacent"],
                                  segment_ids=st["segment_ids"], q_out=st["x_out"], k_out=st["k_out"]))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------------------ floors

def work(case):
    """Bytes and operations that one pass cannot do without: every input once, every output once."""
    size = {"bf16": 2, "f32": 4, "int32": 4, "int64": 8}
    live = case["M"] - case["padding"]
    if case["op"] == "product":
        K, N, bits, T = case["K"], case["N"], case["bits"], case["segments"]
        vectors = (1 if case["bias"] else 0) + (T if case["gate"] else 0)
        nbytes = (2 * live * K + N * K * bits // 8 + 4 * N * (K // GROUP) + vectors * N * size[case["params"]] +
                  2 * live * N * (2 if case["residual"] else 1))
        return {"bytes": nbytes, "flops": 2 * live * N * K}
    heads, D = case["heads"] + case.get("kv", 0), case["D"]
    P, axes = sum(_sections(case)), len(_sections(case))
    nbytes = 2 * live * heads * D * size[case["x"]] + axes * live * size[case["positions"]] + 12 * P
    flops = 6 * P * live * heads
    if case["op"] == "qk":
        nbytes += 2 * D * size[case["params"]]
        flops += 4 * D * live * heads
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------------------------------------ 64 bits

def _weights64(codes, scales, biases, bits):
    """W in 64 bits from the code bytes: little-endian words, the lower nibble first."""
    raw = codes.contiguous().view(torch.uint8)
    if bits == 4:
        raw = torch.stack((raw % 16, raw // 16), dim=2).flatten(1)
    w = raw.double()
    return w * scales.double().repeat_interleave(GROUP, 1) + biases.double().repeat_interleave(GROUP, 1)


def _turned64(st, rows, v):
    """v [rows][H][D] turned pair by pair as complex numbers."""
    turns, axes = st["rotary"]
    P = len(turns)
    t = torch.stack([st["positions"][a][rows].double() * f for a, f in zip(axes.tolist(), turns.tolist())], dim=1)
    angle = 2.0 * math.pi * (t - torch.round(t))
    unit = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    head, rest = v[..., :2 * P], v[..., 2 * P:]
    if st["adjacent"]:
        pairs = torch.complex(head[..., ::2].contiguous(), head[..., 1::2].contiguous()) * unit
        return torch.cat((torch.view_as_real(pairs).reshape(head.shape), rest), -1)
    pairs = torch.complex(head[..., :P].contiguous(), head[..., P:].contiguous()) * unit
    return torch.cat((pairs.real, pairs.imag, rest), -1)


def exact(case, seed):
    st = prepare(case, seed)
    M = case["M"]
    ids = st["segment_ids"]
    rows = torch.arange(M, device="cuda") if ids is None else torch.nonzero(ids >= 0).flatten()
    if case["op"] == "product":
        y = torch.mm(st["x"][rows].double(), _weights64(*st["w"], st["bits"]).T)
        if st["bias"] is not None:
            y += st["bias"].double()
        if st["act"] == "silu":
            y = y * torch.sigmoid(y)
        elif st["act"] == "gelu":
            y = 0.5 * y * torch.special.erfc(-y / math.sqrt(2.0))
        elif st["act"] == "gelu_tanh":
            y = y * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3))
        if st["gate"] is not None:
            y *= st["gate"].double()[0 if ids is None else ids[rows].long()]
        if st["residual"] is not None:
            y += st["residual"][rows].double()
        out = torch.zeros((M, case["N"]), dtype=torch.float64, device="cuda")
        out[rows] = y
        return out
    outs = []
    for x, weight in ((st["x"], st.get("q_weight")), (st.get("k"), st.get("k_weight"))):
        if x is None:
            continue
        v = x[rows].double()
        if weight is not None:
            v = v / torch.sqrt(torch.sum(v ** 2, -1, keepdim=True) / case["D"] + st["eps"]) * weight.double()
        out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        out[rows] = _turned64(st, rows, v)
        outs.append(out)
    return outs if case["op"] == "qk" else outs[0]
