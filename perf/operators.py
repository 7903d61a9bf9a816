"""Cases of the operators that stand beside the packed projection, for timing and comparison.

Three operators, each in its plain form (elementary torch operations in 32 bits) and as the library's call:

  lora     y = x . W^T + s_a (x . A_a^T) . B_a^T   low-rank adapters of many requests beside a packed weight
  swiglu   h = silu(g) * u, with g and u two such projections of the same x (a SwiGLU pair with adapters)
  norm     r = c_x x + c_y gate * (RMS(y) w_post),  h = RMS(r) w_pre * (1 + scale) + shift
           (the norms after and before a block, its gate and the residual update between them)

`own` chooses between the two forms.  A case is a dict of plain values; prepare() makes its tensors on the GPU
from a seed, run() makes one pass, exact() gives the same outputs from the definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

GROUP = 64


# ------------------------------------------------------------------------------------------------ cases

def _lora(name, M, K, N, bits, adapters, rank, requests, bare=0, mixed=False):
    return {"name": name, "op": "lora", "M": M, "K": K, "N": N, "bits": bits, "adapters": adapters, "rank": rank,
            "requests": requests, "bare": bare, "mixed": mixed}


def _swiglu(name, M, K, I, adapters, rank, requests, bare=0, mixed=False):
    return {"name": name, "op": "swiglu", "M": M, "K": K, "I": I, "adapters": adapters, "rank": rank,
            "requests": requests, "bare": bare, "mixed": mixed}


def _norm(name, M, D, segments, x="bf16", y="bf16", partials=1, post=True, pre=True, params="bf16", padding=0):
    return {"name": name, "op": "norm", "M": M, "D": D, "segments": segments, "x": x, "y": y, "partials": partials,
            "post": post, "pre": pre, "params": params, "padding": padding}


def listed():
    """The cases that are always measured; what each stands for is said beside it."""
    return [
        # one token of one request through the fused QKV projection: the smallest call, latency counts
        _lora("lora_token", 1, 4608, 13824, 4, 4, 16, 1),
        # a batch of 32 single tokens, each of another request, 30 of them with an adapter of their own
        _lora("lora_tokens_mixed", 32, 4608, 4608, 4, 30, 16, 32, bare=2, mixed=True),
        # the long text-conditioning projection with 8-bit codes, eight prompts' last tokens, three adapters
        _lora("lora_text_w8", 8, 53248, 4608, 8, 3, 32, 8),
        # a few short prompts together, an odd number of rows, between the token and the canvas sizes
        _lora("lora_prompts", 333, 4608, 4608, 4, 5, 24, 9, bare=1),
        # the QKV projection of one 1024^2 canvas, two requests' styles in one batch
        _lora("lora_qkv", 4608, 4608, 13824, 4, 2, 16, 2),
        # ragged requests over twelve adapters of a higher rank, 8-bit codes
        _lora("lora_ragged_w8", 5021, 4608, 4608, 8, 12, 64, 24, bare=2),
        # the output projection of two packed 2048^2 canvases
        _lora("lora_canvas", 33792, 4608, 4608, 4, 2, 32, 2),
        # the MLP's gate and up projections for a few tokens of several requests
        _swiglu("swiglu_tokens", 24, 4608, 12288, 6, 16, 12, bare=1, mixed=True),
        # the same pair for one 1024^2 canvas and its prompt
        _swiglu("swiglu_mlp", 4608, 4608, 12288, 3, 32, 4, bare=1),
        # between two blocks for one token
        _norm("norm_token", 1, 4608, 1),
        # between two blocks for one 1024^2 canvas, two segments with their own modulation
        _norm("norm_canvas", 4608, 4608, 2, padding=37),
        # after a row-parallel projection on two ranks, 2048^2 canvases, residual stream in 32 bits
        _norm("norm_partials", 33792, 4608, 2, x="f32", y="f32", partials=2, params="f32"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["lora", "lora", "swiglu", "norm"])
    if op == "norm":
        D = 8 * _log_int(rng, 8, 2304)
        M = _log_int(rng, 1, min(33792, 33792 * 4608 // D))
        kind = rng.choice(["both", "pre", "post", "partials"])
        return {"op": "norm", "M": M, "D": D, "segments": rng.randint(1, min(8, M)),
                "x": rng.choice(["bf16", "f32"]), "y": "none" if kind == "pre" else
                ("f32" if kind == "partials" else "bf16"), "partials": rng.randint(1, 4) if kind == "partials" else 1,
                "post": kind != "pre" and rng.random() < 0.8, "pre": kind != "post",
                "params": rng.choice(["bf16", "f32"]), "padding": rng.randint(0, M // 16)}
    adapters = _log_int(rng, 1, 32)
    rank = 8 * rng.choice([1, 1, 2, 2, 3, 4, 5, 8])
    K = GROUP * _log_int(rng, 1, 160)
    if op == "lora":
        N = 8 * _log_int(rng, 8, 1728)
        M = _log_int(rng, 1, min(8192, 33792 * 4608 * 4608 // (4 * K * N)))
        case = {"op": "lora", "M": M, "K": K, "N": N, "bits": rng.choice([4, 4, 8])}
    else:
        I = 8 * _log_int(rng, 8, 1536)
        M = _log_int(rng, 1, min(4608, 4608 * 4608 * 12288 // (K * I)))
        case = {"op": "swiglu", "M": M, "K": K, "I": I}
    requests = _log_int(rng, 1, min(M, 48))
    case.update({"adapters": adapters, "rank": rank, "requests": requests,
                 "bare": rng.randint(0, 2) if requests > 2 else 0, "mixed": M <= 256 and rng.random() < 0.5})
    return case


# ------------------------------------------------------------------------------------------------ inputs

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


def _activations(g, M, K):
    sigma = torch.exp(torch.randn(K, generator=g, device="cuda"))
    return (torch.randn((M, K), generator=g, device="cuda") * sigma).bfloat16()


def _adapters(g, L, r, K, N):
    a = torch.randn((L, r, K), generator=g, device="cuda") / math.sqrt(K)
    b = 0.02 * torch.randn((L, N, r), generator=g, device="cuda")
    return a.bfloat16(), b.bfloat16()


def _row_ids(case, g):
    """Adapter of every row: ragged runs of rows, one per request, the last `bare` requests without an adapter."""
    M, n, L = case["M"], case["requests"], case["adapters"]
    cuts = torch.randperm(M - 1, generator=g, device="cuda")[:n - 1] + 1 if n > 1 else torch.empty(0, device="cuda")
    owner = torch.zeros(M, dtype=torch.int64, device="cuda")
    if n > 1:
        owner[cuts] = 1
    owner = torch.cumsum(owner, 0)
    which = torch.randperm(L, generator=g, device="cuda")[torch.arange(n, device="cuda") % L]
    which = torch.where(torch.arange(n, device="cuda") < n - case["bare"], which, torch.full_like(which, -1))
    ids = which[owner]
    if case["mixed"]:                                  # tokens of the requests in no order
        ids = ids[torch.randperm(M, generator=g, device="cuda")]
    return ids.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "norm":
        M, D, T = case["M"], case["D"], case["segments"]
        pt = torch.bfloat16 if case["params"] == "bf16" else torch.float32
        sigma = torch.exp(0.5 * torch.randn(D, generator=g, device="cuda"))
        x = 3.0 * torch.randn((M, D), generator=g, device="cuda") * sigma
        st = {"op": op, "x": x.bfloat16() if case["x"] == "bf16" else x, "y": None}
        if case["y"] == "bf16":
            st["y"] = (torch.randn((M, D), generator=g, device="cuda") * sigma).bfloat16()
        elif case["y"] == "f32":
            st["y"] = torch.randn((case["partials"], M, D), generator=g, device="cuda")

        def vec(rows, mean, std):
            return (mean + std * torch.randn((rows, D), generator=g, device="cuda")).to(pt)
        st["post_norm"], st["pre_norm"] = case["post"], case["pre"]
        st["post_weight"] = vec(1, 1.0, 0.2)[0] if case["post"] else None
        st["gate"] = vec(T, 0.0, 0.5) if st["y"] is not None else None
        st["pre_weight"] = vec(1, 1.0, 0.2)[0] if case["pre"] else None
        st["scale"] = vec(T, 0.0, 0.2) if case["pre"] else None
        st["shift"] = vec(T, 0.0, 0.2) if case["pre"] else None
        ids = (torch.arange(M, device="cuda") * T) // M
        ids[M - case["padding"]:] = -1                 # rows behind the last sequence
        st["segment_ids"] = ids.to(torch.int32)
        st["residual_scale"], st["branch_scale"], st["eps"] = 1.0, 0.5, 1e-5
        # outputs are the program's own buffers, so that rows behind the last sequence have a known value
        st["r"] = torch.zeros_like(st["x"]) if st["y"] is not None else None
        st["h"] = torch.zeros((M, D), dtype=torch.bfloat16, device="cuda") if case["pre"] else None
        return st
    M, K, L, r = case["M"], case["K"], case["adapters"], case["rank"]
    st = {"op": op, "x": _activations(g, M, K), "ids": _row_ids(case, g),
          "lora_scale": torch.empty(L, device="cuda").uniform_(0.5, 2.0, generator=g)}
    if op == "lora":
        st["bits"] = case["bits"]
        st["w"] = _packed(g, case["N"], K, case["bits"])
        st["a"], st["b"] = _adapters(g, L, r, K, case["N"])
    else:
        st["gate"], st["up"] = _packed(g, case["I"], K, 4), _packed(g, case["I"], K, 4)
        st["gate_lora"], st["up_lora"] = _adapters(g, L, r, K, case["I"]), _adapters(g, L, r, K, case["I"])
    return st


# ------------------------------------------------------------------------------------------------ one pass

def _dequant32(codes, scales, biases, bits):
    per = 32 // bits
    shifts = torch.arange(per, device=codes.device, dtype=torch.int32) * bits
    q = (codes[:, :, None] >> shifts) & (2 ** bits - 1)
    q = q.reshape(codes.shape[0], -1, GROUP).float()
    w = q * scales.float()[:, :, None] + biases.float()[:, :, None]
    return w.reshape(codes.shape[0], -1)


def _project32(x, w, bits, a, b, ids, lora_scale):
    """x . W^T plus every row's adapter, all in 32 bits (all adapters at once, masked to each row's own)."""
    L, r, K = a.shape
    y = x @ _dequant32(*w, bits).t()
    t = (x @ a.float().reshape(L * r, K).t()).reshape(-1, L, r)
    pick = ids[:, None] == torch.arange(L, device=ids.device, dtype=ids.dtype)
    t = torch.where(pick[:, :, None], t * lora_scale[None, :, None], torch.zeros((), device=t.device))
    return y + t.reshape(-1, L * r) @ b.float().permute(0, 2, 1).reshape(L * r, -1)


def _run_plain(st):
    if st["op"] == "lora":
        y = _project32(st["x"].float(), st["w"], st["bits"], st["a"], st["b"], st["ids"], st["lora_scale"])
        return y.bfloat16()
    if st["op"] == "swiglu":
        x = st["x"].float()
        g = _project32(x, st["gate"], 4, *st["gate_lora"], st["ids"], st["lora_scale"])
        u = _project32(x, st["up"], 4, *st["up_lora"], st["ids"], st["lora_scale"])
        return (g / (1.0 + torch.exp(-g)) * u).bfloat16()
    ids = st["segment_ids"]
    live = (ids >= 0)[:, None]
    seg = ids.clamp(min=0).long()
    r = st["x"].float()
    out = []
    if st["y"] is not None:
        v = st["y"].float()
        if v.dim() == 3:
            v = v.sum(0)
        if st["post_norm"]:
            v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + st["eps"]) * st["post_weight"].float()
        r = st["residual_scale"] * r + st["branch_scale"] * st["gate"].float()[seg] * v
        out.append(torch.where(live, r, st["r"].float()).to(st["x"].dtype))
    if st["pre_norm"]:
        h = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + st["eps"]) * st["pre_weight"].float()
        h = h * (1.0 + st["scale"].float()[seg]) + st["shift"].float()[seg]
        out.append(torch.where(live, h, st["h"].float()).bfloat16())
    return out


def _run_own(st):
    import group_wise_affine_qlinear_b200 as ql
    if st["op"] == "lora":
        call = ql.forward_lora if st["bits"] == 4 else ql.forward8_lora
        return call(st["x"], *st["w"], st["a"], st["b"], st["ids"], st["lora_scale"])
    if st["op"] == "swiglu":
        return ql.swiglu_lora(st["x"], st["gate"], st["up"], st["gate_lora"], st["up_lora"], st["ids"],
                              st["lora_scale"])
    r, h = ql.norm_residual(st["x"], st["y"], post_norm=st["post_norm"], post_weight=st["post_weight"],
                            gate=st["gate"], residual_scale=st["residual_scale"], branch_scale=st["branch_scale"],
                            pre_norm=st["pre_norm"], pre_weight=st["pre_weight"], scale=st["scale"],
                            shift=st["shift"], segment_ids=st["segment_ids"], eps=st["eps"], out=st["r"], h=st["h"])
    return ([r] if st["y"] is not None else []) + ([h] if st["pre_norm"] else [])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------------------ floors

def work(case):
    """Bytes and operations that one pass cannot do without: every input once, every output once."""
    if case["op"] == "norm":
        M, D, T = case["M"] - case["padding"], case["D"], case["segments"]
        xb, pb = (2 if case["x"] == "bf16" else 4), (2 if case["params"] == "bf16" else 4)
        yb = {"none": 0, "bf16": 2, "f32": 4 * case["partials"]}[case["y"]]
        r_out = xb if case["y"] != "none" else 0
        per = xb + yb + r_out + (2 if case["pre"] else 0)
        vectors = (1 if case["post"] else 0) + (T if case["y"] != "none" else 0) + ((1 + 2 * T) if case["pre"] else 0)
        return {"bytes": M * D * per + vectors * D * pb + 4 * case["M"], "flops": 14 * M * D}
    M, K, r, L = case["M"], case["K"], case["rank"], case["adapters"]
    with_adapter = case["requests"] - case["bare"]
    used = min(L, with_adapter)
    rows = M * with_adapter // case["requests"]        # rows with an adapter, as the requests' lengths average
    if case["op"] == "lora":
        weights = [(case["N"], case["bits"])]
    else:
        weights = [(case["I"], 4), (case["I"], 4)]
    n_out = weights[0][0]
    nbytes = 2 * M * K + 2 * M * n_out + 4 * M + 4 * L
    flops = 0
    for N, bits in weights:
        nbytes += N * K * bits // 8 + 4 * N * (K // GROUP) + 2 * used * r * (K + N)
        flops += 2 * M * N * K + 2 * rows * r * (K + N)
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------------------------------------ 64 bits

def _weights64(codes, scales, biases, bits):
    """W in 64 bits from the code bytes: little-endian words, the lower nibble first."""
    raw = codes.contiguous().view(torch.uint8)
    if bits == 4:
        raw = torch.stack((raw % 16, raw // 16), dim=2).flatten(1)
    w = raw.double()
    return w * scales.double().repeat_interleave(GROUP, 1) + biases.double().repeat_interleave(GROUP, 1)


def _linear64(x, w, bits, a, b, ids, lora_scale):
    y = torch.mm(x.double(), _weights64(*w, bits).T)
    for i in sorted(set(ids.tolist())):
        if i < 0:
            continue
        rows = torch.nonzero(ids == i).flatten()
        low = torch.mm(x[rows].double(), a[i].double().T) * lora_scale[i].double()
        y[rows] += torch.mm(low, b[i].double().T)
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "lora":
        return _linear64(st["x"], st["w"], st["bits"], st["a"], st["b"], st["ids"], st["lora_scale"])
    if case["op"] == "swiglu":
        g = _linear64(st["x"], st["gate"], 4, *st["gate_lora"], st["ids"], st["lora_scale"])
        g = g * torch.sigmoid(g)
        return g.mul_(_linear64(st["x"], st["up"], 4, *st["up_lora"], st["ids"], st["lora_scale"]))
    M, D = st["x"].shape
    r_out = torch.zeros((M, D), dtype=torch.float64, device="cuda") if st["y"] is not None else None
    h_out = torch.zeros((M, D), dtype=torch.float64, device="cuda") if st["pre_norm"] else None

    def normed(v):
        return v / torch.sqrt(torch.sum(v ** 2, 1, keepdim=True) / D + st["eps"])
    for seg in range(case["segments"]):
        rows = torch.nonzero(st["segment_ids"] == seg).flatten()
        v = st["x"][rows].double()
        if r_out is not None:
            y = st["y"][rows].double() if st["y"].dim() == 2 else sum(p[rows].double() for p in st["y"])
            if st["post_norm"]:
                y = normed(y) * st["post_weight"].double()
            v = v * st["residual_scale"] + y * st["gate"][seg].double() * st["branch_scale"]
            r_out[rows] = v
        if h_out is not None:
            n = normed(v) * st["pre_weight"].double()
            h_out[rows] = n + n * st["scale"][seg].double() + st["shift"][seg].double()
    return [o for o in (r_out, h_out) if o is not None]
