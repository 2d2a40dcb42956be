"""Cases that measure the norm in front of the layer and the layer's experts in
8 and 4 bits: their plain forms in elementary torch operations, and the calls
that a program makes of this framework.

Blocks of 32 values along the last axis share a power-of-two scale, held as a
byte s that stands for 2^(s - 127).  Elements are e4m3 (one byte, largest 448)
or e2m1 (four bits, largest 6; element 2i in the low half of byte i).  Scale
rows are padded to a multiple of four bytes.
"""
import math

import torch

own = False

EPS = 1e-6
BF16, F32 = "bf16", "f32"
DTYPE = {BF16: torch.bfloat16, F32: torch.float32}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one new token on its way into the layer: the residual's addition, the
        # norm for the router and its 8-bit rows for the experts
        {"name": "norm_token", "op": "norm", "T": 1, "d": 2048, "act": BF16, "res": True,
         "quant": True},
        # the same for a long prompt (the mid-size layer's tokens)
        {"name": "norm_prompt", "op": "norm", "T": 16384, "d": 2048, "act": BF16, "res": True,
         "quant": True},
        # forward and backward of the norm in an fp32 layer, odd sizes
        {"name": "norm_train_odd_f32", "op": "train", "T": 1999, "d": 320, "act": F32,
         "res": False},
        # forward and backward of the norm in the mid-size layer's training step
        {"name": "norm_train", "op": "train", "T": 16384, "d": 2048, "act": BF16, "res": True},
        # one weight tensor of the mid-size layer to 4 bits, and read back
        {"name": "weights_e2m1", "op": "mx", "rows": 65536, "d": 2048, "act": BF16,
         "fmt": "e2m1"},
        # fp32 rows of the tiny layer to 8 bits, and read back
        {"name": "rows_e4m3_f32", "op": "mx", "rows": 2048, "d": 256, "act": F32, "fmt": "e4m3"},
        # decoding one sequence through the mid-size layer's 4-bit experts
        {"name": "token_1", "op": "token", "T": 1, "d": 2048, "E": 64, "f": 1024, "k": 6,
         "act": BF16},
        # decoding sixteen sequences together
        {"name": "token_16", "op": "token", "T": 16, "d": 2048, "E": 64, "f": 1024, "k": 6,
         "act": BF16},
        # a few tokens through the tiny fp32 layer
        {"name": "token_odd_f32", "op": "token", "T": 7, "d": 256, "E": 8, "f": 256, "k": 2,
         "act": F32},
        # a long prompt through the mid-size layer's experts
        {"name": "experts_prompt", "op": "experts", "T": 16384, "d": 2048, "E": 64, "f": 1024,
         "k": 6},
        # a short prompt: few rows for each expert, some with none
        {"name": "experts_short", "op": "experts", "T": 512, "d": 2048, "E": 64, "f": 1024,
         "k": 2},
        # odd sizes
        {"name": "experts_odd", "op": "experts", "T": 777, "d": 320, "E": 16, "f": 192, "k": 4},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, hi):
    return 64 * _log(rng, 1, hi // 64)


def draw(rng):
    op = rng.choice(["norm", "train", "mx", "token", "experts"])
    act = rng.choice([BF16, BF16, F32])
    if op in ("norm", "train"):
        d = _width(rng, 4096)
        T = _log(rng, 1, 16384)
        if act == F32 or d > 2048:
            T = min(T, 16384 * 2048 // (2 * d))
        case = {"op": op, "T": T, "d": d, "act": act, "res": rng.random() < 0.7}
        if op == "norm":
            case["quant"] = rng.random() < 0.7
        return case
    if op == "mx":
        d = _width(rng, 4096)
        return {"op": op, "rows": min(_log(rng, 1, 65536), 65536 * 1024 // d), "d": d,
                "act": act, "fmt": rng.choice(["e4m3", "e2m1"])}
    E = rng.choice([4, 8, 16, 23, 32, 64])
    k = rng.randint(1, min(E, 8))
    d, f = _width(rng, 2048), _width(rng, 1024)
    if op == "token":
        return {"op": op, "T": _log(rng, 1, 16), "d": d, "E": E, "f": f, "k": min(k, 6),
                "act": act}
    return {"op": op, "T": _log(rng, 1, 16384), "d": d, "E": E, "f": f, "k": min(k, 6)}


def _scale_cols(n):
    return 4 * ((n + 127) // 128)


def work(case):
    op, d = case["op"], case["d"]
    size = 2 if case.get("act", BF16) == BF16 else 4
    if op in ("norm", "train"):
        n = case["T"] * d
        moved = n * size * (4 if case["res"] else 2) + 4 * d   # x, y; the residual and the sum
        if op == "norm":
            moved += n * 33 / 32 if case["quant"] else 0
            return {"bytes": moved, "flops": 6 * n}
        # dy, the gradient that the residual carries, dx; the weight's gradient
        moved += n * size * (3 if case["res"] else 2) + 4 * d
        return {"bytes": moved, "flops": 16 * n}
    if op == "mx":
        n = case["rows"] * d
        held = n * ((1 if case["fmt"] == "e4m3" else 0.5) + 1 / 32)
        return {"bytes": 2 * (n * size + held), "flops": 4 * n}
    E, f, T, k = case["E"], case["f"], case["T"], case["k"]
    R = T * k
    experts = E * (1 - (1 - k / E) ** T)   # that some token chose, on average
    weights = experts * 3 * d * f * 17 / 32
    if op == "token":
        return {"bytes": weights + 2 * T * d * size + R * 8, "flops": 6 * R * d * f}
    return {"bytes": weights + T * d * 33 / 32 + R * (4 + 2 * f * 33 / 32 + 2 * d),
            "flops": 6 * R * d * f}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, d = case["op"], case["d"]
    act = DTYPE[case.get("act", BF16)]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def new(*shape, dtype=act):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    s = {"case": dict(case), "scratch": new(1 << 26, dtype=torch.uint8)}
    if op in ("norm", "train"):
        T = case["T"]
        s["x"] = normal(T, d).to(act)
        s["res"] = (2.0 * normal(T, d)).to(act) if case["res"] else None
        s["weight"] = 1.0 + 0.1 * normal(d)
        s["sum"] = new(T, d) if case["res"] else None
        s["y"] = new(T, d)
        if op == "norm":
            s["q"] = new(T, d, dtype=torch.float8_e4m3fn) if case["quant"] else None
            s["q_scale"] = new(T, _scale_cols(d), dtype=torch.uint8) if case["quant"] else None
        else:
            s["rstd"] = new(T, dtype=torch.float32)
            s["dy"] = normal(T, d).to(act)
            s["dsum"] = normal(T, d).to(act) if case["res"] else None
            s["dx"] = new(T, d)
            s["dweight"] = new(d, dtype=torch.float32)
        return s
    if op == "mx":
        rows, bits = case["rows"], 8 if case["fmt"] == "e4m3" else 4
        s["src"] = (normal(rows, d) * d ** -0.5).to(act)
        s["q"] = new(rows, d * bits // 8, dtype=torch.uint8)
        s["scale"] = new(rows, _scale_cols(d), dtype=torch.uint8)
        s["values"] = new(rows, d)
        return s
    T, E, f, k = case["T"], case["E"], case["f"], case["k"]
    for name, n, width in (("w1", f, d), ("w3", f, d), ("w2", d, f)):
        codes, scale = _to_blocks(normal(E, n, width) * width ** -0.5, "e2m1")
        s[name] = codes[..., 0::2] | (codes[..., 1::2] << 4)
        s[name + "_scale"] = scale
    # some experts are liked more than others
    logits = normal(T, E) + 0.5 * normal(E)
    chosen, s["topk_idx"] = logits.topk(k, dim=1)
    s["topk_idx"] = s["topk_idx"].to(torch.int32).contiguous()
    s["topk_gate"] = torch.softmax(chosen, 1).contiguous()
    x = normal(T, d)
    if op == "token":
        s["x"] = x.to(act)
        s["y"] = new(T, d)
        return s
    s["x"], s["x_scale"] = _to_blocks(x, "e4m3")
    # the plan: each expert's rows together, tokens ascending
    ids = s["topk_idx"].reshape(-1).long()
    order = torch.sort(ids, stable=True).indices
    counts = torch.bincount(ids, minlength=E)
    s["src_token"] = (order // k).to(torch.int32)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["most"] = int(counts.max())   # rows of the fullest expert
    s["hq"] = new(T * k, f, dtype=torch.float8_e4m3fn)
    s["h_scale"] = new(T * k, _scale_cols(f), dtype=torch.uint8)
    s["y_perm"] = new(T * k, d)
    return s


# ---------------------------------------------------------------- plain forms

def _power(code):
    """2^(code - 127) of scale bytes, exactly."""
    c = code.to(torch.int32)
    return torch.where(c > 0, c << 23, torch.full_like(c, 1 << 22)).view(torch.float32)


def _to_blocks(v, fmt):
    """Elements (e4m3 as a tensor of that type, e2m1 as one code per value) and
    the padded scale bytes of v, an fp32 tensor."""
    blocks = v.unflatten(-1, (-1, 32))
    bits = blocks.abs().amax(-1).view(torch.int32)
    # smallest power of two p with amax <= 448 p, or 6 p: by exponent and fraction
    over, top = (0x1FFFFF, 8) if fmt == "e4m3" else (0x3FFFFF, 2)
    code = (((bits + over) >> 23) - top).clamp_min(0)
    scaled = blocks * ((254 - code) << 23).view(torch.float32).unsqueeze(-1)
    if fmt == "e4m3":
        q = scaled.to(torch.float8_e4m3fn)
    else:
        a = scaled.abs()
        q = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
             + (a >= 3.5) + (a > 5.0))
        q = (q | ((scaled < 0).to(torch.uint8) << 3)).to(torch.uint8)
    scale = code.to(torch.uint8)
    pad = _scale_cols(v.shape[-1]) - scale.shape[-1]
    return q.flatten(-2), torch.nn.functional.pad(scale, (0, pad)).contiguous()


def _values(q, scale):
    """fp32 values of e4m3 elements, or of e2m1 bytes (two to a byte)."""
    if q.dtype == torch.uint8:
        table = torch.tensor(E2M1 + [-x for x in E2M1], device=q.device)
        v = table[torch.stack([q & 15, q >> 4], -1).flatten(-2).int()]
    else:
        v = q.float()
    n = v.shape[-1] // 32
    return (v.unflatten(-1, (n, 32)) * _power(scale[..., :n]).unsqueeze(-1)).flatten(-2)


def _norm(s):
    total = s["x"].float()
    if s["res"] is not None:
        total = (total + s["res"].float()).to(s["x"].dtype).float()
    rstd = torch.rsqrt((total * total).mean(-1, keepdim=True) + EPS)
    return total, rstd, total * rstd * s["weight"]


def _swiglu(a, b):
    return a / (1.0 + torch.exp(-a)) * b


def _run_plain(s):
    case = s["case"]
    op, act = case["op"], DTYPE[case.get("act", BF16)]
    if op == "norm":
        total, _, y = _norm(s)
        out = {"y": y.to(act), "sum": total.to(act) if s["res"] is not None else None}
        if case["quant"]:
            out["q"], scale = _to_blocks(y, "e4m3")
            out["q_scale"] = scale[:, :case["d"] // 32].view(torch.float8_e8m0fnu)
        return out
    if op == "train":
        total, rstd, y = _norm(s)
        n, dy = total * rstd, s["dy"].float()
        gw = dy * s["weight"]
        dx = rstd * (gw - n * (gw * n).mean(-1, keepdim=True))
        if s["dsum"] is not None:
            dx = dx + s["dsum"].float()
        return {"y": y.to(act), "sum": total.to(act) if s["res"] is not None else None,
                "dx": dx.to(act), "dweight": (dy * n).sum(0)}
    if op == "mx":
        q, scale = _to_blocks(s["src"].float(), case["fmt"])
        if case["fmt"] == "e2m1":
            q = q[:, 0::2] | (q[:, 1::2] << 4)
        return _values(q, scale).to(act)
    if op == "token":
        T, E, k = case["T"], case["E"], case["k"]
        ids, x = s["topk_idx"].long(), s["x"].float()
        if T * k < E:   # the chosen experts' weights, one set for each choice
            pick = ids.reshape(-1)
            w1, w3, w2 = (_values(s[n][pick], s[n + "_scale"][pick]) for n in ("w1", "w3", "w2"))
            rows = x.repeat_interleave(k, 0).unsqueeze(-1)
            h = _swiglu(torch.bmm(w1, rows), torch.bmm(w3, rows))
            y = torch.bmm(w2, h).reshape(T, k, -1)
            return (y * s["topk_gate"].unsqueeze(-1)).sum(1).to(act)
        # every expert on every token, weighted by its gate there
        w1, w3, w2 = (_values(s[n], s[n + "_scale"]) for n in ("w1", "w3", "w2"))
        xe = x.expand(E, -1, -1)
        h = _swiglu(torch.bmm(xe, w1.transpose(1, 2)), torch.bmm(xe, w3.transpose(1, 2)))
        gate = torch.zeros(T, E, device=x.device).scatter_(1, ids, s["topk_gate"])
        y = torch.bmm(h, w2.transpose(1, 2))
        return (y * gate.t().unsqueeze(-1)).sum(0).to(act)
    # each expert's rows side by side, padded to the fullest expert's count
    E, most, offsets = case["E"], s["most"], s["offsets"].long()
    place = offsets[:-1, None] + torch.arange(most, device=offsets.device)
    there = place < offsets[1:, None]
    place = place.clamp_max(case["T"] * case["k"] - 1)
    x = _values(s["x"], s["x_scale"])[s["src_token"].long()[place]]
    w1, w3, w2 = (_values(s[n], s[n + "_scale"]) for n in ("w1", "w3", "w2"))
    h = _swiglu(torch.bmm(x, w1.transpose(1, 2)), torch.bmm(x, w3.transpose(1, 2)))
    y = torch.bmm(_values(*_to_blocks(h, "e4m3")), w2.transpose(1, 2))
    return y[there].to(act)


# ---------------------------------------------------------------- the framework's calls

def _run_own(s):
    import top_routing_grouped_router_amd as M
    case = s["case"]
    op, d = case["op"], case["d"]
    if op == "norm":
        dims = M.make_dims(case["T"], d, 1, 64, 1, s["x"].dtype)
        M.moe_rmsnorm(dims, s["x"], s["res"], s["weight"], EPS, s["sum"], s["y"], s["q"],
                      s["q_scale"], None)
        out = {"y": s["y"], "sum": s["sum"]}
        if case["quant"]:
            out["q"] = s["q"]
            out["q_scale"] = s["q_scale"][:, :d // 32].view(torch.float8_e8m0fnu)
        return out
    if op == "train":
        dims = M.make_dims(case["T"], d, 1, 64, 1, s["x"].dtype)
        M.moe_rmsnorm(dims, s["x"], s["res"], s["weight"], EPS, s["sum"], s["y"], None, None,
                      s["rstd"])
        M.moe_rmsnorm_bwd(dims, s["dy"], s["x"] if s["res"] is None else s["sum"], s["weight"],
                          s["rstd"], s["dsum"], s["dx"], s["dweight"], s["scratch"])
        return {"y": s["y"], "sum": s["sum"], "dx": s["dx"], "dweight": s["dweight"]}
    if op == "mx":
        M.moe_mx_quantize(s["src"], case["fmt"], s["q"], s["scale"])
        M.moe_mx_dequantize(s["q"], s["scale"], case["fmt"], s["values"])
        return s["values"]
    weights = (s["w1"], s["w1_scale"], s["w3"], s["w3_scale"])
    if op == "token":
        dims = M.make_dims(case["T"], d, case["E"], case["f"], case["k"], s["x"].dtype)
        M.moe_token_swiglu(dims, s["x"], s["topk_idx"], s["topk_gate"], *weights, s["w2"],
                           s["w2_scale"], s["y"], s["scratch"])
        return s["y"]
    dims = M.make_dims(case["T"], d, case["E"], case["f"], case["k"], s["y_perm"].dtype)
    M.moe_expert_up_mx(dims, s["x"], s["x_scale"], s["src_token"], s["offsets"], *weights,
                       s["hq"], s["h_scale"])
    M.moe_expert_down_mx(dims, s["hq"], s["h_scale"], s["offsets"], s["w2"], s["w2_scale"],
                         s["y_perm"])
    return s["y_perm"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_blocks(v, fmt):
    """Element values and scales of v (64 bits) by the definition: the smallest
    power of two that leaves nothing above the format's largest value, then
    rounding to the nearest element, ties to the even one."""
    n = v.shape[-1]
    blocks = v.reshape(*v.shape[:-1], n // 32, 32)
    largest, low, fraction = (448.0, -6, 3) if fmt == "e4m3" else (6.0, 0, 1)
    m, e = torch.frexp(blocks.abs().amax(-1) / largest)
    e = torch.where(m > 0.5, e, e - 1).clamp_min(-127)
    scale = torch.ldexp(torch.ones_like(m), e)
    u = blocks / scale.unsqueeze(-1)
    _, ue = torch.frexp(u)
    step = torch.ldexp(torch.ones_like(u), (ue - 1).clamp_min(low) - fraction)
    return (torch.round(u / step) * step).reshape(v.shape), scale


def _exact_values(q, scale):
    n = scale.shape[-1]
    if q.dtype == torch.uint8:
        code = torch.empty(*q.shape, 2, dtype=torch.int64, device=q.device)
        code[..., 0], code[..., 1] = q % 16, q // 16
        code = code.reshape(*q.shape[:-1], -1)
        exponent, half = (code // 2) % 4, (code % 2).double()
        size = torch.where(exponent == 0, half / 2,
                           (1 + half / 2) * torch.pow(2.0, (exponent - 1).double()))
        v = torch.where(code >= 8, -size, size)
    else:
        v = q.double()
    n = v.shape[-1] // 32
    power = torch.ldexp(torch.ones((), dtype=torch.float64, device=v.device),
                        scale[..., :n].int() - 127)
    return v * power.repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "mx":
        v, scale = _exact_blocks(s["src"].double(), case["fmt"])
        return v * scale.repeat_interleave(32, -1)
    if op in ("norm", "train"):
        total = s["x"].double()
        if s["res"] is not None:
            total = (total + s["res"].double()).to(s["x"].dtype).double()
        spread = (total.square().sum(-1, keepdim=True) / case["d"] + EPS).sqrt()
        y = total / spread * s["weight"].double()
        out = {"y": y, "sum": total if s["res"] is not None else None}
        if op == "norm":
            if case["quant"]:
                out["q"], out["q_scale"] = _exact_blocks(y, "e4m3")
            return out
        n, dy = total / spread, s["dy"].double()
        gw = dy * s["weight"].double()
        dx = (gw - n * ((gw * n).sum(-1, keepdim=True) / case["d"])) / spread
        out["dx"] = dx if s["dsum"] is None else dx + s["dsum"].double()
        out["dweight"] = torch.einsum("td,td->d", dy, n)
        return out

    def expert(e, rows, quant):
        w1, w3, w2 = (_exact_values(s[n][e], s[n + "_scale"][e]) for n in ("w1", "w3", "w2"))
        a = rows @ w1.t()
        h = a * torch.sigmoid(a) * (rows @ w3.t())
        if quant:
            v, scale = _exact_blocks(h, "e4m3")
            h = v * scale.repeat_interleave(32, -1)
        return h @ w2.t()

    if op == "token":
        y = torch.zeros(case["T"], case["d"], dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            t, j = torch.nonzero(s["topk_idx"] == e, as_tuple=True)
            if t.numel():
                rows = expert(e, s["x"][t].double(), False)
                y[t] += rows * s["topk_gate"][t, j].double().unsqueeze(-1)
        return y
    x = _exact_values(s["x"], s["x_scale"])
    y = torch.zeros(case["T"] * case["k"], case["d"], dtype=torch.float64, device="cuda")
    ends = s["offsets"].tolist()
    for e in range(case["E"]):
        if ends[e] < ends[e + 1]:
            tokens = s["src_token"][ends[e]:ends[e + 1]].long()
            y[ends[e]:ends[e + 1]] = expert(e, x[tokens], True)
    return y
