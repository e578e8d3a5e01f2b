"""Cases of the operators around the projections, each in a plain form and through the library.

Three families: products with 4-bit weights and group scales (one matrix, or a stack of experts), tokens
sorted by expert and back with their weights (forward and gradient), and the norms after and before a block
with its gate and residual scale (forward and gradient).
"""
import math

import torch

own = False

F32 = torch.float32
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # The smallest call: one decode token through the o projection's shape.
        {"name": "w4 o, 1 token", "op": "w4", "m": 1, "N": 8192, "K": 1024, "group": 128, "zeros": False, "dtype": "bf16"},
        # A verify step of 8 tokens on the pooler's shape, asymmetric codes.
        {"name": "w4 pooler, 8 tokens", "op": "w4", "m": 8, "N": 4096, "K": 8192, "group": 64, "zeros": True, "dtype": "fp16"},
        # Odd everything: rows and columns that end inside tiles and groups, an odd batch.
        {"name": "w4 odd sizes, 33 tokens", "op": "w4", "m": 33, "N": 2305, "K": 8103, "group": 32, "zeros": True, "dtype": "bf16"},
        # The widest verify load on the unpooler's shape.
        {"name": "w4 unpooler, 256 tokens", "op": "w4", "m": 256, "N": 8192, "K": 4096, "group": 128, "zeros": False, "dtype": "bf16"},
        # Experts' up product in a decode step of 8 tokens: most experts have no row, the others one or two.
        {"name": "experts up, 8 tokens", "op": "experts", "tokens": 8, "k": 8, "E": 256, "N": 1024, "K": 8192, "group": 128,
         "zeros": False, "dtype": "bf16", "skew": 0.0},
        # Experts' down product of 1000 tokens with crowded and idle experts.
        {"name": "experts down, 1000 tokens", "op": "experts", "tokens": 1000, "k": 8, "E": 256, "N": 8192, "K": 512, "group": 32,
         "zeros": True, "dtype": "fp16", "skew": 1.0},
        # One decode token to its experts and back: latency.
        {"name": "moe forward, 1 token", "op": "moe_forward", "m": 1, "E": 256, "k": 8, "D": 8192, "mode": 0, "masked": False,
         "dtype": "bf16"},
        # A prompt chunk, with padding tokens and experts that are switched off.
        {"name": "moe forward, 4096 tokens", "op": "moe_forward", "m": 4096, "E": 256, "k": 8, "D": 8192, "mode": 1, "masked": True,
         "dtype": "bf16"},
        # Gradient of the same path on an odd batch and an odd width.
        {"name": "moe backward, 1000 tokens", "op": "moe_backward", "m": 1000, "E": 256, "k": 6, "D": 4100, "mode": 1, "masked": True,
         "dtype": "fp16"},
        # One decode token at the hidden width: latency.
        {"name": "norm forward, 1 token", "op": "norm_forward", "m": 1, "D": 8192, "gate": 1, "dtype": "bf16"},
        # An odd batch of an odd width, gated element by element.
        {"name": "norm forward, 1000 tokens", "op": "norm_forward", "m": 1000, "D": 5001, "gate": 2, "dtype": "fp16"},
        # A training step's rows at the hidden width.
        {"name": "norm backward, 8192 tokens", "op": "norm_backward", "m": 8192, "D": 8192, "gate": 2, "dtype": "bf16"},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _drawn(rng):
    op = rng.choice(["w4", "experts", "moe_forward", "moe_backward", "norm_forward", "norm_backward"])
    if op == "w4":
        return {"op": op, "m": _spread(rng, 1, 256), "N": _spread(rng, 256, 8192), "K": _spread(rng, 512, 8192),
                "group": rng.choice([32, 64, 128]), "zeros": rng.random() < 0.5, "dtype": rng.choice(["bf16", "fp16"])}
    if op == "experts":
        E = rng.choice([8, 60, 128, 256])
        return {"op": op, "tokens": _spread(rng, 1, 1000), "k": rng.choice([1, 2, 4, 6, 8]), "E": E, "N": _spread(rng, 256, 8192),
                "K": _spread(rng, 512, 8192), "group": rng.choice([32, 64, 128]), "zeros": rng.random() < 0.5,
                "dtype": rng.choice(["bf16", "fp16"]), "skew": rng.choice([0.0, 0.5, 1.0])}
    if op in ("moe_forward", "moe_backward"):
        return {"op": op, "m": _spread(rng, 1, 4096), "E": rng.choice([8, 60, 128, 256]), "k": rng.choice([1, 2, 4, 6, 8]),
                "D": _spread(rng, 512, 8192), "mode": rng.choice([0, 1]), "masked": rng.random() < 0.5,
                "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    return {"op": op, "m": _spread(rng, 1, 8192), "D": _spread(rng, 512, 8192), "gate": rng.choice([0, 1, 2, 3]),
            "dtype": rng.choice(["bf16", "fp16", "fp32"])}


def draw(rng):
    known = [work(c) for c in listed()]
    most_bytes, most_flops = max(w["bytes"] for w in known), max(w["flops"] for w in known)
    while True:
        case = _drawn(rng)
        w = work(case)
        cells = case["E"] * case["N"] * case["K"] if case["op"] == "experts" else 0
        if w["bytes"] <= most_bytes and w["flops"] <= most_flops and cells <= 256 * 1024 * 8192:
            return case


def _popularity(case):
    """Share of the tokens' choices by expert: 1 / rank ** skew."""
    p = [1.0 / (i + 1) ** case["skew"] for i in range(case["E"])]
    return [v / sum(p) for v in p]


def work(case):
    op = case["op"]
    if op in ("w4", "experts"):
        N, K = case["N"], case["K"]
        groups = -(-K // case["group"])
        if op == "w4":
            rows, hit = case["m"], 1.0
        else:
            rows = case["tokens"] * min(case["k"], case["E"])
            hit = sum(1.0 - max(0.0, 1.0 - case["k"] * p) ** case["tokens"] for p in _popularity(case))
        matrix = N * (-(-K // 2) + groups * (3 if case["zeros"] else 2))
        return {"bytes": hit * matrix + 2.0 * rows * (N + K), "flops": 2.0 * rows * N * K}
    el = SIZES[case["dtype"]]
    m, D = case["m"], case["D"]
    if op.startswith("moe"):
        k, E = case["k"], case["E"]
        row = m * D * el
        if op == "moe_forward":
            return {"bytes": (2.0 * k + 2) * row + 4.0 * m * E + 16.0 * m * k + 4.0 * (E + 1), "flops": 2.0 * m * k * D}
        return {"bytes": (3.0 * k + 2) * row + 4.0 * m * E * (1 + case["mode"]) + 16.0 * m * k, "flops": 4.0 * m * k * D}
    gate = {0: 0, 1: D, 2: m * D, 3: m}[case["gate"]] * el
    if op == "norm_forward":
        return {"bytes": 4.0 * m * D * el + 2.0 * D * el + gate + 8.0 * m, "flops": 10.0 * m * D}
    grads = (8.0 * D if case["gate"] != 1 else 12.0 * D) + (gate if case["gate"] in (2, 3) else 0)
    return {"bytes": 6.0 * m * D * el + 2.0 * D * el + gate + 8.0 * m + grads, "flops": 24.0 * m * D}


class _Handle:
    """A prepared stack of 4-bit matrices, freed with its state."""

    def __init__(self, lib, *args):
        self.lib, self.h = lib, lib.proj_w4_prepare(*args)

    def __del__(self):
        self.lib.proj_w4_destroy(self.h)


def _lib():
    from gemv_projection_layers_gb300 import binding
    return binding


def _plan(logits, k, mode):
    """Chosen experts, their weights, and the rows sorted by expert (stable), from the logits."""
    m, E = logits.shape
    clean = torch.where(torch.isnan(logits), torch.full_like(logits, -math.inf), logits)
    top, expert = torch.sort(clean, dim=1, descending=True, stable=True)
    taken = top[:, :k] > -math.inf
    best = torch.where(top[:, :1] > -math.inf, top[:, :1], torch.zeros_like(top[:, :1]))
    parts = torch.exp(top - best)
    total = (parts[:, :k] if mode == 0 else parts).sum(1, keepdim=True)
    weight = torch.where(taken, parts[:, :k] / torch.where(total > 0, total, torch.ones_like(total)), torch.zeros_like(parts[:, :k]))
    expert = torch.where(taken, expert[:, :k], torch.full_like(expert[:, :k], -1)).to(torch.int32)
    flat = expert.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    order = torch.sort(key, stable=True).indices
    places = torch.arange(m * k, device=logits.device)
    slot = torch.empty_like(places)
    slot[order] = places
    slot = torch.where(flat < 0, torch.full_like(slot, -1), slot)
    counts = (key[:, None] == torch.arange(E, device=logits.device)[None, :]).sum(0)
    offsets = torch.cat([torch.zeros(1, dtype=torch.long, device=logits.device), torch.cumsum(counts, 0)])
    order = torch.where(places < offsets[-1], order, torch.full_like(order, -1))
    return {"expert": expert, "weight": weight, "offsets": offsets.to(torch.int32), "order": order.to(torch.int32),
            "slot": slot.reshape(m, k).to(torch.int32)}


def _rows(m, width, dtype, gen, scale=1.0):
    """m rows whose stride is the width rounded up to 16 bytes, as a program that pads its buffers keeps them."""
    pad = -(-width // 8) * 8
    return (torch.randn(m, pad, device="cuda", generator=gen) * scale).to(dtype)[:, :width]


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    s = {"case": case}
    if op in ("w4", "experts"):
        N, K, group = case["N"], case["K"], case["group"]
        E = 1 if op == "w4" else case["E"]
        groups = -(-K // group)
        # Codes of normal weights at about a third of a standard deviation a step; scales spread by a factor of a few.
        codes = (torch.randn(E, N, -(-K // 2) * 2, device="cuda", generator=gen) * 2.6 + 8.0).round_().clamp_(0, 15).to(torch.uint8)
        s["codes"] = codes[..., 0::2] | (codes[..., 1::2] << 4)
        del codes
        s["scales"] = (torch.exp(0.3 * torch.randn(E, N, groups, device="cuda", generator=gen)) / (2.6 * math.sqrt(K))).to(dtype)
        s["zeros"] = torch.randint(6, 11, (E, N, groups), device="cuda", generator=gen, dtype=torch.uint8) if case["zeros"] else None
        if op == "w4":
            m = case["m"]
        else:
            k = min(case["k"], E)
            p = torch.tensor(_popularity(case), device="cuda")[torch.randperm(E, device="cuda", generator=gen)]
            picks = torch.multinomial(p.expand(case["tokens"], E), k, generator=gen)
            counts = torch.bincount(picks.reshape(-1), minlength=E)
            s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), torch.cumsum(counts, 0)]).to(torch.int32)
            s["most"] = int(counts.max())
            m = case["tokens"] * k
        s["x"] = _rows(m, K, dtype, gen)
        if own:
            B = _lib()
            s["handle"] = _Handle(B, s["codes"], s["scales"], s["zeros"], E, N, K, group, B.PROJ_BF16 if case["dtype"] == "bf16" else B.PROJ_FP16)
            s["out"] = torch.empty(m, N, device="cuda", dtype=dtype)
        return s
    m, D = case["m"], case["D"]
    if op.startswith("moe"):
        E, k = case["E"], min(case["k"], case["E"])
        logits = torch.randn(m, E, device="cuda", generator=gen) * 2.0
        logits = torch.round(logits * 64.0) / 64.0  # coarse enough that ties come up
        if case["masked"]:
            logits[:, torch.randperm(E, device="cuda", generator=gen)[: max(1, E // 16)]] = -math.inf
            logits[torch.rand(m, device="cuda", generator=gen) < 0.05] = -math.inf
        s["logits"], s["k"] = logits, k
        s["ys"] = torch.randn(m * k, D, device="cuda", generator=gen).to(dtype)
        if op == "moe_forward":
            s["x"] = torch.randn(m, D, device="cuda", generator=gen).to(dtype)
            if own:
                B = _lib()
                new = lambda *shape, t=torch.int32: torch.zeros(*shape, device="cuda", dtype=t)  # noqa: E731
                s.update(expert=new(m, k), weight=new(m, k, t=F32), offsets=new(E + 1), order=new(m * k), slot=new(m, k),
                         xs=new(m * k, D, t=dtype), out=new(m, D, t=dtype))
                s["room"] = new(max(16, B.proj_moe_workspace(m, E, k)), t=torch.uint8)
        else:
            s["plan"] = _plan(logits, k, case["mode"])
            s["dout"] = torch.randn(m, D, device="cuda", generator=gen).to(dtype)
            s["dxs"] = torch.randn(m * k, D, device="cuda", generator=gen).to(dtype)
            if own:
                s.update(dys=torch.zeros(m * k, D, device="cuda", dtype=dtype), dweight=torch.zeros(m, k, device="cuda"),
                         dx=torch.zeros(m, D, device="cuda", dtype=dtype), dlogits=torch.zeros(m, E, device="cuda"))
        return s
    rand = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)  # noqa: E731
    s["y"] = (rand(m, D) * torch.exp(0.5 * rand(m, 1))).to(dtype)
    s["residual"] = (rand(m, D) * 2.0).to(dtype)
    s["gate"] = [None, lambda: rand(D), lambda: rand(m, D), lambda: rand(m)][case["gate"]]
    s["gate"] = s["gate"]().to(dtype) if s["gate"] else None
    s["w_post"], s["w_pre"] = (1.0 + 0.2 * rand(D)).to(dtype), (1.0 + 0.2 * rand(D)).to(dtype)
    s["eps"], s["alpha"], s["beta"] = 1e-6, 0.75, 0.5
    if op == "norm_backward":
        s["dout"], s["dnormed"] = rand(m, D).to(dtype), rand(m, D).to(dtype)
        f = _norm_forward(s)
        s["rstd_post"], s["rstd_pre"] = f["rstd_post"], f["rstd_pre"]
    if own:
        B = _lib()
        kind = {"bf16": B.PROJ_BF16, "fp16": B.PROJ_FP16, "fp32": B.PROJ_FP32}[case["dtype"]]
        like = torch.empty_like
        named = {"m": m, "D": D, "dtype": kind, "gate_mode": case["gate"], "gate_act": B.PROJ_GATE_SIGMOID, "eps": s["eps"],
                 "alpha": s["alpha"], "beta": s["beta"], "y": s["y"], "ldy": D, "residual": s["residual"], "ldr": D, "gate": s["gate"],
                 "ldg": D, "w_post": s["w_post"], "w_pre": s["w_pre"]}
        if op == "norm_forward":
            s["made"] = {"out": like(s["y"]), "normed": like(s["y"]), "rstd_post": torch.empty(m, device="cuda"),
                         "rstd_pre": torch.empty(m, device="cuda")}
            s["args"] = B.norm_args(**named, **s["made"], ldo=D, ldn=D)
        else:
            f32 = lambda *shape: torch.empty(*shape, device="cuda")  # noqa: E731
            s["made"] = {"dy": like(s["y"]), "dresidual": like(s["y"]), "dw_post": f32(D), "dw_pre": f32(D)}
            if case["gate"]:
                s["made"]["dgate"] = f32(D) if case["gate"] == 1 else like(s["gate"])
            s["room"] = torch.empty(max(16, B.proj_norm_workspace(m, D)), device="cuda", dtype=torch.uint8)
            s["args"] = B.norm_grad_args(**named, **s["made"], rstd_post=s["rstd_post"], rstd_pre=s["rstd_pre"], dout=s["dout"], lddo=D,
                                         dnormed=s["dnormed"], lddn=D, lddy=D, lddr=D, lddg=D, workspace=s["room"],
                                         workspace_bytes=s["room"].numel())
    return s


# ------------------------------------------------------------- plain forms --


def _weights(s):
    K, group = s["case"]["K"], s["case"]["group"]
    q = torch.stack((s["codes"] & 15, s["codes"] >> 4), dim=-1).flatten(-2)[..., :K].float()
    z = 8.0 if s["zeros"] is None else s["zeros"].float().repeat_interleave(group, dim=-1)[..., :K]
    return (q - z) * s["scales"].float().repeat_interleave(group, dim=-1)[..., :K]


def _w4_plain(s):
    return (s["x"].float() @ _weights(s)[0].t()).to(s["x"].dtype)


def _experts_plain(s):
    x, w, offsets = s["x"].float(), _weights(s), s["offsets"].long()
    rows = torch.arange(x.shape[0], device=x.device)
    expert = torch.searchsorted(offsets[1:], rows, right=True)
    place = rows - offsets[expert]
    padded = torch.zeros(w.shape[0], s["most"], x.shape[1], device=x.device)
    padded[expert, place] = x
    return torch.bmm(padded, w.transpose(1, 2))[expert, place].to(s["x"].dtype)


def _moe_forward_plain(s):
    plan = _plan(s["logits"], s["k"], s["case"]["mode"])
    x, k = s["x"], s["k"]
    kept = (plan["order"] >= 0)[:, None]
    xs = torch.where(kept, x[plan["order"].clamp(min=0).long() // k], torch.zeros((), device=x.device, dtype=x.dtype))
    picked = torch.where((plan["slot"] >= 0)[..., None], s["ys"].float()[plan["slot"].clamp(min=0).long()], torch.zeros((), device=x.device))
    out = (plan["weight"][..., None] * picked).sum(1).to(x.dtype)
    return {**plan, "xs": xs, "out": out}


def _moe_backward_plain(s):
    plan, mode = s["plan"], s["case"]["mode"]
    dout, ys, dxs = s["dout"].float(), s["ys"].float(), s["dxs"].float()
    slot, valid = plan["slot"].clamp(min=0).long(), plan["slot"] >= 0
    zero = torch.zeros((), device=dout.device)
    dweight = torch.where(valid, (dout[:, None, :] * ys[slot]).sum(-1), zero)
    dx = torch.where(valid[..., None], dxs[slot], zero).sum(1).to(s["dout"].dtype)
    order = plan["order"].clamp(min=0).long()
    scaled = plan["weight"].reshape(-1)[order][:, None] * dout[order // s["k"]]
    dys = torch.where((plan["order"] >= 0)[:, None], scaled, zero).to(s["dout"].dtype)
    inner = (plan["weight"] * dweight).sum(1, keepdim=True)
    into = torch.zeros_like(s["logits"])
    column = plan["expert"].clamp(min=0).long()
    if mode == 0:
        into.scatter_add_(1, column, torch.where(valid, plan["weight"] * (dweight - inner), zero))
        dlogits = into
    else:
        into.scatter_add_(1, column, torch.where(valid, dweight, zero))
        logits = torch.where(torch.isnan(s["logits"]), zero - math.inf, s["logits"])
        best = logits.max(1, keepdim=True).values
        parts = torch.exp(logits - torch.where(best > -math.inf, best, zero))
        total = parts.sum(1, keepdim=True)
        dlogits = parts / torch.where(total > 0, total, zero + 1) * (into - inner)
    return {"dys": dys, "dweight": dweight, "dx": dx, "dlogits": dlogits}


def _gate(s):
    g = s["gate"]
    if g is None:
        return None, 1.0
    g = torch.sigmoid(g.float())
    return g, (g[:, None] if s["case"]["gate"] == 3 else g)


def _norm_forward(s):
    y, r = s["y"].float(), s["residual"].float()
    _, g = _gate(s)
    rstd_post = torch.rsqrt((y * y).mean(1) + s["eps"])
    u = s["alpha"] * r + s["beta"] * g * (y * rstd_post[:, None] * s["w_post"].float())
    rstd_pre = torch.rsqrt((u * u).mean(1) + s["eps"])
    normed = u * rstd_pre[:, None] * s["w_pre"].float()
    dtype = s["y"].dtype
    return {"out": u.to(dtype), "normed": normed.to(dtype), "rstd_post": rstd_post, "rstd_pre": rstd_pre}


def _norm_backward_plain(s):
    dtype, mode = s["y"].dtype, s["case"]["gate"]
    y, r, w_post, w_pre = s["y"].float(), s["residual"].float(), s["w_post"].float(), s["w_pre"].float()
    raw, g = _gate(s)
    rp, ru = s["rstd_post"][:, None], s["rstd_pre"][:, None]
    yn = y * rp
    n = yn * w_post
    u = s["alpha"] * r + s["beta"] * g * n
    un = u * ru
    dh = s["dnormed"].float()
    t = dh * w_pre
    du = s["dout"].float() + ru * (t - un * (t * un).mean(1, keepdim=True))
    c = s["beta"] * g * du
    b = c * w_post
    dy = rp * (b - yn * (b * yn).mean(1, keepdim=True))
    res = {"dy": dy.to(dtype), "dresidual": (s["alpha"] * du).to(dtype), "dw_post": (c * yn).sum(0), "dw_pre": (dh * un).sum(0)}
    if mode:
        dg = s["beta"] * n * du
        if mode == 1:
            res["dgate"] = dg.sum(0) * raw * (1.0 - raw)
        elif mode == 2:
            res["dgate"] = (dg * raw * (1.0 - raw)).to(dtype)
        else:
            res["dgate"] = (dg.sum(1) * raw * (1.0 - raw)).to(dtype)
    return res


def _own(s):
    B, case = _lib(), s["case"]
    op = case["op"]
    if op == "w4":
        B.proj_w4_run(s["handle"].h, s["x"], s["x"].stride(0), case["m"], s["out"], case["N"])
        return s["out"]
    if op == "experts":
        B.proj_w4_run_experts(s["handle"].h, s["x"], s["x"].stride(0), s["x"].shape[0], s["offsets"], s["out"], case["N"])
        return s["out"]
    if op == "norm_forward":
        B.proj_norm(s["args"])
        return s["made"]
    if op == "norm_backward":
        B.proj_norm_backward(s["args"])
        return s["made"]
    m, D, E, k, mode = case["m"], case["D"], case["E"], s["k"], case["mode"]
    kind = {"bf16": B.PROJ_BF16, "fp16": B.PROJ_FP16, "fp32": B.PROJ_FP32}[case["dtype"]]
    if op == "moe_forward":
        B.proj_moe_route(s["logits"], E, m, E, k, mode, s["expert"], s["weight"], s["offsets"], s["order"], s["slot"], s["room"],
                         s["room"].numel())
        B.proj_moe_gather(s["x"], D, s["slot"], m, D, k, kind, s["xs"], D)
        B.proj_moe_combine(s["ys"], D, s["slot"], s["weight"], m, D, k, kind, s["out"], D)
        return {n: s[n] for n in ("expert", "weight", "offsets", "order", "slot", "xs", "out")}
    plan = s["plan"]
    B.proj_moe_combine_backward(s["dout"], D, s["ys"], D, plan["slot"], plan["weight"], m, D, k, kind, s["dys"], D, s["dweight"])
    B.proj_moe_combine(s["dxs"], D, plan["slot"], None, m, D, k, kind, s["dx"], D)
    B.proj_moe_route_backward(s["logits"], E, m, E, k, mode, plan["expert"], plan["weight"], s["dweight"], s["dlogits"], E)
    return {n: s[n] for n in ("dys", "dweight", "dx", "dlogits")}


def run(state):
    if own:
        return _own(state)
    return {"w4": _w4_plain, "experts": _experts_plain, "moe_forward": _moe_forward_plain, "moe_backward": _moe_backward_plain,
            "norm_forward": _norm_forward, "norm_backward": _norm_backward_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------ 64-bit values --


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    op = case["op"]
    if op in ("w4", "experts"):
        K, N = case["K"], case["N"]
        column = torch.arange(K, device="cuda")
        x = d["x"]
        out = torch.zeros(x.shape[0], N, device="cuda", dtype=torch.float64)
        ends = [0, x.shape[0]] if op == "w4" else s["offsets"].tolist()
        for e in range(len(ends) - 1):
            if ends[e] == ends[e + 1]:
                continue
            byte = s["codes"][e][:, column // 2].int()
            q = torch.where(column % 2 == 1, byte // 16, byte % 16).double()
            q -= 8 if s["zeros"] is None else s["zeros"][e][:, column // case["group"]].double()
            w = q * d["scales"][e][:, column // case["group"]]
            out[ends[e]:ends[e + 1]] = torch.einsum("ik,nk->in", x[ends[e]:ends[e + 1]], w)
        return out
    if op.startswith("moe"):
        m, E, D, k, mode = case["m"], case["E"], case["D"], s["k"], case["mode"]
        lg = torch.nan_to_num(d["logits"], nan=-math.inf, posinf=math.inf, neginf=-math.inf)
        prob = torch.nan_to_num(torch.softmax(lg, dim=1), nan=0.0)
        pick = torch.argsort(-lg, dim=1, stable=True)[:, :k]
        real = torch.gather(lg, 1, pick) > -math.inf
        weight = torch.gather(prob, 1, pick) * real
        if mode == 0:
            weight = torch.nan_to_num(torch.softmax(torch.gather(lg, 1, pick), dim=1), nan=0.0) * real
        key = torch.where(real, pick, E).reshape(-1)
        ranked = torch.argsort(key, stable=True)
        n = int(real.sum())
        token = torch.div(ranked[:n], k, rounding_mode="floor")
        if op == "moe_forward":
            xs = torch.zeros(m * k, D, device="cuda", dtype=torch.float64)
            xs[:n] = d["x"][token]
            out = torch.zeros(m, D, device="cuda", dtype=torch.float64)
            out.index_add_(0, token, d["ys"][:n] * weight.reshape(-1)[ranked[:n]][:, None])
            return {"expert": None, "weight": weight, "offsets": None, "order": None, "slot": None, "xs": xs, "out": out}
        w = s["plan"]["weight"].double()  # the gradient is taken at the weights that the forward pass gave
        dys = torch.zeros(m * k, D, device="cuda", dtype=torch.float64)
        dys[:n] = d["dout"][token] * w.reshape(-1)[ranked[:n]][:, None]
        dweight = torch.zeros(m * k, device="cuda", dtype=torch.float64)
        dweight[ranked[:n]] = torch.einsum("sd,sd->s", d["dout"][token], d["ys"][:n])
        dweight = dweight.reshape(m, k)
        dx = torch.zeros(m, D, device="cuda", dtype=torch.float64)
        dx.index_add_(0, token, d["dxs"][:n])
        chosen = torch.zeros(m, E, device="cuda", dtype=torch.float64)
        row = torch.arange(m, device="cuda")[:, None].expand(m, k)
        inner = torch.einsum("mk,mk->m", w, dweight)[:, None]
        if mode == 0:
            chosen[row[real], pick[real]] = (w * (dweight - inner))[real]
            dlogits = chosen
        else:
            chosen[row[real], pick[real]] = dweight[real]
            dlogits = prob * (chosen - inner)
        return {"dys": dys, "dweight": dweight, "dx": dx, "dlogits": dlogits}
    # With v = alpha r + beta G(g) N(y), the gradients come from differentiating the definition itself in 64 bits.
    mode, D = case["gate"], case["D"]
    leaf = {n: d[n].clone().requires_grad_(op == "norm_backward") for n in ("y", "residual", "w_post", "w_pre")}
    gate = d["gate"].clone().requires_grad_(op == "norm_backward") if mode else None
    ms_y = leaf["y"].pow(2).sum(1, keepdim=True) / D
    v = leaf["y"] / torch.sqrt(ms_y + s["eps"]) * leaf["w_post"] * s["beta"]
    if mode:
        v = v / (1 + torch.exp(-(gate.unsqueeze(1) if mode == 3 else gate)))
    v = v + s["alpha"] * leaf["residual"]
    ms_v = v.pow(2).sum(1, keepdim=True) / D
    h = v / torch.sqrt(ms_v + s["eps"]) * leaf["w_pre"]
    if op == "norm_forward":
        return {"out": v, "normed": h, "rstd_post": (ms_y + s["eps"]).pow(-0.5)[:, 0], "rstd_pre": (ms_v + s["eps"]).pow(-0.5)[:, 0]}
    wanted = [leaf["y"], leaf["residual"], leaf["w_post"], leaf["w_pre"]] + ([gate] if mode else [])
    found = torch.autograd.grad([v, h], wanted, [d["dout"], d["dnormed"]])
    return dict(zip(["dy", "dresidual", "dw_post", "dw_pre"] + (["dgate"] if mode else []), found))
