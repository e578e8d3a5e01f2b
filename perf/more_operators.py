"""Cases of the cache of keys and values between the qkv_gate and o projections, each in a plain form and through
the library.

Four operators: rows of keys and values quantised as they are written to a paged cache, rows of it read back,
accepted drafts moved to their places in it, and attention of drafted tokens (a tree, or a single token) over it.
"""
import math

import torch

own = False

F32 = torch.float32
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
FORMATS = ["rows", "e4m3", "int8"]
LARGEST = {"e4m3": 448.0, "int8": 127.0}


def listed():
    # Heads and widths are those of the qkv_gate rows (1024 + 128 + 128 + 1024 columns: eight query heads of 128 on
    # one of keys and values, and a gate) unless the comment says otherwise.
    return [
        # The row of one decode step, one sequence: latency.
        {"name": "write, 1 token", "op": "write", "B": 1, "T": 1, "ragged": False, "ctx": 1000, "kv": 1, "group": 8, "D": 128, "page": 64,
         "format": "e4m3", "dtype": "bf16"},
        # A chunk of four prompts with many heads; pages that are no power of two.
        {"name": "write, 8192 tokens", "op": "write", "B": 4, "T": 2048, "ragged": False, "ctx": 1001, "kv": 8, "group": 4, "D": 128, "page": 48,
         "format": "int8", "dtype": "fp16"},
        # A short context read back for another use: latency.
        {"name": "read, 1 sequence", "op": "read", "B": 1, "ctx": 333, "kv": 2, "group": 4, "D": 64, "page": 16, "format": "int8", "dtype": "fp16"},
        # Contexts of a batch read back, of unequal lengths.
        {"name": "read, 32 sequences", "op": "read", "B": 32, "ctx": 8192, "kv": 8, "group": 8, "D": 128, "page": 64, "format": "e4m3",
         "dtype": "bf16"},
        # After a verify step of 32 sequences with 8 drafts.
        {"name": "move, 32 sequences of 8 drafts", "op": "move", "B": 32, "T": 8, "ragged": False, "ctx": 500, "kv": 1, "group": 8, "D": 128,
         "page": 64, "format": "e4m3", "dtype": "bf16"},
        # Large trees, many heads, an unquantised cache.
        {"name": "move, 256 sequences of 64 drafts", "op": "move", "B": 256, "T": 64, "ragged": True, "ctx": 100, "kv": 8, "group": 4, "D": 128,
         "page": 32, "format": "rows", "dtype": "fp16"},
        # One decode token over a short context: latency.
        {"name": "attention, 1 token", "op": "attention", "B": 1, "T": 1, "ragged": False, "ctx": 8192, "kv": 1, "group": 8, "D": 128, "page": 64,
         "format": "e4m3", "dtype": "bf16", "tree": False, "gate": True},
        # A decode step of 32 sequences of unequal lengths over an unquantised cache.
        {"name": "attention, 32 tokens", "op": "attention", "B": 32, "T": 1, "ragged": False, "ctx": 16384, "kv": 1, "group": 8, "D": 128,
         "page": 64, "format": "rows", "dtype": "bf16", "tree": False, "gate": True},
        # A verify step of 16 sequences with trees of 8 drafts over long contexts.
        {"name": "attention, 16 trees of 8", "op": "attention", "B": 16, "T": 8, "ragged": False, "ctx": 32768, "kv": 1, "group": 8, "D": 128,
         "page": 128, "format": "e4m3", "dtype": "bf16", "tree": True, "gate": True},
        # Odd everything: heads in groups of three, uneven trees, pages that end inside tiles.
        {"name": "attention, 5 trees of up to 13", "op": "attention", "B": 5, "T": 13, "ragged": True, "ctx": 5001, "kv": 5, "group": 3, "D": 64,
         "page": 48, "format": "int8", "dtype": "fp16", "tree": True, "gate": False},
        # A verify step of 32 sequences with all of a model's heads on one GPU, chains of drafts, an unquantised cache.
        {"name": "attention, 32 chains of 8, 64 heads", "op": "attention", "B": 32, "T": 8, "ragged": False, "ctx": 8192, "kv": 8, "group": 8,
         "D": 128, "page": 64, "format": "rows", "dtype": "fp16", "tree": False, "gate": False},
        # The widest trees: products weigh more than the cache's bytes.
        {"name": "attention, 32 trees of up to 64", "op": "attention", "B": 32, "T": 64, "ragged": True, "ctx": 16384, "kv": 1, "group": 8,
         "D": 128, "page": 64, "format": "e4m3", "dtype": "bf16", "tree": True, "gate": True},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _drawn(rng):
    op = rng.choice(["write", "read", "move", "attention", "attention", "attention"])
    case = {"op": op, "kv": rng.choice([1, 2, 4, 5, 8]), "group": rng.choice([1, 2, 3, 4, 7, 8, 12, 16]), "D": rng.choice([64, 128]),
            "page": rng.choice([16, 32, 48, 64, 100, 128]), "format": rng.choice(FORMATS), "dtype": rng.choice(["bf16", "fp16"])}
    if op == "write":
        return {**case, "B": _spread(rng, 1, 64), "T": _spread(rng, 1, 2048), "ragged": rng.random() < 0.5, "ctx": _spread(rng, 1, 2000)}
    if op == "read":
        return {**case, "B": _spread(rng, 1, 64), "ctx": _spread(rng, 16, 16384)}
    if op == "move":
        return {**case, "B": _spread(rng, 1, 256), "T": _spread(rng, 1, 64), "ragged": rng.random() < 0.5, "ctx": _spread(rng, 1, 1000)}
    return {**case, "B": _spread(rng, 1, 64), "T": _spread(rng, 1, 64), "ragged": rng.random() < 0.5, "ctx": _spread(rng, 16, 32768),
            "tree": rng.random() < 0.6, "gate": rng.random() < 0.5}


def _values(case):
    """Numbers that the plain form holds at a time: the contexts of a batch, and their products with the rows of q."""
    drafts = case.get("T", 0)
    held = case["B"] * (case["ctx"] + drafts) * case["kv"] * case["D"]
    return max(held, case["B"] * case["kv"] * case["group"] * drafts * (case["ctx"] + drafts) if case["op"] == "attention" else 0)


def draw(rng):
    known = [work(c) for c in listed()]
    most_bytes, most_flops, most_values = max(w["bytes"] for w in known), max(w["flops"] for w in known), max(_values(c) for c in listed())
    while True:
        case = _drawn(rng)
        w = work(case)
        if w["bytes"] <= most_bytes and w["flops"] <= most_flops and _values(case) <= most_values:
            return case


def _contexts(case):
    """Tokens of each sequence that the cache holds before the call: the first has all of ctx, the others less."""
    return [max(1, int(case["ctx"] * (1.0 - 0.75 * ((0.6180339887 * b) % 1.0)))) for b in range(case["B"])]


def _drafts(case):
    """Rows of each sequence in the call; of ragged batches some sequences have none."""
    if not case["ragged"]:
        return [case["T"]] * case["B"]
    return [case["T"] if b % 3 == 0 else 0 if b % 8 == 5 else 1 + 5 * b % case["T"] for b in range(case["B"])]


def _row_bytes(case):
    """Bytes of one head's entry of keys or values, its scale with it."""
    return 2 * case["D"] if case["format"] == "rows" else case["D"] + 4


def work(case):
    kv, D, op = case["kv"], case["D"], case["op"]
    entry = 2.0 * kv * _row_bytes(case)
    if op in ("write", "read"):
        m = sum(_drafts(case)) if op == "write" else sum(_contexts(case))
        return {"bytes": m * (entry + 4.0 * kv * D) + 4.0 * (2 * case["B"] + 1), "flops": 2.0 * m * 2 * kv * D}
    if op == "move":
        moved = sum(max(1, t // 2) if t else 0 for t in _drafts(case))
        return {"bytes": 2.0 * moved * entry + 8.0 * case["B"] + 4.0 * case["B"] * case["T"], "flops": 0.0}
    heads = kv * case["group"]
    rows, lens = _drafts(case), _contexts(case)
    keys = sum(n + t for n, t in zip(lens, rows) if t)
    pairs = sum(t * (n + t) for n, t in zip(lens, rows))
    m = sum(rows)
    words = -(-case["T"] // 32) if case["tree"] else 0
    out = m * heads * (D * (6.0 if case["gate"] else 4.0) + 4.0)
    return {"bytes": keys * entry + out + 4.0 * m * words + 4.0 * keys / case["page"], "flops": 4.0 * pairs * heads * D}


def _lib():
    from gemv_projection_layers_gb300 import binding
    return binding


def _quantise(x, format):
    """Codes and scales of rows x (fp32, [..., D]): scale = largest magnitude / largest code, code = round(x (1 / scale))."""
    top = x.abs().amax(-1)
    scale = torch.maximum(top / torch.full_like(top, LARGEST[format]), torch.full_like(top, 2.0 ** -126))
    scale = torch.where(torch.isfinite(top), scale, torch.full_like(top, math.nan))
    code = torch.where(torch.isfinite(top)[..., None], x * torch.reciprocal(scale)[..., None], torch.zeros_like(x))
    if format == "e4m3":
        return code.to(torch.float8_e4m3fn), scale
    return code.round().to(torch.int8), scale


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _offsets(counts):
    total = [0]
    for n in counts:
        total.append(total[-1] + n)
    return _int32(total)


def _trees(case, gen):
    """Random trees of drafts: for each row the set of drafts it sees (its ancestors and itself), 32 to a word."""
    B, T = case["B"], case["T"]
    back = (torch.rand(B, T, generator=gen) ** 2 * 4.0).long() + 1  # most drafts follow one of the last few
    parent = torch.arange(T)[None, :] - back
    sees = torch.zeros(B, T, T, dtype=torch.bool)
    for i in range(T):
        p = parent[:, i]
        sees[:, i] = sees[torch.arange(B), p.clamp(min=0)] & (p >= 0)[:, None]
        sees[:, i, i] = True
    words = -(-T // 32)
    bits = torch.zeros(B, T, words * 32, dtype=torch.int64)
    bits[:, :, :T] = sees.long()
    packed = (bits.view(B, T, words, 32) << torch.arange(32)).sum(-1)
    packed = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).to(torch.int32)
    return torch.cat([packed[b, :t] for b, t in enumerate(_drafts(case))]).cuda()


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    op, dtype, format = case["op"], DTYPES[case["dtype"]], case["format"]
    B, kv, D, page = case["B"], case["kv"], case["D"], case["page"]
    heads = kv * case["group"]
    rand = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)  # noqa: E731
    lens = _contexts(case)
    rows = lens if op == "read" else _drafts(case)
    ends = lens if op == "read" else [n + t for n, t in zip(lens, rows)]
    # Pages are dealt out in no order, a tenth are free; a table's unused places hold -1.
    need = [-(-n // page) for n in ends]
    width = max(need) + 1
    pages = sum(need) + sum(need) // 10 + 1
    deal = torch.randperm(pages, generator=host).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = deal[at:at + n]
        at += n
    s = {"case": case, "table": table.cuda(), "width": width, "most": max(ends), "rows": max(rows), "offsets": _offsets(rows)}
    s["start"] = _int32([0] * B if op == "read" else lens)
    m = sum(rows)
    # A few channels of the keys are larger than the others by some factor, as in a model; values differ in size by token.
    channel = 1.0 + 5.0 * (torch.rand(kv, 1, D, device="cuda", generator=gen) < 0.05)
    for name in ("k", "v"):
        x = rand(pages, kv, page, D) * (channel if name == "k" else torch.exp(0.4 * rand(pages, kv, page, 1)))
        if format == "rows":
            s[name] = x.to(dtype)
        else:
            s[name], s[name + "_scale"] = _quantise(x, format)
        del x
    if op == "attention":
        # What stands behind a sequence's last token was never written: NaN.
        spot = torch.arange(width * page, device="cuda")
        page_of = s["table"].long()[:, spot // page]
        stale = (spot[None, :] >= _int32(ends)[:, None]) & (page_of >= 0)
        into = page_of[stale], (spot % page).expand(B, -1)[stale]
        for name in ("k", "v"):
            if format == "rows":
                s[name][into[0], :, into[1]] = math.nan
            else:
                s[name + "_scale"][into[0], :, into[1]] = math.nan
    s["m"] = m
    if op in ("write", "attention"):
        # Rows as the projection leaves them: queries, keys, values and gate side by side.
        s["ld"] = (2 * heads + 2 * kv) * D
        qkvg = torch.cat([rand(m, heads * D), (rand(m, kv, D) * channel[:, 0]).reshape(m, kv * D), rand(m, kv * D), rand(m, heads * D)], 1).to(dtype)
        s["q"], s["new_k"], s["new_v"], gate = torch.split(qkvg, [heads * D, kv * D, kv * D, heads * D], 1)
    if op == "move":
        depth = case["T"]
        # Half of a sequence's drafts are accepted, along a path that skips some.
        taken = torch.full((B, depth), -1, dtype=torch.int32)
        for b, t in enumerate(rows):
            n = max(1, t // 2) if t else 0
            taken[b, :n] = torch.randperm(t, generator=host)[:n].sort().values.to(torch.int32)
        s["path"], s["next"] = taken.cuda(), torch.zeros(B, dtype=torch.int32, device="cuda")
    if op == "read":
        s["out_k"], s["out_v"] = (torch.zeros(m, kv * D, device="cuda", dtype=dtype) for _ in range(2))
    if op == "attention":
        s["mask"] = _trees(case, host) if case["tree"] else None
        s["gate"] = gate if case["gate"] else None
        s["scale"] = 1.0 / math.sqrt(D)
    if own:
        L = _lib()
        s["cache"] = L.kv_cache(format={"rows": L.PROJ_KV_ROWS, "e4m3": L.PROJ_KV_E4M3, "int8": L.PROJ_KV_INT8}[format],
                                dtype=L.PROJ_BF16 if case["dtype"] == "bf16" else L.PROJ_FP16, pages=pages, page=page, heads=kv, D=D,
                                k=s["k"], v=s["v"], k_scale=s.get("k_scale"), v_scale=s.get("v_scale"), page_stride=kv * page * D,
                                head_stride=page * D, token_stride=D, table=s["table"], ldt=width, width=width, sequences=B)
        if op == "attention":
            s["out"], s["lse"] = torch.zeros(m, heads * D, device="cuda", dtype=dtype), torch.zeros(m, heads, device="cuda")
            room = L.proj_attn_workspace(s["cache"], m, heads)
            s["room"] = torch.empty(max(16, room), device="cuda", dtype=torch.uint8)
            words = s["mask"].shape[1] if case["tree"] else 0
            s["args"] = L.attn_args(cache=s["cache"], m=m, heads=heads, q=s["q"], ldq=s["ld"], offsets=s["offsets"], start=s["start"],
                                    mask=s["mask"], ldm=words, words=words, scale=s["scale"], gate=s["gate"], ldg=s["ld"],
                                    gate_act=L.PROJ_GATE_SIGMOID, out=s["out"], ldo=heads * D, lse=s["lse"], workspace=s["room"],
                                    workspace_bytes=s["room"].numel())
    return s


# ------------------------------------------------------------- plain forms --


def _sequence_of(s, m):
    """Each row's sequence and its place among that sequence's rows."""
    row = torch.arange(m, device="cuda")
    sequence = torch.searchsorted(s["offsets"].long()[1:], row, right=True)
    return sequence, row - s["offsets"].long()[sequence]


def _entry(s, sequence, position):
    """Page and place in it of the positions of sequences."""
    page = s["case"]["page"]
    return s["table"].long()[sequence, position // page], position % page


def _cache_out(s):
    return {n: s[n] for n in ("k", "v", "k_scale", "v_scale") if n in s}


def _bytes(t):
    """A cache of 8-bit floating point as bytes, which can be indexed."""
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _write_plain(s):
    kv, D = s["case"]["kv"], s["case"]["D"]
    m = s["m"]
    sequence, place = _sequence_of(s, m)
    page, spot = _entry(s, sequence, s["start"].long()[sequence] + place)
    for name in ("k", "v"):
        x = s["new_" + name].reshape(m, kv, D)
        if s["case"]["format"] == "rows":
            s[name][page, :, spot] = x
        else:
            code, scale = _quantise(x.float(), s["case"]["format"])
            _bytes(s[name])[page, :, spot] = _bytes(code)
            s[name + "_scale"][page, :, spot] = scale
    return _cache_out(s)


def _values_at(s, name, page, spot):
    """Entries of the cache as the numbers they stand for, fp32 [..., kv, D]."""
    got = _bytes(s[name])[page, :, spot]
    if s["case"]["format"] == "rows":
        return got.float()
    got = got.view(s[name].dtype).float()
    return got * s[name + "_scale"][page, :, spot][..., None]


def _read_plain(s):
    m = s["m"]
    sequence, place = _sequence_of(s, m)
    page, spot = _entry(s, sequence, s["start"].long()[sequence] + place)
    return {n: _values_at(s, n, page, spot).reshape(m, -1).to(s["out_k"].dtype) for n in ("k", "v")}


def _move_plain(s):
    path, start = s["path"].long(), s["start"].long()
    B, depth = path.shape
    taken = path >= 0
    sequence = torch.arange(B, device="cuda")[:, None].expand(B, depth)[taken]
    source = _entry(s, sequence, (start[:, None] + path)[taken])
    target = _entry(s, sequence, (start[:, None] + torch.arange(depth, device="cuda"))[taken])
    for name, t in _cache_out(s).items():
        t = _bytes(t)
        t[target[0], :, target[1]] = t[source[0], :, source[1]]
    return {**_cache_out(s), "next": (start + taken.sum(1)).to(torch.int32)}


def _attention_plain(s):
    case = s["case"]
    kv, G, D, B, T = case["kv"], case["group"], case["D"], case["B"], s["rows"]
    m = s["m"]
    sequence, place = _sequence_of(s, m)
    start, count = s["start"].long(), s["offsets"].long()[1:] - s["offsets"].long()[:-1]
    spot = torch.arange(s["most"], device="cuda")
    page, at = _entry(s, torch.arange(B, device="cuda")[:, None], spot[None, :].expand(B, -1))
    here = spot[None, :] < (start + count)[:, None]
    zero = torch.zeros((), device="cuda")
    k = torch.where(here[..., None, None], _values_at(s, "k", page.clamp(min=0), at), zero).permute(0, 2, 3, 1)  # [B, kv, D, keys]
    q = torch.zeros(B, T, kv, G, D, device="cuda")
    q[sequence, place] = s["q"].reshape(m, kv, G, D).float()
    score = (q.permute(0, 2, 1, 3, 4).reshape(B, kv, T * G, D) @ k).reshape(B, kv, T, G, -1) * s["scale"]
    del k
    draft = spot[None, :] - start[:, None]
    if case["tree"]:
        words = torch.zeros(B, T, s["mask"].shape[1], device="cuda", dtype=torch.long)
        words[sequence, place] = s["mask"].long()
        bit = draft.clamp(0, T - 1)
        word = torch.gather(words, 2, (bit // 32)[:, None, :].expand(B, T, -1))
        sees = (word >> (bit % 32)[:, None, :]) % 2 == 1
    else:
        sees = draft[:, None, :] <= torch.arange(T, device="cuda")[None, :, None]
    sees = ((draft < 0)[:, None, :] | sees) & here[:, None, :]
    score = torch.where(sees[:, None, :, None, :], score, zero - math.inf)
    best = score.amax(-1, keepdim=True)
    score = torch.exp(score - torch.where(best > -math.inf, best, zero))
    total = score.sum(-1, keepdim=True)
    v = torch.where(here[..., None, None], _values_at(s, "v", page.clamp(min=0), at), zero).permute(0, 2, 1, 3)
    out = (score.reshape(B, kv, T * G, -1) @ v).reshape(B, kv, T, G, D) / torch.where(total > 0, total, zero + 1)
    out = out.permute(0, 2, 1, 3, 4)[sequence, place].reshape(m, -1)
    if s["gate"] is not None:
        out = out * torch.sigmoid(s["gate"].float())
    lse = (best + torch.log(total))[..., 0].permute(0, 2, 1, 3)[sequence, place].reshape(m, -1)
    return {"out": out.to(s["q"].dtype), "lse": lse}


def _own(s):
    L, case = _lib(), s["case"]
    op, m = case["op"], s["m"]
    if op == "write":
        L.proj_kv_write(s["cache"], s["offsets"], s["start"], m, s["new_k"], s["ld"], s["new_v"], s["ld"])
        return _cache_out(s)
    if op == "read":
        width = case["kv"] * case["D"]
        L.proj_kv_read(s["cache"], s["offsets"], s["start"], m, s["out_k"], width, s["out_v"], width)
        return {"k": s["out_k"], "v": s["out_v"]}
    if op == "move":
        L.proj_kv_move(s["cache"], s["start"], s["path"], case["T"], case["T"], s["next"])
        return {**_cache_out(s), "next": s["next"]}
    L.proj_attn(s["args"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"write": _write_plain, "read": _read_plain, "move": _move_plain, "attention": _attention_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------ 64-bit values --


def exact(case, seed):
    s = prepare(case, seed)
    op, kv, D, format, page = case["op"], case["kv"], case["D"], case["format"], case["page"]
    tables, starts, ends = s["table"].tolist(), s["start"].tolist(), s["offsets"].tolist()
    real = lambda t: t.to(F32).double() if t.dtype == torch.float8_e4m3fn else t.double()  # noqa: E731

    def flat(name):
        """The cache as one row of heads a place: [pages page, kv, D] and the scales [pages page, kv]."""
        whole = real(s[name]).transpose(1, 2).reshape(-1, kv, D)
        return whole, (s[name + "_scale"].double().transpose(1, 2).reshape(-1, kv) if format != "rows" else None)

    def back(whole):
        return whole.reshape(-1, page, *whole.shape[1:]).transpose(1, 2).contiguous()

    def places(b, first, n):
        """Rows of flat() that hold n positions of sequence b, from `first` on."""
        return torch.tensor([tables[b][p // page] * page + p % page for p in range(first, first + n)], dtype=torch.long, device="cuda")

    if op == "read":
        out = {}
        for name in ("k", "v"):
            whole, scale = flat(name)
            got = torch.cat([whole[places(b, 0, ends[b + 1] - ends[b])] for b in range(case["B"])])
            if scale is not None:
                got = got * torch.cat([scale[places(b, 0, ends[b + 1] - ends[b])] for b in range(case["B"])])[..., None]
            out[name] = got.reshape(got.shape[0], kv * D)
        return out
    if op in ("write", "move"):
        out = {}
        for name in ("k", "v"):
            whole, scale = flat(name)
            for b in range(case["B"]):
                if op == "write":
                    into, x = places(b, starts[b], ends[b + 1] - ends[b]), s["new_" + name][ends[b]:ends[b + 1]].double().reshape(-1, kv, D)
                    if format == "rows":
                        whole[into] = x
                        continue
                    size = x.abs().max(-1).values / LARGEST[format]
                    scale[into] = size
                    # Steps of 2^-3 relative to the power of two below, none finer than 2^-9: 8-bit floating point.
                    y = x / size[..., None]
                    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3) if format == "e4m3" else torch.ones_like(y)
                    whole[into] = torch.round(y / step) * step
                else:
                    taken = [p for p in s["path"][b].tolist() if p >= 0]
                    source = torch.cat([places(b, starts[b] + p, 1) for p in taken]) if taken else places(b, 0, 0)
                    into = places(b, starts[b], len(taken))
                    whole[into] = whole[source]
                    if scale is not None:
                        scale[into] = scale[source]
            out[name] = back(whole) if format != "int8" else None
            if scale is not None:
                out[name + "_scale"] = back(scale)
        return out if op == "write" else {**out, "next": None}
    G = case["group"]
    outs, lses = [], []
    cache = {n: flat(n) for n in ("k", "v")}
    for b in range(case["B"]):
        n, t = starts[b], ends[b + 1] - ends[b]
        if not t:
            continue
        at = places(b, 0, n + t)
        k, v = (cache[i][0][at] if cache[i][1] is None else cache[i][0][at] * cache[i][1][at][..., None] for i in ("k", "v"))
        rows = slice(ends[b], ends[b + 1])
        q = s["q"][rows].double().reshape(t, kv, G, D)
        blocked = torch.zeros(t, n + t, dtype=torch.bool, device="cuda")
        if case["tree"]:
            bits = s["mask"][rows].long()[:, torch.arange(t, device="cuda") // 32] >> (torch.arange(t, device="cuda") % 32)
            blocked[:, n:] = bits % 2 == 0
        else:
            blocked[:, n:] = torch.ones(t, t, device="cuda").triu(1) > 0
        a = torch.einsum("thgd,khd->thgk", q, k) * s["scale"]
        a.masked_fill_(blocked[:, None, None, :], -math.inf)
        lses.append(torch.logsumexp(a, -1).reshape(t, kv * G))
        o = torch.einsum("thgk,khd->thgd", torch.softmax(a, -1), v).reshape(t, kv * G * D)
        if s["gate"] is not None:
            o = o / (1 + torch.exp(-s["gate"][rows].double()))
        outs.append(o)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
