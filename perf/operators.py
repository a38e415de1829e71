"""What is measured of the attention operators: rotary positions, the paged key-value cache as it is
written and read back, and the attention of one new token over it.

Every case has one operator ("op") and its sizes.  ``own`` false: the operators in elementary torch
operations; true: the calls a program makes of this package.
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
FORMATS = {"int8": torch.int8, "fp8": FP8, "bf16": torch.bfloat16}
TOP = {"int8": 127.0, "fp8": 448.0}
HALF, INTERLEAVED = 0, 1


# ---------------------------------------------------------------- cases


def listed():
    return [
        # one token of a 3B-sized model (dim 2560, 32 heads of 80): latency alone
        {"name": "rope_token", "op": "rope", "T": 1, "H": 32, "D": 80, "rot": 80, "layout": "half", "far": 2047, "parts": False},
        # a prompt of a context's length, half of each head rotated, far positions of a stretched context
        {"name": "rope_prompt_far", "op": "rope", "T": 2048, "H": 32, "D": 80, "rot": 40, "layout": "interleaved", "far": 900000, "parts": True},
        # the cache write of one decode step, one sequence
        {"name": "append_token_int8", "op": "append", "T": 1, "B": 1, "Hq": 32, "Hkv": 32, "D": 80, "rot": 80, "layout": "half", "far": 2047, "page": 64, "format": "int8"},
        # the cache write of a decode step of 64 sequences of a 1.3B-sized model (dim 2048, 16 heads of 128)
        {"name": "append_batch_fp8", "op": "append", "T": 64, "B": 64, "Hq": 16, "Hkv": 16, "D": 128, "rot": 128, "layout": "interleaved", "far": 2047, "page": 32, "format": "fp8"},
        # three prompts of a 3B-sized model packed into one call, odd lengths
        {"name": "append_prompts_int8", "op": "append", "T": 2039, "B": 3, "Hq": 32, "Hkv": 32, "D": 80, "rot": 80, "layout": "half", "far": 700, "page": 64, "format": "int8"},
        # a cached prompt back as fp32, for a prefill on top of it or for moving it out
        {"name": "read_prompt_int8", "op": "read", "T": 2048, "B": 1, "Hkv": 32, "D": 80, "page": 64, "format": "int8"},
        # shared heads, unquantised, an odd number of rows from several sequences
        {"name": "read_shared_bf16", "op": "read", "T": 4999, "B": 7, "Hkv": 5, "D": 128, "page": 16, "format": "bf16"},
        # the first tokens of an answer: almost nothing to read
        {"name": "attend_short_int8", "op": "attend", "B": 1, "Hq": 16, "Hkv": 16, "D": 128, "L": 37, "ragged": False, "window": 0, "page": 32, "format": "int8"},
        # one sequence at the context's end, every head with keys of its own
        {"name": "attend_token_int8", "op": "attend", "B": 1, "Hq": 32, "Hkv": 32, "D": 80, "L": 2048, "ragged": False, "window": 0, "page": 64, "format": "int8"},
        # a served batch of sequences of different ages
        {"name": "attend_batch_int8", "op": "attend", "B": 64, "Hq": 32, "Hkv": 32, "D": 80, "L": 2048, "ragged": True, "window": 0, "page": 64, "format": "int8"},
        # heads that share keys, e4m3, some long sequences
        {"name": "attend_shared_fp8", "op": "attend", "B": 8, "Hq": 32, "Hkv": 8, "D": 128, "L": 8192, "ragged": True, "window": 0, "page": 32, "format": "fp8"},
        # one very long sequence: the work is split over its length
        {"name": "attend_long_bf16", "op": "attend", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "L": 131071, "ragged": False, "window": 0, "page": 64, "format": "bf16"},
    ]


def _spread(rng, lo, hi):
    """An integer of lo..hi, even over its logarithm, odd ones among them."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "attend", "attend"])
    D = rng.choice([64, 80, 96, 112, 128])
    fmt, page = rng.choice(["int8", "fp8", "bf16"]), rng.choice([16, 32, 64, 128])
    Hkv, G = rng.choice([1, 2, 4, 5, 8, 16, 32]), rng.choice([1, 1, 2, 4, 7, 8])
    if Hkv * G > 64:
        G = 1
    rot, layout = rng.choice([D, D, D // 2, 32]), rng.choice(["half", "interleaved"])
    far = _spread(rng, 100, 1000000)
    if op == "rope":
        H = rng.choice([1, 5, 8, 16, 20, 32, 40])
        return {"op": op, "T": _spread(rng, 1, 2048), "H": H, "D": D, "rot": rot, "layout": layout, "far": far, "parts": rng.random() < 0.5}
    if op == "append":
        B = _spread(rng, 1, 64)
        return {"op": op, "T": max(B, _spread(rng, 1, 2048)), "B": B, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "rot": rot, "layout": layout,
                "far": min(far, 4000), "page": page, "format": fmt}
    if op == "read":
        return {"op": op, "T": _spread(rng, 1, 5000), "B": _spread(rng, 1, 16), "Hkv": Hkv, "D": D, "page": page, "format": fmt}
    B = _spread(rng, 1, 64)
    most = 80_000_000 // (B * Hkv * D * (2 if fmt == "bf16" else 1))  # tokens a sequence: below the largest listed case
    L = _spread(rng, 1, max(1, min(131072, most)))
    return {"op": op, "B": B, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "L": L, "ragged": rng.random() < 0.6,
            "window": rng.choice([0, 0, 0, _spread(rng, 1, max(1, L))]), "page": page, "format": fmt}


# ---------------------------------------------------------------- inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _frequencies(rot, parts):
    """Radians a position, fp64; `parts`: stretched by 16 where a pair turns seldom within 4096 positions."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    if parts:
        turns = 4096.0 * f / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0, 1)
        f = f * (keep + (1 - keep) / 16.0)
    return f


def _quantised(x, fmt):
    """fp32 rows [..., D] -> what a cache of the format holds, and the rows' steps."""
    if fmt == "bf16":
        return x.to(torch.bfloat16), None
    top = x.abs().amax(-1).clamp(min=1e-5)
    scaled = x * (TOP[fmt] / top)[..., None]
    codes = scaled.round().clamp(-128, 127).to(torch.int8) if fmt == "int8" else scaled.clamp(-448, 448).to(FP8)
    return codes, top / TOP[fmt]


def _pool(g, c, pages):
    """Keys and values of `pages` pages: channels of different size, as projections give them."""
    shape = (pages, c["Hkv"], c["page"], c["D"])
    size = torch.rand(c["Hkv"], 1, c["D"], generator=g, device="cuda") * 1.5 + 0.25
    out = {}
    for name in "kv":
        codes, step = _quantised(torch.randn(shape, generator=g, device="cuda") * size, c["format"])
        out[name], out[name + "_step"] = codes, step
    return out


def _lengths(c, seed):
    """Tokens of each sequence (attend)."""
    if not c["ragged"]:
        return torch.full((c["B"],), c["L"], dtype=torch.int32)
    g = torch.Generator()
    g.manual_seed(int(seed))
    return torch.randint(1, c["L"] + 1, (c["B"],), generator=g, dtype=torch.int32)


def _table(g, B, width):
    """Every sequence's pages, in no order."""
    return torch.randperm(B * width, generator=g, device="cuda").to(torch.int32).view(B, width)


def prepare(case, seed):
    c, g = dict(case), _generator(seed)
    s = {"case": c}
    if c["op"] == "rope":
        s["x"] = torch.randn(c["T"], c["H"], c["D"], generator=g, device="cuda")
        s["positions"] = (c["far"] - torch.arange(c["T"], device="cuda")).abs().to(torch.int32)
        s["freq"], s["amplitude"] = _frequencies(c["rot"], c["parts"]), 0.1 * math.log(16) + 1 if c["parts"] else 1.0
        s["out"] = torch.empty_like(s["x"])
        return s
    if c["op"] == "attend":
        width = -(-c["L"] // c["page"])
        s["cache"], s["table"] = _pool(g, c, c["B"] * width), _table(g, c["B"], width)
        s["lengths"] = _lengths(c, seed).cuda()
        s["q"] = torch.randn(c["B"], c["Hq"], c["D"], generator=g, device="cuda") * 1.5
        s["out"] = torch.empty_like(s["q"])
        if c["B"] * c["Hkv"] < 152:  # where a call may split a sequence over more workers than one cluster holds
            s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
        return s
    # rows packed sequence after sequence; each sequence's rows follow what it already holds (at most `far`)
    T, B = c["T"], c["B"]
    rows = torch.arange(T, device="cuda")
    s["seq"] = (rows * B // T).to(torch.int32)
    first = torch.searchsorted(s["seq"], torch.arange(B, device="cuda", dtype=torch.int32))
    old = torch.randint(0, c.get("far", 0) + 1, (B,), generator=g, device="cuda")
    s["positions"] = (rows - first[s["seq"].long()] + old[s["seq"].long()]).to(torch.int32)
    width = -(-(-(-T // B) + c.get("far", 0) + 1) // c["page"])
    s["table"] = _table(g, B, width)
    s["cache"] = _pool(g, c, B * width)
    if c["op"] == "append":
        s["freq"], s["amplitude"] = _frequencies(c["rot"], False), 1.0
        s["q"] = torch.randn(T, c["Hq"], c["D"], generator=g, device="cuda")
        s["k"] = torch.randn(T, c["Hkv"], c["D"], generator=g, device="cuda")
        s["v"] = torch.randn(T, c["Hkv"], c["D"], generator=g, device="cuda")
        s["q_out"] = torch.empty_like(s["q"])
    else:
        s["k_out"] = torch.empty(T, c["Hkv"], c["D"], device="cuda")
        s["v_out"] = torch.empty(T, c["Hkv"], c["D"], device="cuda")
    return s


# ---------------------------------------------------------------- plain forms


def _rotated(x, positions, freq, layout, amplitude):
    """x [T, H, D] fp32 with its first 2 * len(freq) dims rotated; angles in 64 bits, rounded once."""
    angle = positions.double()[:, None] * freq[None, :]
    c, s = (angle.cos().float() * amplitude)[:, None], (angle.sin().float() * amplitude)[:, None]
    n = freq.numel()
    out = x.clone()
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if layout == "interleaved" else (x[..., :n], x[..., n:2 * n])
    ra, rb = a * c - b * s, b * c + a * s
    if layout == "interleaved":
        out[..., 0:2 * n:2], out[..., 1:2 * n:2] = ra, rb
    else:
        out[..., :n], out[..., n:2 * n] = ra, rb
    return out


def _places(s):
    """(page, offset) of each row."""
    pos, page = s["positions"].long(), s["case"]["page"]
    return s["table"][s["seq"].long(), pos // page].long(), pos % page


def _plain_append(s):
    c = s["case"]
    q = _rotated(s["q"], s["positions"], s["freq"], c["layout"], s["amplitude"])
    page, at = _places(s)
    for name, x in (("k", _rotated(s["k"], s["positions"], s["freq"], c["layout"], s["amplitude"])), ("v", s["v"])):
        codes, step = _quantised(x, c["format"])
        held = s["cache"][name]
        if c["format"] == "fp8":
            held, codes = held.view(torch.uint8), codes.view(torch.uint8)
        held[page, :, at] = codes
        if step is not None:
            s["cache"][name + "_step"][page, :, at] = step
    return q


def _values(cache, name, index):
    """fp32 values of cache[name][index]."""
    held = cache[name]
    got = held.view(torch.uint8)[index].view(FP8).float() if held.dtype == FP8 else held[index].float()
    step = cache[name + "_step"]
    return got if step is None else got * step[index][..., None]


def _plain_attend(s):
    c = s["case"]
    B, Hkv, D, G = c["B"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    table = s["table"].long()
    keys, values = (_values(s["cache"], n, table).transpose(1, 2).reshape(B, Hkv, -1, D) for n in "kv")
    t, n = torch.arange(keys.shape[2], device="cuda")[None], s["lengths"].long()[:, None]
    there = (t < n) & (t >= n - c["window"]) if c["window"] else t < n
    x = s["q"].view(B, Hkv, G, D) @ keys.transpose(2, 3) * (1.0 / math.sqrt(D))
    x = torch.where(there[:, None, None], x, -math.inf)
    p = (x - x.amax(-1, keepdim=True)).exp()
    return (p @ values / p.sum(-1, keepdim=True)).view(B, c["Hq"], D)


# ---------------------------------------------------------------- one pass


def run(state):
    s, c = state, state["case"]
    if own:
        import bitlinear_w1_a8_gb300 as bl
        layout = bl.ROPE_INTERLEAVED if c.get("layout") == "interleaved" else bl.ROPE_HALF
    if c["op"] == "rope":
        if not own:
            return _rotated(s["x"], s["positions"], s["freq"], c["layout"], s["amplitude"])
        bl.bitlinear_rope(s["x"], s["positions"], (s["freq"], layout, s["amplitude"]), s["out"])
        return s["out"]
    h = s["cache"]
    cache = (h["k"], h["v"], h["k_step"], h["v_step"])
    if c["op"] == "append":
        if own:
            bl.bitlinear_kv_append(s["k"], s["v"], cache, s["positions"], s["table"], seq=s["seq"], q=s["q"], q_out=s["q_out"],
                                   rope=(s["freq"], layout, s["amplitude"]))
        q = s["q_out"] if own else _plain_append(s)
        return {"q": q, **{n: x for n, x in h.items() if x is not None}}
    if c["op"] == "read":
        if own:
            bl.bitlinear_kv_read(cache, s["positions"], s["table"], s["k_out"], s["v_out"], seq=s["seq"])
            return [s["k_out"], s["v_out"]]
        page, at = _places(s)
        return [_values(h, n, (page, slice(None), at)) for n in "kv"]
    if not own:
        return _plain_attend(s)
    bl.bitlinear_attention(s["q"], cache, s["table"], s["lengths"], s["out"], workspace=s.get("workspace"), window=c["window"])
    return s["out"]


def work(case):
    c = case
    size = {"int8": 1, "fp8": 1, "bf16": 2}[c.get("format", "bf16")]
    row = 2 * c["D"] * size + (8 if size == 1 else 0)  # a token's key and value of one head, with their steps
    if c["op"] == "rope":
        return {"bytes": 8 * c["T"] * c["H"] * c["D"] + 4 * c["T"], "flops": 3 * c["T"] * c["H"] * c["rot"]}
    if c["op"] == "append":
        return {"bytes": c["T"] * (8 * c["Hq"] * c["D"] + c["Hkv"] * (8 * c["D"] + row) + 8), "flops": c["T"] * c["D"] * (3 * c["Hq"] + 9 * c["Hkv"])}
    if c["op"] == "read":
        return {"bytes": c["T"] * (c["Hkv"] * (row + 8 * c["D"]) + 8), "flops": 2 * c["T"] * c["Hkv"] * c["D"]}
    tokens = c["B"] * (c["L"] if not c["ragged"] else (c["L"] + 1) / 2)
    if c["window"]:
        tokens = c["B"] * min(c["window"], c["L"]) if not c["ragged"] else c["B"] * sum(min(c["window"], n) for n in range(1, c["L"] + 1)) / c["L"]
    return {"bytes": tokens * c["Hkv"] * row + 8 * c["B"] * c["Hq"] * c["D"], "flops": 4 * tokens * c["Hq"] * c["D"]}


# ---------------------------------------------------------------- 64 bits


def _exact_rotation(x, positions, freq, layout, amplitude):
    """Every pair as a complex number times amplitude * exp(i * angle)."""
    n = freq.numel()
    head, rest = x[..., :2 * n].double(), x[..., 2 * n:].double()
    pairs = head.unflatten(-1, (n, 2)) if layout == "interleaved" else head.unflatten(-1, (2, n)).transpose(-1, -2)
    turn = torch.polar(torch.full_like(freq, amplitude).expand(len(positions), n), torch.outer(positions.double(), freq))
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
    return torch.cat([(z if layout == "interleaved" else z.transpose(-1, -2)).flatten(-2), rest], -1)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "rope":
        return _exact_rotation(s["x"], s["positions"], s["freq"], c["layout"], s["amplitude"])
    h = s["cache"]
    if c["op"] == "append":
        turned = {"k": _exact_rotation(s["k"], s["positions"], s["freq"], c["layout"], 1.0), "v": s["v"].double()}
        out = {"q": _exact_rotation(s["q"], s["positions"], s["freq"], c["layout"], 1.0), "k": None, "v": None}
        row = s["table"][s["seq"].long(), torch.div(s["positions"], c["page"], rounding_mode="floor").long()].long()
        for n, x in turned.items():
            if c["format"] == "bf16":  # the rows that the call writes, and the others as they were
                out[n] = h[n].double()
                out[n][row, :, (s["positions"] % c["page"]).long()] = x
            else:
                out[n + "_step"] = h[n + "_step"].double()
                out[n + "_step"][row, :, (s["positions"] % c["page"]).long()] = x.abs().amax(-1).clamp(min=1e-5) / TOP[c["format"]]
        return out

    def held(n, pages, at):  # [rows, Hkv, D]
        codes = (h[n].view(torch.uint8)[pages, :, at].view(FP8) if c["format"] == "fp8" else h[n][pages, :, at]).double()
        return codes if h[n + "_step"] is None else codes * h[n + "_step"][pages, :, at].double().unsqueeze(-1)

    if c["op"] == "read":
        pages = s["table"][s["seq"].long(), torch.div(s["positions"], c["page"], rounding_mode="floor").long()].long()
        return [held(n, pages, (s["positions"] % c["page"]).long()) for n in "kv"]
    rows = []
    for b in range(c["B"]):
        n = int(s["lengths"][b])
        t = torch.arange(max(0, n - c["window"]) if c["window"] else 0, n, device="cuda")
        k, v = (held(x, s["table"][b, t // c["page"]].long(), t % c["page"]) for x in "kv")
        q = s["q"][b].double().view(c["Hkv"], -1, c["D"])
        p = torch.softmax(torch.einsum("hgd,thd->hgt", q, k) / c["D"] ** 0.5, -1)
        rows.append(torch.einsum("hgt,thd->hgd", p, v).reshape(c["Hq"], c["D"]))
    return torch.stack(rows)
