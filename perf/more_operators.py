"""What is measured of the serving operators: attention of rows that share a prefix, attention over chosen
blocks of the cache (their summaries, the choice, the attention), probabilities of logits, and the
verification of drafted tokens.

Every case has one operator ("op") and its sizes.  ``own`` false: the operators in elementary torch
operations; true: the calls a program makes of this package.
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
TOP = {"int8": 127.0, "fp8": 448.0}


# ---------------------------------------------------------------- cases


def listed():
    return [
        # two answers to one short question begin: latency alone
        {"name": "shared_pair_int8", "op": "shared", "groups": 1, "R": 2, "Hq": 16, "Hkv": 16, "D": 128, "S": 37, "own": 1, "ragged": False, "page": 32, "format": "int8"},
        # drafted tokens of eight sequences of different ages: the five rows of each share its pages, every one sees a token more
        {"name": "shared_drafts_int8", "op": "shared", "groups": 8, "R": 5, "Hq": 32, "Hkv": 32, "D": 80, "S": 2048, "own": 5, "ragged": True, "page": 64, "format": "int8"},
        # a served batch behind one system prompt, answers of different lengths
        {"name": "shared_prompt_int8", "op": "shared", "groups": 1, "R": 64, "Hq": 32, "Hkv": 32, "D": 80, "S": 2039, "own": 256, "ragged": True, "page": 64, "format": "int8"},
        # one long document, many questions, heads that share keys
        {"name": "shared_document_bf16", "op": "shared", "groups": 1, "R": 64, "Hq": 32, "Hkv": 8, "D": 128, "S": 16384, "own": 100, "ragged": True, "page": 64, "format": "bf16"},
        # three prompts are cached, odd lengths: the summaries of all of their pages
        {"name": "summarise_prompts_int8", "op": "summarise", "B": 3, "Hkv": 32, "D": 80, "L": 2039, "page": 64, "format": "int8"},
        # a decode step of one sequence whose context is still short
        {"name": "sparse_short_fp8", "op": "sparse", "B": 1, "Hq": 16, "Hkv": 16, "D": 128, "L": 700, "count": 8, "ragged": False, "page": 32, "format": "fp8"},
        # a served batch of long sequences of different ages, 2048 tokens of each attended to
        {"name": "sparse_batch_int8", "op": "sparse", "B": 16, "Hq": 32, "Hkv": 32, "D": 80, "L": 16384, "count": 32, "ragged": True, "page": 64, "format": "int8"},
        # one very long sequence, 4096 of its tokens attended to
        {"name": "sparse_long_bf16", "op": "sparse", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "L": 131071, "count": 64, "ragged": False, "page": 64, "format": "bf16"},
        # the LM head's logits of one token
        {"name": "softmax_token", "op": "softmax", "M": 1, "V": 50000, "warm": True},
        # of 64 sequences with four drafted tokens each, every sequence with a temperature of its own
        {"name": "softmax_drafts", "op": "softmax", "M": 320, "V": 50000, "warm": True},
        # one sequence's four drafted tokens
        {"name": "verify_one", "op": "verify", "B": 1, "K": 4, "V": 50000},
        # those of 64 sequences
        {"name": "verify_batch", "op": "verify", "B": 64, "K": 4, "V": 50000},
    ]


def _spread(rng, lo, hi):
    """An integer of lo..hi, even over its logarithm, odd ones among them."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "sparse", "sparse", "summarise", "softmax", "verify"])
    D = rng.choice([64, 80, 96, 112, 128])
    fmt, page = rng.choice(["int8", "fp8", "bf16"]), rng.choice([16, 32, 64, 128])
    Hkv, G = rng.choice([1, 2, 4, 5, 8, 16, 32]), rng.choice([1, 1, 2, 4, 7, 8])
    if Hkv * G > 64:
        G = 1
    if op == "shared":
        R = _spread(rng, 1, 64)
        groups = _spread(rng, 1, max(1, 64 // R))
        B, codes = groups * R, Hkv * D * (2 if fmt == "bf16" else 1)
        most = min((1 << 32) // (B * Hkv * G * D), (1 << 25) // (groups * codes))  # products and bytes of a pass: below the largest listed cases'
        S, mine = _spread(rng, 1, max(1, min(16384, most))), _spread(rng, 1, max(1, min(300, (1 << 24) // (B * codes))))
        return {"op": op, "groups": groups, "R": R, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "S": S, "own": mine, "ragged": rng.random() < 0.6,
                "page": page, "format": fmt}
    if op == "summarise":
        B = _spread(rng, 1, 16)
        return {"op": op, "B": B, "Hkv": Hkv, "D": D, "L": _spread(rng, 1, 16384 // B), "page": page, "format": fmt}
    if op == "sparse":
        B = _spread(rng, 1, 16)
        L = _spread(rng, 1, min(131072, (1 << 28) // (B * Hkv * D)))  # tokens a sequence: below the largest listed case
        most = min(64, -(-L // page), (1 << 24) // (B * Hkv * D * page))
        return {"op": op, "B": B, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "L": L, "count": _spread(rng, 2, max(2, most)), "ragged": rng.random() < 0.6,
                "page": page, "format": fmt}
    V = _spread(rng, 1000, 130000)
    if op == "softmax":
        return {"op": op, "M": _spread(rng, 1, 16_000_000 // V), "V": V, "warm": rng.random() < 0.5}
    K = _spread(rng, 1, 8)
    return {"op": op, "B": _spread(rng, 1, min(64, 16_000_000 // (V * (K + 1)))), "K": K, "V": V}


# ---------------------------------------------------------------- inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _host_ints(seed, lo, hi, n):
    """n whole numbers of lo..hi on the host."""
    g = torch.Generator()
    g.manual_seed(int(seed))
    return torch.randint(lo, hi + 1, (n,), generator=g, dtype=torch.int32)


def _quantised(x, fmt):
    """fp32 rows [..., D] -> what a cache of the format holds, and the rows' steps."""
    if fmt == "bf16":
        return x.to(torch.bfloat16), None
    top = x.abs().amax(-1).clamp(min=1e-5)
    scaled = x * (TOP[fmt] / top)[..., None]
    codes = scaled.round().clamp(-128, 127).to(torch.int8) if fmt == "int8" else scaled.clamp(-448, 448).to(FP8)
    return codes, top / TOP[fmt]


def _pool(g, c, pages):
    """Keys and values of `pages` pages: channels of different size, as projections give them, and keys of a page
    that resemble one another, as those of one passage do."""
    shape = (pages, c["Hkv"], c["page"], c["D"])
    size = torch.rand(c["Hkv"], 1, c["D"], generator=g, device="cuda") * 1.5 + 0.25
    out = {}
    for name in "kv":
        x = torch.randn(shape, generator=g, device="cuda")
        if name == "k":
            x = 0.8 * x + 0.6 * torch.randn(pages, c["Hkv"], 1, c["D"], generator=g, device="cuda")
        out[name], out[name + "_step"] = _quantised(x * size, c["format"])
        del x
    return out


def _rows(g, B, width):
    """Every sequence's pages, in no order."""
    return torch.randperm(B * width, generator=g, device="cuda").to(torch.int32).view(B, width)


def prepare(case, seed):
    c, g = dict(case), _generator(seed)
    s = {"case": c}
    if c["op"] == "shared":
        groups, R, page = c["groups"], c["R"], c["page"]
        B = groups * R
        shared = _host_ints(seed, max(1, c["S"] // 2), c["S"], groups) if c["ragged"] and groups > 1 else torch.full((groups,), c["S"], dtype=torch.int32)
        drafts = c["own"] == R and groups > 1  # the rows of a sequence see one token more each, and share all of its pages
        if drafts:
            more = torch.arange(1, R + 1, dtype=torch.int32).repeat(groups)
        else:
            more = _host_ints(seed + 1, 1, c["own"], B) if c["ragged"] else torch.full((B,), c["own"], dtype=torch.int32)
        lengths = shared.repeat_interleave(R) + more
        if drafts:
            shared = shared + R
        # a page table as a serving program keeps it: whole pages of the prefix are one and the same, later ones a row's own
        whole, width = c["S"] // page, -(-(c["S"] + c["own"]) // page)
        tail = width - whole
        ids = torch.randperm(groups * whole + B * tail, generator=g, device="cuda").to(torch.int32)
        table = torch.cat([ids[:groups * whole].view(groups, 1, whole).expand(-1, R, -1).reshape(B, whole), ids[groups * whole:].view(B, tail)], 1)
        # where a prefix ends before its last whole pages, or inside a page, those pages are the group's first row's
        ends = torch.div(shared + page - 1, page, rounding_mode="floor").cuda().repeat_interleave(R)
        first_row = table.view(groups, R, width)[:, :1].expand(-1, R, -1).reshape(B, width)
        columns = torch.arange(width, device="cuda")[None]
        s["table"] = torch.where(columns < ends[:, None], first_row, table).contiguous()
        s["cache"] = _pool(g, c, groups * whole + B * tail)
        s["shared"], s["lengths"] = shared.cuda(), lengths.cuda()
        s["most"], s["most_own"] = int(shared.max()), 1 if drafts else int(more.max())
        s["q"] = torch.randn(B, c["Hq"], c["D"], generator=g, device="cuda") * 1.5
        s["out"] = torch.empty_like(s["q"])
        s["workspace"] = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
        return s
    if c["op"] == "summarise":
        width = -(-c["L"] // c["page"])
        s["cache"], s["table"] = _pool(g, c, c["B"] * width), _rows(g, c["B"], width)
        s["lengths"] = _host_ints(seed, max(1, c["L"] * 3 // 4), c["L"], c["B"]).cuda()
        s["first"] = torch.zeros_like(s["lengths"])
        s["bounds"] = torch.zeros(c["B"] * width, c["Hkv"], 2, c["D"], dtype=torch.int8, device="cuda")
        s["step"] = torch.zeros(c["B"] * width, c["Hkv"], device="cuda")
        return s
    if c["op"] == "sparse":
        width = -(-c["L"] // c["page"])
        s["cache"], s["table"] = _pool(g, c, c["B"] * width), _rows(g, c["B"], width)
        lengths = _host_ints(seed, max(1, c["L"] // 4), c["L"], c["B"]) if c["ragged"] else torch.full((c["B"],), c["L"], dtype=torch.int32)
        s["lengths"] = lengths.cuda()
        # every page but a sequence's last was summarised when it filled; the last one's summary is of the step before
        s["bounds"], s["step"] = _summaries(s["cache"], torch.arange(c["B"] * width, device="cuda"), torch.full((c["B"] * width,), c["page"], device="cuda"))
        s["first"] = s["lengths"] - 1
        s["q"] = torch.randn(c["B"], c["Hq"], c["D"], generator=g, device="cuda") * 1.5
        s["blocks"] = torch.empty(c["B"], c["Hkv"], c["count"], dtype=torch.int32, device="cuda")
        s["out"] = torch.empty_like(s["q"])
        return s
    if c["op"] == "softmax":
        s["y"] = torch.randn(c["M"], c["V"], generator=g, device="cuda") * 2.5
        s["temperature"] = (torch.rand(c["M"], generator=g, device="cuda") * 1.2 + 0.3) if c["warm"] else None
        s["p"] = torch.empty_like(s["y"])
        return s
    B, K, V = c["B"], c["K"], c["V"]
    y = torch.randn(B, K + 1, V, generator=g, device="cuda") * 2.5
    s["p"] = torch.softmax(y, -1)
    s["q"] = torch.softmax(y[:, :K] + 0.5 * torch.randn(B, K, V, generator=g, device="cuda"), -1)  # a draft model that is near
    s["draft"] = torch.multinomial(s["q"].view(B * K, V), 1, generator=g).view(B, K).to(torch.int32)
    s["uniform"] = torch.rand(B, K + 1, generator=g, device="cuda")
    s["tokens"] = torch.empty(B, K + 1, dtype=torch.int32, device="cuda")
    s["accepted"] = torch.empty(B, dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms


def _values(cache, name, index):
    """fp32 values of cache[name][index]."""
    held, step = cache[name], cache[name + "_step"]
    got = held.view(torch.uint8)[index].view(FP8).float() if held.dtype == FP8 else held[index].float()
    return got if step is None else got * step[index][..., None]


def _tokens(cache, name, table, t, page):
    """fp32 values [..., n, Hkv, D] of the tokens t [..., n] of the sequences whose pages `table` [..., columns] lists."""
    column = torch.div(t, page, rounding_mode="floor").clamp(max=table.shape[-1] - 1)
    return _values(cache, name, (table.long().gather(-1, column), slice(None), t % page))


def _summaries(cache, pages, filled):
    """Bounds of the keys of `pages` [n], of which the first `filled` [n] tokens are there: codes [n, Hkv, 2, D], steps [n, Hkv]."""
    x = _values(cache, "k", pages)
    there = (torch.arange(x.shape[2], device="cuda")[None] < filled[:, None])[:, None, :, None]
    lo, hi = torch.where(there, x, math.inf).amin(2), torch.where(there, x, -math.inf).amax(2)
    top = torch.maximum(lo.abs(), hi.abs()).amax(-1).clamp(min=1e-5)
    s = (torch.full_like(top, 127.0) / top)[..., None]
    codes = torch.stack([(lo * s).floor().clamp(-127, 127), (hi * s).ceil().clamp(-127, 127)], 2)
    return codes.to(torch.int8), top / torch.full_like(top, 127.0)


def _plain_summarise(s):
    """Writes the summaries of the pages that hold tokens first .. lengths - 1."""
    page, table = s["case"]["page"], s["table"].long()
    column = torch.arange(table.shape[1], device="cuda")[None]
    n, first = s["lengths"].long()[:, None], s["first"].long()[:, None]
    touched = (column * page < n) & ((column + 1) * page > first)
    ids, filled = table[touched], (n - column * page).clamp(max=page)[touched]
    s["bounds"][ids], s["step"][ids] = _summaries(s["cache"], ids, filled)


def _plain_select(s):
    c = s["case"]
    B, Hkv, D, page, count = c["B"], c["Hkv"], c["D"], c["page"], c["count"]
    top = s["q"].abs().amax(-1).clamp(min=1e-5)
    codes = (s["q"] * (torch.full_like(top, 127.0) / top)[..., None]).round().clamp(-127, 127).view(B, Hkv, -1, D)
    q_step = (top / torch.full_like(top, 127.0)).view(B, Hkv, -1, 1)
    bounds = s["bounds"][s["table"].long()].transpose(1, 2).double()  # whole numbers, their sums as well
    acc = codes.clamp(min=0).double() @ bounds[..., 1, :].transpose(2, 3) + codes.clamp(max=0).double() @ bounds[..., 0, :].transpose(2, 3)
    score = ((acc.float() * s["step"][s["table"].long()].transpose(1, 2)[:, :, None]) * q_step).amax(2)  # [B, Hkv, columns]
    j = torch.arange(score.shape[-1], device="cuda")[None, None]
    blocks = torch.div(s["lengths"].long() + page - 1, page, rounding_mode="floor")[:, None, None]
    score = torch.where((j < 1) | (j == blocks - 1), math.inf, score)
    score = torch.where(j < blocks, score, -math.inf)
    order = score.sort(dim=-1, descending=True, stable=True).indices[..., :count]
    order = torch.where(order < blocks, order, score.shape[-1]).sort(-1).values
    s["blocks"].fill_(-1)
    s["blocks"][..., :order.shape[-1]] = torch.where(order < blocks, order, -1)


def _attend(x, there, values):
    """softmax over the last dim of x where `there`, times values -> (out, maximum, sum)."""
    x = torch.where(there, x, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (x - m).exp()
    return p @ values, m, p.sum(-1, keepdim=True)


def _plain_blocks(s):
    c = s["case"]
    B, Hkv, D, page = c["B"], c["Hkv"], c["D"], c["page"]
    blocks = s["blocks"].long()
    pages = s["table"].long()[:, None].expand(-1, Hkv, -1).gather(-1, blocks.clamp(min=0))
    head = torch.arange(Hkv, device="cuda")[None, :, None]
    k, v = (_values(s["cache"], n, (pages, head)).reshape(B, Hkv, -1, D) for n in "kv")
    t = blocks[..., None] * page + torch.arange(page, device="cuda")
    there = ((blocks[..., None] >= 0) & (t < s["lengths"].long()[:, None, None, None])).view(B, Hkv, 1, -1)
    out, _, total = _attend(s["q"].view(B, Hkv, -1, D) @ k.transpose(2, 3) * (1.0 / math.sqrt(D)), there, v)
    return (out / total).reshape(B, c["Hq"], D)


def _plain_shared(s):
    c = s["case"]
    groups, R, Hkv, D, page = c["groups"], c["R"], c["Hkv"], c["D"], c["page"]
    G, B, scale = c["Hq"] // Hkv, groups * R, 1.0 / math.sqrt(D)
    # the prefix of a group, once for all of its rows
    t = torch.arange(s["most"], device="cuda").expand(groups, -1)
    k, v = (_tokens(s["cache"], n, s["table"][::R], t, page).transpose(1, 2) for n in "kv")
    q = s["q"].view(groups, R, Hkv, G, D).transpose(1, 2).reshape(groups, Hkv, R * G, D)
    limits = torch.minimum(s["lengths"].view(groups, R), s["shared"][:, None]).repeat_interleave(G, 1)  # of a key head's rows
    there = (t[:, None] < limits.long()[..., None])[:, None]
    a, ma, za = (x.reshape(groups, Hkv, R, G, -1).transpose(1, 2).reshape(B, Hkv, G, -1) for x in _attend(q @ k.transpose(2, 3) * scale, there, v))
    # each row's own tokens
    t = s["shared"].long().repeat_interleave(R)[:, None] + torch.arange(s["most_own"], device="cuda")
    k, v = (_tokens(s["cache"], n, s["table"], t, page).transpose(1, 2) for n in "kv")
    there = (t < s["lengths"].long()[:, None])[:, None, None]
    b, mb, zb = _attend(s["q"].view(B, Hkv, G, D) @ k.transpose(2, 3) * scale, there, v)
    m = torch.maximum(ma, mb)
    fa, fb = (ma - m).exp(), (mb - m).exp()
    return ((a * fa + b * fb) / (za * fa + zb * fb)).reshape(B, c["Hq"], D)


def _plain_softmax(s):
    y = s["y"]
    z = y - y.amax(-1, keepdim=True)
    e = (z if s["temperature"] is None else z / s["temperature"][:, None]).exp()
    return e / e.sum(-1, keepdim=True)


def _plain_verify(s):
    c = s["case"]
    K, V = c["K"], c["V"]
    x = s["draft"].long()
    px, qx = s["p"][:, :K].gather(-1, x[..., None])[..., 0], s["q"].gather(-1, x[..., None])[..., 0]
    n = (s["uniform"][:, :K].double() * qx.double() < px.double()).long().cumprod(1).sum(1)
    row = torch.arange(c["B"], device="cuda")
    p, q = s["p"][row, n], s["q"][row, n.clamp(max=K - 1)]
    rest = (p - q).clamp(min=0)
    w = torch.where(((n < K) & (rest > 0).any(-1))[:, None], rest, p).double()
    upto = w.cumsum(-1)
    token = (upto <= s["uniform"][:, K:].double() * upto[:, -1:]).sum(-1).clamp(max=V - 1)
    i = torch.arange(K + 1, device="cuda")[None]
    s["tokens"].copy_(torch.where(i < n[:, None], torch.nn.functional.pad(x, (0, 1)), torch.where(i == n[:, None], token[:, None], -1)))
    s["accepted"].copy_(n)


# ---------------------------------------------------------------- one pass


def run(state):
    s, c = state, state["case"]
    if own:
        import bitlinear_w1_a8_gb300 as bl
    if c["op"] == "softmax":
        if not own:
            return _plain_softmax(s)
        bl.bitlinear_softmax(s["y"], s["p"], s["temperature"])
        return s["p"]
    if c["op"] == "verify":
        if own:
            bl.bitlinear_verify(s["p"], s["q"], s["draft"], s["uniform"], s["tokens"], s["accepted"])
        else:
            _plain_verify(s)
        return [s["tokens"], s["accepted"]]
    h = s["cache"]
    cache = (h["k"], h["v"], h["k_step"], h["v_step"])
    if c["op"] == "shared":
        if not own:
            return _plain_shared(s)
        bl.bitlinear_attention_shared(s["q"], cache, s["table"], s["lengths"], s["shared"], s["out"], s["workspace"])
        return s["out"]
    if own:
        bl.bitlinear_kv_summarise(cache, (s["bounds"], s["step"]), s["table"], s["first"], s["lengths"])
    else:
        _plain_summarise(s)
    if c["op"] == "summarise":
        return [s["bounds"], s["step"]]
    if own:
        bl.bitlinear_attention_select(s["q"], cache, (s["bounds"], s["step"]), s["table"], s["lengths"], s["blocks"], keep_first=1, keep_last=1)
        bl.bitlinear_attention_blocks(s["q"], cache, s["table"], s["lengths"], s["blocks"], s["out"])
        out = s["out"]
    else:
        _plain_select(s)
        out = _plain_blocks(s)
    return {"bounds": s["bounds"], "step": s["step"], "blocks": s["blocks"], "out": out}


def work(case):
    c = case
    if c["op"] == "softmax":
        return {"bytes": 8 * c["M"] * c["V"], "flops": 4 * c["M"] * c["V"]}
    if c["op"] == "verify":
        return {"bytes": c["B"] * (8 * c["V"] + 20 * c["K"]), "flops": 3 * c["B"] * c["V"]}
    size = {"int8": 1, "fp8": 1, "bf16": 2}[c["format"]]
    D, Hkv, page = c["D"], c["Hkv"], c["page"]
    key = D * size + (4 if size == 1 else 0)  # a token's key of one head, with its step
    if c["op"] == "shared":
        S = c["S"] * (0.75 if c["ragged"] and c["groups"] > 1 else 1.0)
        mine = (c["own"] + 1) / 2 if c["ragged"] or (c["own"] == c["R"] and c["groups"] > 1) else c["own"]
        B = c["groups"] * c["R"]
        return {"bytes": (c["groups"] * S + B * mine) * Hkv * 2 * key + 8 * B * c["Hq"] * D, "flops": 4 * B * c["Hq"] * D * (S + mine)}
    if c["op"] == "summarise":
        tokens = c["B"] * c["L"] * 0.875
        return {"bytes": tokens * Hkv * key + tokens / page * Hkv * (2 * D + 4), "flops": 3 * tokens * Hkv * D}
    tokens = c["L"] * (0.625 if c["ragged"] else 1.0)
    blocks, chosen = tokens / page, min(tokens, c["count"] * page)
    return {"bytes": c["B"] * (Hkv * (page * key + blocks * (2 * D + 4) + chosen * 2 * key) + 8 * c["Hq"] * D),
            "flops": c["B"] * c["Hq"] * D * (2 * blocks + 4 * chosen)}


# ---------------------------------------------------------------- 64 bits


def _exact_rows(cache, fmt, name, pages, at):
    """float64 values [n, Hkv, D] of the tokens at (pages, at)."""
    codes = cache[name].view(torch.uint8)[pages, :, at].view(FP8) if fmt == "fp8" else cache[name][pages, :, at]
    codes = codes.double()
    return codes if cache[name + "_step"] is None else codes * cache[name + "_step"][pages, :, at].double().unsqueeze(-1)


def _exact_attention(q, k, v):
    """q [Hq, D], k and v [n, Hkv, D], float64."""
    x = torch.einsum("hgd,thd->hgt", q.view(k.shape[1], -1, k.shape[2]), k) / k.shape[2] ** 0.5
    return torch.einsum("hgt,thd->hgd", torch.softmax(x, -1), v).reshape(q.shape)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "softmax":
        y = s["y"].double()
        return torch.softmax(y if s["temperature"] is None else y / s["temperature"].double()[:, None], -1)
    if c["op"] == "verify":
        return None  # whole numbers
    fmt, page, h = c["format"], c["page"], s["cache"]
    if c["op"] == "shared":
        rows = []
        for b in range(c["groups"] * c["R"]):
            t = torch.arange(int(s["lengths"][b]), device="cuda")
            k, v = (_exact_rows(h, fmt, n, s["table"][b, t // page].long(), t % page) for n in "kv")
            rows.append(_exact_attention(s["q"][b].double(), k, v))
        return torch.stack(rows)
    step = s["step"].double()
    for b in range(c["B"]):
        n = int(s["lengths"][b])
        for col in range(int(s["first"][b]) // page, -(-n // page)):
            at = torch.arange(min(page, n - col * page), device="cuda")
            x = _exact_rows(h, fmt, "k", s["table"][b, col].long().expand(len(at)), at)
            step[s["table"][b, col].long()] = x.abs().amax((0, 2)).clamp(min=1e-5) / 127
    if c["op"] == "summarise":
        return [None, step]
    # the attention over the blocks that the definition chooses: its own sum of whole numbers and rounding of scores
    _plain_summarise(s)
    out = torch.empty(c["B"], c["Hq"], c["D"], dtype=torch.float64, device="cuda")
    G = c["Hq"] // c["Hkv"]
    for b in range(c["B"]):
        n = int(s["lengths"][b])
        cols = torch.arange(-(-n // page), device="cuda")
        ids = s["table"][b, cols].long()
        for hk in range(c["Hkv"]):
            q = s["q"][b, hk * G:(hk + 1) * G]
            top = q.abs().amax(-1).clamp(min=1e-5)
            codes = torch.round(q * (torch.full_like(top, 127.0) / top)[:, None]).double()
            lo, hi = s["bounds"][ids, hk].double().unbind(1)
            bound = torch.maximum(codes[:, None] * lo, codes[:, None] * hi).sum(-1)
            score = ((bound * s["step"][ids, hk].double()).float().double() * (top.double() / 127).float().double()[:, None]).float().amax(0)
            score[0] = score[-1] = math.inf
            chosen = score.sort(dim=-1, descending=True, stable=True).indices[:c["count"]]
            t = (chosen[:, None] * page + torch.arange(page, device="cuda")).flatten()
            t = t[t < n]
            k, v = (_exact_rows(h, fmt, x, s["table"][b, t // page].long(), t % page)[:, hk:hk + 1] for x in "kv")
            out[b, hk * G:(hk + 1) * G] = _exact_attention(q.double(), k, v)
    return {"bounds": None, "step": step, "blocks": None, "out": out}
