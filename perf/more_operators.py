"""Measured cases of the paged key-value cache of a decode step: its writing, its reading back, and the attention over it.

A cache is two buffers of pages, keys and values, each [pages, page size, key-value heads, head size], in bf16 or in
e4m3 with one fp32 scale per token and head; a table gives each sequence its pages.  Three operators:

* ``write``: the keys and values of new tokens to their places, rounded to the cache's type;
* ``read``: the keys and values of a range of each sequence's positions as rows in the working type;
* ``attend``: attention of the newest tokens of each sequence (one, or a few drafted ones) over all it has in the
  cache; the output in the working type, the logarithm of the softmax's sum, and e4m3 codes for a product in 8 bits.

``run`` computes them in elementary torch operations where ``own`` is false, and through the library's entry
points where it is true.
"""
import math

import torch

own = False

BLOCK = 128          # columns of an output row that share a scale
E4M3_MAX = 448.0     # largest e4m3 value
MIN_AMAX = 2.0 ** -100  # a block's largest magnitude is taken as at least this

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------ cases
#
# length: tokens of the longest sequence, the new ones among them; spread: the others have down to (1 - spread) of
# that; new: new tokens of a sequence (ragged: one to that many, in buffers for that many each, whose last rows are
# then nobody's and stay as they were); rows: the working type

def listed():
    return [
        # one decoded token's keys and values into an 8-bit cache: latency of a few rows
        {"name": "write_decode", "op": "write", "seqs": 1, "kv_heads": 2, "head_dim": 256, "length": 1000, "spread": 0.0, "new": 1, "ragged": False, "page": 64, "cache": "e4m3", "rows": "bf16"},
        # the prompts of eight sequences, 2048 tokens at most, into an 8-bit cache: bandwidth
        {"name": "write_prompts", "op": "write", "seqs": 8, "kv_heads": 8, "head_dim": 128, "length": 2048, "spread": 0.0, "new": 2048, "ragged": False, "page": 64, "cache": "e4m3", "rows": "bf16"},
        # a short prefix back as rows
        {"name": "read_prefix", "op": "read", "seqs": 1, "kv_heads": 4, "head_dim": 80, "length": 333, "spread": 0.0, "new": 333, "ragged": False, "page": 17, "cache": "e4m3", "rows": "f32"},
        # long shared prefixes back for a prompt's attention: bandwidth
        {"name": "read_long", "op": "read", "seqs": 4, "kv_heads": 8, "head_dim": 128, "length": 8192, "spread": 0.0, "new": 8192, "ragged": False, "page": 64, "cache": "e4m3", "rows": "bf16"},
        # one token of one conversation: latency
        {"name": "attend_decode", "op": "attend", "seqs": 1, "heads": 16, "kv_heads": 2, "head_dim": 256, "length": 1000, "spread": 0.0, "new": 1, "ragged": False, "window": 0, "page": 64, "cache": "bf16",
         "rows": "bf16", "out": True, "lse": False, "codes": False},
        # one token over a very long context: the cache's length split over the whole GPU
        {"name": "attend_long", "op": "attend", "seqs": 1, "heads": 16, "kv_heads": 2, "head_dim": 256, "length": 131072, "spread": 0.0, "new": 1, "ragged": False, "window": 0, "page": 64, "cache": "e4m3",
         "rows": "bf16", "out": True, "lse": False, "codes": False},
        # a served batch of uneven conversations: bandwidth
        {"name": "attend_batch", "op": "attend", "seqs": 64, "heads": 32, "kv_heads": 8, "head_dim": 128, "length": 8192, "spread": 1.0, "new": 1, "ragged": False, "window": 0, "page": 64, "cache": "bf16",
         "rows": "bf16", "out": True, "lse": False, "codes": False},
        # the same with an 8-bit cache, the output as codes for an 8-bit projection
        {"name": "attend_batch_codes", "op": "attend", "seqs": 64, "heads": 32, "kv_heads": 8, "head_dim": 128, "length": 8192, "spread": 1.0, "new": 1, "ragged": False, "window": 0, "page": 64, "cache": "e4m3",
         "rows": "bf16", "out": False, "lse": False, "codes": True},
        # up to eight drafted tokens a sequence
        {"name": "attend_verify8", "op": "attend", "seqs": 16, "heads": 16, "kv_heads": 2, "head_dim": 128, "length": 16384, "spread": 0.5, "new": 8, "ragged": True, "window": 0, "page": 32, "cache": "bf16",
         "rows": "bf16", "out": True, "lse": False, "codes": False},
        # many short conversations of odd sizes, a sliding window, fp32 rows, the sums for joining with another part
        {"name": "attend_ragged", "op": "attend", "seqs": 200, "heads": 15, "kv_heads": 5, "head_dim": 80, "length": 517, "spread": 1.0, "new": 3, "ragged": True, "window": 301, "page": 17, "cache": "e4m3",
         "rows": "f32", "out": True, "lse": True, "codes": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "write", "read"])
    c = {"op": op, "seqs": _log(rng, 1, 256), "kv_heads": rng.choice([1, 2, 4, 8, 8, 16, rng.randint(1, 16)]), "head_dim": rng.choice([64, 128, 128, 256, 16 * rng.randint(1, 16)])}
    c["cache"], c["rows"] = rng.choice(["bf16", "e4m3"]), rng.choice(["bf16", "bf16", "f32"])
    c["page"] = rng.choice([16, 32, 64, 64, 256, rng.randint(1, 100)])
    token = c["kv_heads"] * c["head_dim"] * 2  # values a cached token has
    if op == "attend":
        c["heads"] = c["kv_heads"] * rng.choice([1, 2, 4, 8, rng.randint(1, 16)])
        c["new"] = rng.choice([1, 1, 1, rng.randint(2, 8)])
        # bytes, or operations where there are more of them, within those of the largest listed case
        per = token * max(TYPES[c["cache"]].itemsize, c["heads"] // c["kv_heads"] * c["new"] / 25.0)
        most = 1.0e9
    else:
        c["new"] = _log(rng, 1, 8192)
        per, most = token * 8.0, 2.0e8
        c["seqs"] = max(1, min(c["seqs"], int(most / per / c["new"])))
        c["new"] = max(1, min(c["new"], int(most / per)))
    top = max(c["new"] + 1, min(131072 if c["seqs"] == 1 else 16384, int(most / per / c["seqs"])))
    c["length"] = _log(rng, c["new"], top) if op == "attend" else c["new"] + rng.choice([0, rng.randint(0, 500)])
    c["spread"] = rng.choice([0.0, 0.5, 1.0])
    c["ragged"] = rng.random() < 0.4
    if op == "attend":
        c["window"] = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
        c["codes"] = c["head_dim"] % BLOCK == 0 and rng.random() < 0.3
        c["out"] = not c["codes"] or rng.random() < 0.5
        c["lse"] = rng.random() < 0.3
    return c


# ------------------------------------------------------------------ inputs

def _e4m3_heads(v):
    """(codes, scales) of fp32 rows, one scale per row."""
    scale = v.abs().amax(-1).clamp_min(MIN_AMAX) / E4M3_MAX
    return (v / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
    n, kv, d, page = case["seqs"], case["kv_heads"], case["head_dim"], case["page"]
    kind = TYPES[case["rows"]]
    share = torch.rand(n, generator=g, device=dev)
    share[0] = 0.0
    fresh = torch.randint(1, case["new"] + 1, (n,), generator=g, device=dev) if case["ragged"] else torch.full((n,), case["new"], device=dev)
    fresh[0] = case["new"]
    lens = torch.maximum((case["length"] * (1.0 - case["spread"] * share)).long(), fresh)
    lens[0] = case["length"]
    s = {"case": case, "lens": lens, "starts": (lens - fresh).to(torch.int32), "tokens": n * case["new"], "most_new": case["new"]}
    s["offsets"] = torch.cat([fresh.new_zeros(1), fresh.cumsum(0)]).to(torch.int32)
    # the pages that a sequence needs, handed out in no order; the table's other entries name no page
    each = -(-case["length"] // page)
    total = n * each
    order = torch.randperm(total + 1, generator=g, device=dev).to(torch.int32)  # one page at least is nobody's
    s["table"] = torch.where(torch.arange(each, device=dev)[None] < -(-lens // page)[:, None], order[:total].view(n, each), torch.full((), -1, dtype=torch.int32, device=dev)).contiguous()
    loud = torch.where(torch.rand(kv, d, generator=g, device=dev) < 0.02, 8.0, 1.0)  # a few channels of the keys are large, as in trained models
    shape = (total + 1, page, kv, d)
    if case["cache"] == "e4m3":
        s["k"], s["v"] = torch.empty(shape, dtype=TYPES["e4m3"], device=dev), torch.empty(shape, dtype=TYPES["e4m3"], device=dev)
        s["k_scale"], s["v_scale"] = torch.empty(shape[:3], device=dev), torch.empty(shape[:3], device=dev)
        for codes, scale, loudness in ((s["k"], s["k_scale"], loud), (s["v"], s["v_scale"], 1.0)):
            q, u = _e4m3_heads(randn(*shape) * loudness)
            codes.copy_(q)
            scale.copy_(u)
    else:
        s["k"], s["v"] = (randn(*shape) * loud).to(TYPES["bf16"]), randn(*shape).to(TYPES["bf16"])
        s["k_scale"] = s["v_scale"] = None
    if case["op"] == "attend":
        h = case["heads"]
        s["q"] = (1.5 * randn(s["tokens"], h, d)).to(kind)
        s["scale"] = 1.0 / math.sqrt(d)
        s["out"] = torch.zeros(s["tokens"], h, d, dtype=kind, device=dev) if case["out"] else None
        s["lse"] = torch.zeros(s["tokens"], h, device=dev) if case["lse"] else None
        s["codes"] = torch.zeros(s["tokens"], h * d, dtype=TYPES["e4m3"], device=dev) if case["codes"] else None
        s["codes_scale"] = torch.zeros(s["tokens"], h * d // BLOCK, device=dev) if case["codes"] else None
    elif case["op"] == "write":
        s["new_k"], s["new_v"] = (randn(s["tokens"], kv, d) * loud).to(kind), randn(s["tokens"], kv, d).to(kind)
    else:
        s["k_rows"], s["v_rows"] = torch.zeros(s["tokens"], kv, d, dtype=kind, device=dev), torch.zeros(s["tokens"], kv, d, dtype=kind, device=dev)
    return s


# ------------------------------------------------------------------ plain forms

def _token_places(s):
    """(token, page, slot) of each new token, in the order of the tokens."""
    off = s["offsets"].long()
    token = torch.arange(s["tokens"], device=off.device)
    token = token[token < off[-1]]
    seq = torch.searchsorted(off[1:].contiguous(), token, right=True)
    at = s["starts"].long()[seq] + token - off[seq]
    return token, s["table"].long()[seq, at // s["case"]["page"]], at % s["case"]["page"]


def _placed(rows, token, n):
    """[n, ...] with these rows at those tokens, zeros elsewhere."""
    all_rows = torch.zeros(n, *rows.shape[1:], dtype=rows.dtype, device=rows.device)
    all_rows[token] = rows
    return all_rows


def _plain_write(s):
    token, page, slot = _token_places(s)
    r = {}
    for name in ("k", "v"):
        rows = s["new_" + name][token].float()
        if s["k_scale"] is not None:
            codes, scale = _e4m3_heads(rows)
            s[name].view(torch.uint8)[page, slot] = codes.view(torch.uint8)
            s[name + "_scale"][page, slot] = scale
            r[name + "_scale"] = s[name + "_scale"]
        else:
            s[name][page, slot] = rows.to(s[name].dtype)
        r[name] = s[name]
    return r


def _wide(s, name, page, slot):
    """Cached rows in 32 bits."""
    rows = (s[name].view(torch.uint8)[page, slot].view(TYPES["e4m3"]) if s["k_scale"] is not None else s[name][page, slot]).float()
    return rows if s["k_scale"] is None else rows * s[name + "_scale"][page, slot][..., None]


def _plain_read(s):
    token, page, slot = _token_places(s)
    return {name: _placed(_wide(s, name, page, slot).to(s["k_rows"].dtype), token, s["tokens"]) for name in ("k", "v")}


def _plain_attend(s):
    c, dev = s["case"], s["table"].device
    kv, d, most = c["kv_heads"], c["head_dim"], s["most_new"]
    group = c["heads"] // kv
    off, starts, lens = s["offsets"].long(), s["starts"].long(), s["lens"]
    at = torch.arange(c["length"], device=dev)
    page = s["table"].long()[:, at // c["page"]].clamp_min(0)
    slot = (at % c["page"])[None].expand_as(page)
    there = at[None] < lens[:, None]
    token = off[:-1, None] + torch.arange(most, device=dev)[None]           # [seqs, new]
    real = token < off[1:, None]
    q = s["q"].float()[token.clamp_max(s["tokens"] - 1)]                    # [seqs, new, heads, d]
    q = q.view(-1, most, kv, group, d).permute(0, 2, 1, 3, 4).reshape(-1, kv, most * group, d)
    scores = q @ _wide(s, "k", page, slot).permute(0, 2, 3, 1) * s["scale"]   # [seqs, kv, new * group, length]
    last = starts[:, None] + torch.arange(most, device=dev)[None]           # a token's own position
    seen = there[:, None] & (at[None, None] <= last[..., None])             # [seqs, new, length]
    if c["window"]:
        seen = seen & (at[None, None] > last[..., None] - c["window"])
    seen = seen.repeat_interleave(group, 1)[:, None]
    scores = torch.where(seen, scores, torch.full((), -math.inf, device=dev))
    top = scores.amax(-1, keepdim=True).clamp_min(-3.0e38)
    weight = torch.exp(scores - top)
    total = weight.sum(-1, keepdim=True)
    out = weight @ _wide(s, "v", page, slot).permute(0, 2, 1, 3) / total
    back = lambda v: _placed(v.view(-1, kv, most, group, v.shape[-1]).permute(0, 2, 1, 3, 4).reshape(-1, most, kv * group, v.shape[-1])[real], token[real], s["tokens"])  # noqa: E731
    r, out = {}, back(out)
    if s["out"] is not None:
        r["out"] = out.to(s["out"].dtype)
    if s["lse"] is not None:
        r["lse"] = back(top + torch.log(total))[..., 0]
    if s["codes"] is not None:
        codes, scale = _e4m3_heads(out.reshape(s["tokens"], -1, BLOCK))
        r["codes"], r["codes_scale"] = codes.reshape(s["tokens"], -1), torch.where(torch.arange(s["tokens"], device=dev)[:, None] < off[-1], scale, torch.zeros((), device=dev))
    return r


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend}[op](s)
    from bit_quantized_moe_router_gb300 import qs_moe as qm
    if "cache" not in s:  # the program's own, kept between calls
        s["cache"] = qm.make_cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["seqs"] = qm.make_seqs(s["table"], s["starts"], s["offsets"])
        if op == "attend":
            s["workspace"] = qm.alloc_cache_attention_workspace(s["case"]["heads"], s["case"]["kv_heads"], s["case"]["head_dim"], s["most_new"])
    if op == "write":
        qm.qs_cache_write(s["cache"], s["seqs"], s["new_k"], s["new_v"])
        return {k: s[k] for k in ("k", "v", "k_scale", "v_scale") if s[k] is not None}
    if op == "read":
        qm.qs_cache_read(s["cache"], s["seqs"], s["k_rows"], s["v_rows"])
        return {"k": s["k_rows"], "v": s["v_rows"]}
    qm.qs_cache_attention(s["cache"], s["seqs"], s["q"], s["scale"], s["out"], s["workspace"], max_new=s["most_new"], window=s["case"]["window"], lse=s["lse"],
                          codes=s["codes"], codes_scale=s["codes_scale"])
    return {k: s[k] for k in ("out", "lse", "codes", "codes_scale") if s[k] is not None}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    kv, d, page = case["kv_heads"], case["head_dim"], case["page"]
    fresh = (1 + case["new"]) / 2.0 if case["ragged"] else float(case["new"])
    length = max(fresh, case["length"] * (1.0 - case["spread"] / 2.0))
    tokens = int(case["seqs"] * fresh)
    cached = d * TYPES[case["cache"]].itemsize + (4 if case["cache"] == "e4m3" else 0)  # a token and head, keys or values
    z = TYPES[case["rows"]].itemsize
    if case["op"] != "attend":
        return {"bytes": int(2 * tokens * kv * (d * z + cached) + 4 * tokens / page + 8 * case["seqs"]), "flops": 2 * tokens * kv * d * 2}
    seen = min(length, case["window"] + fresh - 1) if case["window"] else length
    rows = tokens * case["heads"]
    b = 2 * case["seqs"] * seen * kv * cached + rows * d * z + 4 * case["seqs"] * (2 + seen / page)
    b += (rows * d * z if case["out"] else 0) + (4 * rows if case["lse"] else 0) + (rows * d * (1 + 4 / BLOCK) if case["codes"] else 0)
    return {"bytes": int(b), "flops": int(4 * rows * d * (min(length, case["window"]) if case["window"] else length))}


# ------------------------------------------------------------------ the definitions in 64 bits

def _nearest_e4m3(v):
    """v (64 bits) rounded to the nearest e4m3 value, ties to even: 3 bits after the leading one, exponents from -6."""
    exponent = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -20)))
    step = torch.exp2(exponent.clamp_min(-6.0) - 3.0)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_codes(v):
    amax = v.abs().max(-1).values
    scale = torch.maximum(amax, torch.full_like(amax, MIN_AMAX)) / E4M3_MAX
    return _nearest_e4m3(v / scale.unsqueeze(-1)), scale


def exact(case, seed):
    s = prepare(case, seed)
    page, eight = case["page"], case["cache"] == "e4m3"
    offsets, starts, lens = s["offsets"].tolist(), s["starts"].tolist(), s["lens"].tolist()

    def cached(name, i, lo, hi):
        """Positions lo .. hi - 1 of sequence i, [positions, kv_heads, head_dim]."""
        pages = s["table"][i, lo // page: -(-hi // page)].long()
        rows = s[name].view(torch.uint8)[pages].view(TYPES["e4m3"]).double() if eight else s[name][pages].double()
        if eight:
            rows = rows * s[name + "_scale"][pages].double()[..., None]
        return rows.flatten(0, 1)[lo % page: lo % page + hi - lo]

    def whole(rows):
        """The rows of the sequences' tokens with those behind them, which stay zeros."""
        return torch.cat([rows, rows.new_zeros(s["tokens"] - rows.shape[0], *rows.shape[1:])])

    if case["op"] == "write":
        r = {name: s[name].double() for name in ("k", "v")}
        if eight:
            r.update({name + "_scale": s[name + "_scale"].double() for name in ("k", "v")})
        for i in range(case["seqs"]):
            at = torch.arange(starts[i], lens[i], device="cuda")
            where = s["table"][i].long()[at // page], at % page
            for name in ("k", "v"):
                rows = s["new_" + name][offsets[i]: offsets[i + 1]].double()
                if eight:
                    rows, r[name + "_scale"][where] = _exact_codes(rows)
                r[name][where] = rows
        return r
    if case["op"] == "read":
        return {name: whole(torch.cat([cached(name, i, starts[i], lens[i]) for i in range(case["seqs"])])) for name in ("k", "v")}
    group = case["heads"] // case["kv_heads"]
    outs, sums = [], []
    for i in range(case["seqs"]):
        first = max(0, starts[i] + 1 - case["window"]) if case["window"] else 0
        k, v = cached("k", i, first, lens[i]).repeat_interleave(group, 1), cached("v", i, first, lens[i]).repeat_interleave(group, 1)
        for j in range(offsets[i + 1] - offsets[i]):
            hi = starts[i] + j + 1 - first
            lo = max(0, hi - case["window"]) if case["window"] else 0
            logits = torch.einsum("hd,lhd->hl", s["q"][offsets[i] + j].double(), k[lo:hi]) * s["scale"]
            sums.append(torch.logsumexp(logits, 1))
            outs.append(torch.einsum("hl,lhd->hd", torch.softmax(logits, 1), v[lo:hi]))
    out, r = torch.stack(outs), {}
    if case["out"]:
        r["out"] = whole(out)
    if case["lse"]:
        r["lse"] = whole(torch.stack(sums))
    if case["codes"]:
        codes, scale = _exact_codes(out.flatten(1).unflatten(1, (-1, BLOCK)))
        r["codes"], r["codes_scale"] = whole(codes.flatten(1)), whole(scale)
    return r
