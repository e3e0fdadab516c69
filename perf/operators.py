"""Measured cases of the operators around 8-bit mixture-of-experts products.

Four operators that stand next to the layer of this library, from the residual stream to the experts' rows and back:

* ``norm`` / ``norm_backward``: root-mean-square norm with the residual's addition, its output in the
  working type and in e4m3 with one scale per row and 128 columns; and its gradient;
* ``matmul`` / ``grouped``: products of e4m3 rows (one scale per row and 128 columns) with e4m3 weights (one scale
  per 128 x 128 block), for one matrix and for rows sorted by expert;
* ``route`` / ``route_train``: token rows sorted by expert, and the experts' rows weighted and summed back; with
  ``route_train`` the gradients of both;
* ``silu``: silu(gate) * up of the gate/up product, its output in e4m3 with scales.

``run`` computes them in elementary torch operations where ``own`` is false, and through the library's entry
points where it is true.
"""
import math

import torch

own = False

BLOCK = 128          # columns (and weight rows) that share a scale
E4M3_MAX = 448.0     # largest e4m3 value
MIN_AMAX = 2.0 ** -100  # a block's largest magnitude is taken as at least this
EPS = 1e-6

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token between attention and the FFN: latency of a single row
        {"name": "norm_decode", "op": "norm", "rows": 1, "hidden": 2048, "type": "bf16", "residual": True, "y": True, "q": True},
        # a long prompt at the wider hidden size: bandwidth
        {"name": "norm_prompt", "op": "norm", "rows": 16384, "hidden": 4096, "type": "bf16", "residual": True, "y": False, "q": True},
        # the gradient of the same step over a training batch
        {"name": "norm_grad", "op": "norm_backward", "rows": 8192, "hidden": 2048, "type": "bf16"},
        # one decoded token through a projection: the weights are read once
        {"name": "matmul_decode", "op": "matmul", "rows": 1, "cols": 4096, "inner": 2048, "out": "bf16"},
        # a ragged chunk through a narrow projection, nothing a multiple of a tile
        {"name": "matmul_ragged", "op": "matmul", "rows": 333, "cols": 1000, "inner": 1200, "out": "f32"},
        # a long prompt through a wide projection: tensor-core rate
        {"name": "matmul_prompt", "op": "matmul", "rows": 8192, "cols": 8192, "inner": 4096, "out": "bf16"},
        # eight drafted tokens through the experts' gate/up product: one or two rows an expert
        {"name": "grouped_verify8", "op": "grouped", "tokens": 8, "experts": 256, "top_k": 8, "cols": 1024, "inner": 2048, "skew": 1.0, "out": "bf16"},
        # a prompt of 2048 tokens through all experts' gate/up product: about 64 rows an expert
        {"name": "grouped_prompt", "op": "grouped", "tokens": 2048, "experts": 256, "top_k": 8, "cols": 1024, "inner": 2048, "skew": 0.0, "out": "bf16"},
        # eight drafted tokens: rows in 8 bits to the experts and bf16 rows back
        {"name": "route_verify8", "op": "route", "tokens": 8, "experts": 256, "top_k": 8, "hidden": 2048, "type": "e4m3", "out": "f32", "skew": 1.0, "drop": 0.0},
        # a training batch: rows out, back, and the gradients of rows and weights
        {"name": "route_train", "op": "route_train", "tokens": 8192, "experts": 256, "top_k": 8, "hidden": 2048, "type": "bf16", "out": "bf16", "skew": 0.5, "drop": 0.0},
        # the experts' activation for eight drafted tokens
        {"name": "silu_verify8", "op": "silu", "rows": 64, "ffn": 512, "type": "bf16"},
        # the same for the rows of a long prompt
        {"name": "silu_prompt", "op": "silu", "rows": 65536, "ffn": 512, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "matmul", "matmul", "matmul", "grouped", "grouped", "route", "route", "route_train", "silu"])
    if op in ("norm", "norm_backward"):
        hidden = _log(rng, 64, 8192)
        hidden = rng.choice([hidden, hidden // 8 * 8, max(128, hidden // 128 * 128)])
        c = {"op": op, "rows": _log(rng, 1, (16384 * 4096 if op == "norm" else 8192 * 2048) // max(hidden, 4096)), "hidden": hidden, "type": rng.choice(["bf16", "f32"])}
        if op == "norm":
            y = rng.random() < 0.6
            c.update(residual=rng.random() < 0.7, y=y, q=not y or rng.random() < 0.6)
        return c
    if op == "matmul":
        cols, inner = _log(rng, 64, 8192), _log(rng, 64, 4096)
        return {"op": op, "rows": _log(rng, 1, 8192), "cols": rng.choice([cols, -(-cols // 64) * 64]), "inner": rng.choice([inner, -(-inner // 128) * 128]),
                "out": rng.choice(["bf16", "f32"])}
    experts = _log(rng, 4, 256)
    k = rng.randint(1, min(8, experts))
    if op == "grouped":
        return {"op": op, "tokens": _log(rng, 1, 2048), "experts": experts, "top_k": k, "cols": _log(rng, 64, 1024), "inner": _log(rng, 64, 2048),
                "skew": rng.choice([0.0, 0.5, 1.0]), "out": rng.choice(["bf16", "f32"])}
    if op in ("route", "route_train"):
        hidden = _log(rng, 64, 4096)
        kind = rng.choice(["bf16", "f32", "e4m3"] if op == "route" else ["bf16", "f32"])
        return {"op": op, "tokens": _log(rng, 1, 8192 * 2048 // max(hidden, 2048)) // (2 if kind == "f32" else 1) or 1, "experts": experts, "top_k": k,
                "hidden": rng.choice([hidden, -(-hidden // 128) * 128]), "type": kind, "out": rng.choice(["bf16", "f32"]) if op == "route" else kind, "skew": rng.choice([0.0, 0.5, 1.0]),
                "drop": rng.choice([0.0, 0.1])}
    return {"op": "silu", "rows": _log(rng, 1, 16384), "ffn": rng.choice([_log(rng, 64, 2048), 512, 1024]), "type": rng.choice(["bf16", "f32"])}


# ------------------------------------------------------------------ inputs

def _padded(rows, cols, dtype, device):
    """[rows, cols] whose rows start on 16-byte boundaries, as the 8-bit operands' do."""
    step = 16 // torch.empty(0, dtype=dtype).element_size()
    return torch.zeros(rows, -(-cols // step) * step, dtype=dtype, device=device)[:, :cols]


def _blocks(n):
    return -(-n // BLOCK)


def _e4m3_rows(v):
    """(q, scale) of fp32 rows: one scale per row and 128 columns."""
    q = _padded(*v.shape, torch.float8_e4m3fn, v.device)
    p = torch.nn.functional.pad(v, (0, -v.shape[1] % BLOCK)).view(v.shape[0], -1, BLOCK)
    scale = p.abs().amax(2).clamp_min(MIN_AMAX) / E4M3_MAX
    q.copy_((p / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).view(v.shape[0], -1)[:, : v.shape[1]].to(torch.float8_e4m3fn))
    return q, scale


def _e4m3_weights(w):
    """(q, scale) of fp32 weights [experts, cols, inner]: one scale per 128 x 128 block."""
    e, n, k = w.shape
    p = torch.nn.functional.pad(w, (0, -k % BLOCK, 0, -n % BLOCK)).view(e, _blocks(n), BLOCK, _blocks(k), BLOCK)
    scale = p.abs().amax((2, 4)).clamp_min(MIN_AMAX) / E4M3_MAX
    p = (p / scale[:, :, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(e, _blocks(n) * BLOCK, -1)[:, :n, :k]
    q = torch.zeros(e, n, -(-k // 16) * 16, dtype=torch.float8_e4m3fn, device=w.device)[:, :, :k]
    q.copy_(p.to(torch.float8_e4m3fn))
    return q, scale


def _routing(case, g, device):
    """Top-k ids and weights of a router whose experts' popularity falls off with rank^-skew; a share of the entries dropped."""
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    bias = -case["skew"] * torch.log1p(torch.arange(e, device=device, dtype=torch.float32))
    bias = bias[torch.randperm(e, generator=g, device=device)]
    top, ids = torch.topk(torch.randn(t, e, generator=g, device=device) + bias, k, dim=1)
    ids = ids.to(torch.int32)
    if case.get("drop", 0.0):
        ids = torch.where(torch.rand(t, k, generator=g, device=device) < case["drop"], torch.full_like(ids, -1), ids)
    return ids.contiguous(), torch.softmax(top, 1).contiguous()


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
    s, op = {"case": case}, case["op"]
    kind = TYPES[case.get("type", "bf16")]
    if op in ("norm", "norm_backward"):
        t, h = case["rows"], case["hidden"]
        loud = torch.where(torch.rand(h, generator=g, device=dev) < 0.01, 20.0, 1.0)  # a few channels are large, as in trained models
        s["weight"] = 1.0 + 0.1 * randn(h)
        if op == "norm":
            s["x"] = (randn(t, h) * loud).to(kind)
            s["residual"] = (3.0 * randn(t, h) * loud).to(kind) if case["residual"] else None
            s["total"] = torch.empty(t, h, dtype=kind, device=dev) if case["residual"] else None
            s["y"] = torch.empty(t, h, dtype=kind, device=dev) if case["y"] else None
            s["q"] = _padded(t, h, torch.float8_e4m3fn, dev) if case["q"] else None
            s["q_scale"] = torch.empty(t, _blocks(h), device=dev) if case["q"] else None
        else:
            s["total"] = (3.0 * randn(t, h) * loud).to(kind)
            s["dy"], s["dtotal"] = randn(t, h).to(kind), randn(t, h).to(kind)
            s["dx"], s["dweight"] = torch.empty(t, h, dtype=kind, device=dev), torch.empty(h, device=dev)
    elif op == "matmul":
        s["a"], s["a_scale"] = _e4m3_rows(randn(case["rows"], case["inner"]))
        w, ws = _e4m3_weights(0.02 * randn(1, case["cols"], case["inner"]))
        s["w"], s["w_scale"] = w[0], ws[0]
        s["out"] = torch.empty(case["rows"], case["cols"], dtype=TYPES[case["out"]], device=dev)
    elif op == "grouped":
        ids, _ = _routing(case, g, dev)
        counts = torch.bincount(ids.flatten().long(), minlength=case["experts"])
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["most"] = int(counts.max())  # the largest group, which padded forms need
        s["a"], s["a_scale"] = _e4m3_rows(randn(ids.numel(), case["inner"]))
        s["w"], s["w_scale"] = _e4m3_weights(0.02 * randn(case["experts"], case["cols"], case["inner"]))
        s["out"] = torch.empty(ids.numel(), case["cols"], dtype=TYPES[case["out"]], device=dev)
    elif op in ("route", "route_train"):
        s["ids"], s["w"] = _routing(case, g, dev)
        n, h = s["ids"].numel(), case["hidden"]
        x = randn(case["tokens"], h)
        s["x"], s["x_scale"] = _e4m3_rows(x) if case["type"] == "e4m3" else (x.to(kind), None)
        s["xs"] = _padded(n, h, kind, dev) if case["type"] == "e4m3" else torch.zeros(n, h, dtype=kind, device=dev)
        s["xs_scale"] = torch.zeros(n, _blocks(h), device=dev) if case["type"] == "e4m3" else None
        s["counts"], s["offsets"] = (torch.empty(case["experts"] + i, dtype=torch.int32, device=dev) for i in (0, 1))
        s["perm"] = torch.empty(n, dtype=torch.int32, device=dev)
        s["pos"] = torch.empty_like(s["ids"])
        rows = torch.bfloat16 if case["type"] == "e4m3" else kind  # the experts' outputs
        s["y"] = randn(n, h).to(rows)
        s["out"] = torch.empty(case["tokens"], h, dtype=TYPES[case["out"]], device=dev)
        if op == "route_train":
            s["dout"], s["dxs"] = randn(case["tokens"], h).to(kind), randn(n, h).to(kind)
            s["dy"], s["dw"], s["dx"] = torch.zeros(n, h, dtype=kind, device=dev), torch.empty_like(s["w"]), torch.empty(case["tokens"], h, dtype=kind, device=dev)
    else:
        s["gate_up"] = (1.5 * randn(case["rows"], 2 * case["ffn"])).to(kind)
        s["q"] = _padded(case["rows"], case["ffn"], torch.float8_e4m3fn, dev)
        s["q_scale"] = torch.empty(case["rows"], _blocks(case["ffn"]), device=dev)
    return s


# ------------------------------------------------------------------ plain forms

def _widen(q, scale):
    """The values of e4m3 rows, in 32 bits."""
    return q.float() * scale.repeat_interleave(BLOCK, -1)[..., : q.shape[-1]]


def _widen_weights(q, scale):
    return q.float() * scale.repeat_interleave(BLOCK, -2)[..., : q.shape[-2], :].repeat_interleave(BLOCK, -1)[..., : q.shape[-1]]


def _plain_norm(s):
    x = s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"].float()
    y = x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * s["weight"]
    r = {}
    if s["residual"] is not None:
        r["total"] = x.to(s["x"].dtype)
    if s["y"] is not None:
        r["y"] = y.to(s["x"].dtype)
    if s["q"] is not None:
        r["q"], r["q_scale"] = _e4m3_rows(y)
    return r


def _plain_norm_backward(s):
    x, dy, h = s["total"].float(), s["dy"].float(), s["total"].shape[1]
    r = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    g = dy * s["weight"]
    dx = r * g - x * r ** 3 * ((g * x).sum(1, keepdim=True) / h) + s["dtotal"].float()
    return {"dx": dx.to(s["dx"].dtype), "dweight": (dy * x * r).sum(0)}


def _plain_grouped(s):
    off = s["offsets"].long()
    row = torch.arange(s["a"].shape[0], device=off.device)
    e = torch.searchsorted(off[1:].contiguous(), row, right=True)
    rank = row - off[e]
    a = torch.zeros(s["w"].shape[0], s["most"], s["a"].shape[1], device=off.device)
    a[e, rank] = _widen(s["a"], s["a_scale"])
    return torch.bmm(a, _widen_weights(s["w"], s["w_scale"]).transpose(1, 2))[e, rank].to(s["out"].dtype)


def _plain_sort(s):
    """(counts, offsets, perm, pos): entries by expert, in the order of entries within one; dropped entries have position -1."""
    n, e = s["ids"].numel(), s["counts"].numel()
    flat = s["ids"].flatten().long()
    key = torch.where((flat >= 0) & (flat < e), flat, torch.full_like(flat, e))
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=e + 1)[:e]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    at = torch.arange(n, device=flat.device)
    kept = at < offsets[-1]
    pos = torch.empty_like(order)
    pos[order] = torch.where(kept, at, torch.full_like(at, -1))
    return counts, offsets, torch.where(kept, order, torch.full_like(order, -1)), pos.view(s["ids"].shape), kept


def _plain_gather(v, pos):
    """v[pos] in 32 bits, [tokens, k, hidden], zeros where pos is -1."""
    return torch.where((pos >= 0)[..., None], v[pos.clamp_min(0)].float(), torch.zeros((), device=v.device))


def _plain_route(s):
    counts, offsets, perm, pos, kept = _plain_sort(s)
    token = perm.clamp_min(0) // s["ids"].shape[1]
    rows = lambda v: torch.where(kept[:, None], v.float()[token], torch.zeros((), device=v.device)).to(v.dtype)  # noqa: E731
    r = {"counts": counts.int(), "offsets": offsets.int(), "perm": perm.int(), "pos": pos.int(), "xs": rows(s["x"])}
    if s["x_scale"] is not None:
        r["xs_scale"] = rows(s["x_scale"])
    y = _plain_gather(s["y"], pos)
    r["out"] = (y * s["w"][..., None]).sum(1).to(s["out"].dtype)
    if "dout" in s:
        dout = s["dout"].float()
        dy = s["w"].flatten()[perm.clamp_min(0)][:, None] * dout[token]
        r["dy"] = torch.where(kept[:, None], dy, torch.zeros((), device=dy.device)).to(s["dy"].dtype)
        r["dw"] = (y * dout[:, None, :]).sum(2)
        r["dx"] = _plain_gather(s["dxs"], pos).sum(1).to(s["dx"].dtype)
    return r


def _plain_silu(s):
    gate, up = s["gate_up"].float().chunk(2, 1)
    q, scale = _e4m3_rows(gate / (1.0 + torch.exp(-gate)) * up)
    return {"q": q, "q_scale": scale}


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        if op == "norm":
            return _plain_norm(s)
        if op == "norm_backward":
            return _plain_norm_backward(s)
        if op == "matmul":
            return (_widen(s["a"], s["a_scale"]) @ _widen_weights(s["w"], s["w_scale"]).t()).to(s["out"].dtype)
        if op == "grouped":
            return _plain_grouped(s)
        if op in ("route", "route_train"):
            return _plain_route(s)
        return _plain_silu(s)
    from bit_quantized_moe_router_gb300 import qs_moe as qm
    if op == "norm":
        qm.qs_rmsnorm_residual(s["x"], s["residual"], s["weight"], EPS, s["total"], s["y"], s["q"], s["q_scale"])
        return {k: s[k] for k in ("total", "y", "q", "q_scale") if s[k] is not None}
    if op == "norm_backward":
        if "workspace" not in s:  # the program's own, kept between calls
            s["workspace"] = qm.alloc_rmsnorm_backward_workspace(s["total"].shape[1])
        qm.qs_rmsnorm_residual_backward(s["total"], s["weight"], EPS, s["dy"], s["dtotal"], s["dx"], s["dweight"], s["workspace"])
        return {"dx": s["dx"], "dweight": s["dweight"]}
    if op in ("matmul", "grouped"):
        if "workspace" not in s:
            s["workspace"] = qm.alloc_fp8_matmul_workspace(s["a"].shape[0], s["w"].shape[-2], s["w"].shape[-1], s["w"].shape[0] if op == "grouped" else 1)
        qm.qs_fp8_matmul(s["a"], s["a_scale"], s["w"], s["w_scale"], s["out"], s["workspace"], s.get("offsets"))
        return s["out"]
    if op in ("route", "route_train"):
        if "workspace" not in s:
            s["workspace"] = qm.alloc_dispatch_workspace(s["ids"].shape[0], s["ids"].shape[1], s["counts"].numel())
        qm.qs_dispatch_tokens(s["ids"], s["x"], s["x_scale"], s["counts"], s["offsets"], s["perm"], s["pos"], s["xs"], s["xs_scale"], s["workspace"])
        qm.qs_combine_tokens(s["y"], s["pos"], s["w"], s["out"])
        r = {k: s[k] for k in ("counts", "offsets", "perm", "pos", "xs", "xs_scale", "out") if s[k] is not None}
        if op == "route_train":
            qm.qs_combine_tokens_backward(s["dout"], s["y"], s["pos"], s["w"], s["dy"], s["dw"])
            qm.qs_combine_tokens(s["dxs"], s["pos"], None, s["dx"])
            r.update(dy=s["dy"], dw=s["dw"], dx=s["dx"])
        return r
    qm.qs_silu_mul_quant(s["gate_up"], s["q"], s["q_scale"])
    return {"q": s["q"], "q_scale": s["q_scale"]}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4, "e4m3": 1}
    z = size[case.get("type", "bf16")]
    if op == "norm":
        t, h = case["rows"], case["hidden"]
        per = z + (2 * z if case["residual"] else 0) + (z if case["y"] else 0) + (1 if case["q"] else 0)
        return {"bytes": t * h * per + 4 * h + (4 * t * _blocks(h) if case["q"] else 0), "flops": t * h * 8}
    if op == "norm_backward":
        t, h = case["rows"], case["hidden"]
        return {"bytes": t * h * 4 * z + 8 * h, "flops": t * h * 14}
    if op == "matmul":
        m, n, k = case["rows"], case["cols"], case["inner"]
        return {"bytes": m * k + n * k + 4 * m * _blocks(k) + 4 * _blocks(n) * _blocks(k) + m * n * size[case["out"]], "flops": 2 * m * n * k}
    if op == "grouped":
        m, n, k, e = case["tokens"] * case["top_k"], case["cols"], case["inner"], case["experts"]
        met = e * (1.0 - (1.0 - case["top_k"] / e) ** case["tokens"])  # experts with a row, if all are as likely
        return {"bytes": int(m * k + met * (n * k + 4 * _blocks(n) * _blocks(k)) + 4 * m * _blocks(k) + m * n * size[case["out"]]), "flops": 2 * m * n * k}
    if op in ("route", "route_train"):
        t, k, h = case["tokens"], case["top_k"], case["hidden"]
        n = int(t * k * (1.0 - case["drop"]))
        y = 2 if case["type"] == "e4m3" else z
        row = h * z + (4 * _blocks(h) if case["type"] == "e4m3" else 0)
        b = 4 * (4 * t * k + 2 * case["experts"]) + (t + n) * row + n * h * y + t * h * size[case["out"]]
        f = 2 * n * h
        if op == "route_train":
            b += t * h * z + 2 * n * h * z + 4 * t * k + n * h * z + t * h * z  # dout, y, dy, dw; dxs, dx
            f += 4 * n * h
        return {"bytes": b, "flops": f}
    r, f = case["rows"], case["ffn"]
    return {"bytes": r * f * (2 * z + 1) + 4 * r * _blocks(f), "flops": r * f * 8}


# ------------------------------------------------------------------ the definitions in 64 bits

def _nearest_e4m3(v):
    """v (64 bits) rounded to the nearest e4m3 value, ties to even: 3 bits after the leading one, exponents from -6."""
    exponent = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -20)))
    step = torch.exp2(exponent.clamp_min(-6.0) - 3.0)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_quant(v):
    t, h = v.shape
    nb = _blocks(h)
    wide = v.new_zeros(t, nb * BLOCK)
    wide[:, :h] = v
    amax = wide.abs().reshape(t, nb, BLOCK).max(2).values
    scale = torch.maximum(amax, torch.full_like(amax, MIN_AMAX)) / E4M3_MAX
    column = torch.arange(h, device=v.device) // BLOCK
    return _nearest_e4m3(v / scale[:, column]), scale


def _exact_values(q, scale, weights=False):
    k = torch.arange(q.shape[-1], device=q.device) // BLOCK
    if not weights:
        return q.double() * scale.double()[:, k]
    n = torch.arange(q.shape[-2], device=q.device) // BLOCK
    return q.double() * scale.double()[n][:, k]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "norm":
        v = s["x"].double()
        if s["residual"] is not None:
            v = v + s["residual"].double()
        y = s["weight"].double() * v / torch.sqrt(v.pow(2).sum(1, keepdim=True) / v.shape[1] + EPS)
        r = {}
        if s["residual"] is not None:
            r["total"] = v
        if s["y"] is not None:
            r["y"] = y
        if s["q"] is not None:
            r["q"], r["q_scale"] = _exact_quant(y)
        return r
    if op == "norm_backward":
        v, dy, w = s["total"].double(), s["dy"].double(), s["weight"].double()
        rms = torch.sqrt(v.pow(2).mean(1, keepdim=True) + EPS)
        unit = v / rms
        g = dy * w
        return {"dx": (g - unit * (g * unit).mean(1, keepdim=True)) / rms + s["dtotal"].double(), "dweight": torch.einsum("th,th->h", dy, unit)}
    if op == "matmul":
        return torch.mm(_exact_values(s["a"], s["a_scale"]), _exact_values(s["w"], s["w_scale"], True).T)
    if op == "grouped":
        a, off = _exact_values(s["a"], s["a_scale"]), s["offsets"].tolist()
        out = a.new_zeros(a.shape[0], s["w"].shape[1])
        for e in range(case["experts"]):
            if off[e + 1] > off[e]:
                out[off[e]:off[e + 1]] = a[off[e]:off[e + 1]] @ _exact_values(s["w"][e], s["w_scale"][e], True).T
        return out
    if op in ("route", "route_train"):
        t, k = s["ids"].shape
        ids = s["ids"].flatten()
        lists = [(ids == e).nonzero().flatten() for e in range(case["experts"])]
        perm = torch.cat(lists)
        n = perm.numel()
        pos = torch.full((t * k,), -1, dtype=torch.long, device=ids.device)
        pos[perm] = torch.arange(n, device=ids.device)
        h = case["hidden"]

        def placed(v):
            rows = torch.zeros(t * k, v.shape[1], dtype=torch.float64, device=v.device)
            rows[:n] = v.double()[perm // k]
            return rows

        def summed(v, weight):
            total = torch.zeros(t, h, dtype=torch.float64, device=v.device)
            for j in range(k):
                p = pos.view(t, k)[:, j]
                total += torch.where((p >= 0)[:, None], v[p.clamp_min(0)].double() * (weight[:, j:j + 1].double() if weight is not None else 1.0), 0.0)
            return total

        r = {"counts": None, "offsets": None, "perm": None, "pos": None, "xs": placed(s["x"]), "out": summed(s["y"], s["w"])}
        if s["x_scale"] is not None:
            r["xs_scale"] = placed(s["x_scale"])
        if op == "route_train":
            dy = torch.zeros(t * k, h, dtype=torch.float64, device=ids.device)
            dy[:n] = s["w"].flatten()[perm].double()[:, None] * s["dout"].double()[perm // k]
            dw = torch.zeros(t * k, dtype=torch.float64, device=ids.device)
            dw[perm] = (s["dout"].double()[perm // k] * s["y"][:n].double()).sum(1)
            r.update(dy=dy, dw=dw.view(t, k), dx=summed(s["dxs"], None))
        return r
    gate, up = s["gate_up"].double().split(case["ffn"], 1)
    q, scale = _exact_quant(gate * torch.sigmoid(gate) * up)
    return {"q": q, "q_scale": scale}
