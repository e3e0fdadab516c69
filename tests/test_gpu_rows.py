"""Norm, SwiGLU, dispatch and combine on the GPU against plain forms in 64 bits.

Tolerances are sums of roundings, 2^-24 (U) of the value each: a row's sum of squares of n terms is at most
(longest chain of additions) U off relatively, here under 48 U; rsqrt 2 units in the last place (4 U); the products one
each.  Stored values add half a step of their type: 2^-8 for bf16, 2^-24 for fp32; e4m3 codes half a step of the code,
2^-4 of the value or 2^-10 of the scale below the normal codes.
"""
import numpy as np
import pytest
import torch

from bit_quantized_moe_router_gb300 import qs_moe as qm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
F8 = torch.float8_e4m3fn
EPS = 1e-5


def gen(seed):
    return torch.Generator().manual_seed(seed)


def strided(t, pad, shift=0):
    """t on the GPU inside a wider buffer: rows `pad` elements further apart, the first `shift` elements in."""
    rows, cols = t.shape
    buf = torch.zeros(rows * (cols + pad) + shift, dtype=t.dtype, device="cuda")
    view = buf[shift:].view(rows, cols + pad)[:, :cols]
    view.copy_(t)
    return view


def codes(rows, cols, pad=0):
    q = torch.full((rows, cols + pad), 0x55, dtype=torch.uint8, device="cuda").view(F8)[:, :cols]
    return q, torch.full((rows, (cols + 127) // 128), -1.0, device="cuda")


def check_codes(q, scale, v, slack):
    """Codes and scales of fp64 values v: the scale is amax / 448, each value within half a step of its code."""
    rows, cols = v.shape
    nb = (cols + 127) // 128
    wide = torch.zeros(rows, nb * 128, dtype=torch.float64)
    wide[:, :cols] = v
    amax = wide.abs().view(rows, nb, 128).amax(2).clamp_min(2.0 ** -100)
    got_scale = scale.cpu().double()
    assert torch.all((got_scale - amax / 448).abs() <= (slack + 2 * U) * amax / 448)
    per = got_scale.repeat_interleave(128, 1)[:, :cols]
    got = q.cpu().float().double() * per
    assert torch.all((got - v).abs() <= v.abs() * (2.0 ** -4 + slack + 4 * U) + per * 2.0 ** -10)


def norm_ref(x, r, w):
    s = x.double() + (0 if r is None else r.double())
    return s, s / torch.sqrt(s.pow(2).mean(1, keepdim=True) + EPS) * w.double()


NORM_SLACK = (48 / 2 + 4 + 4) * U + 2 * U


@pytest.mark.parametrize("hidden", [1, 7, 8, 100, 128, 129, 256, 264, 520, 1000, 1032, 2048, 2056, 4096, 5000, 8192, 8200, 16384])
@pytest.mark.parametrize("rows,kind,res", [(1, torch.bfloat16, torch.bfloat16), (5, torch.float32, None), (77, torch.bfloat16, torch.float32),
                                           (311, torch.bfloat16, torch.bfloat16)])
def test_norm(hidden, rows, kind, res):
    g = gen(hidden + rows)
    x = torch.randn(rows, hidden, generator=g).to(kind)
    r = None if res is None else (3 * torch.randn(rows, hidden, generator=g)).to(res)
    w = 1 + 0.2 * torch.randn(hidden, generator=g)
    total = torch.full((rows, hidden), 9.0, dtype=torch.float32, device="cuda")
    y = torch.full((rows, hidden), 9.0, dtype=kind, device="cuda")
    q, scale = codes(rows, hidden, pad=(-hidden) % 16)
    qm.qs_rmsnorm_residual(x.cuda(), None if r is None else r.cuda(), w.cuda(), EPS, total, y, q, scale)
    s, v = norm_ref(x, r, w)
    assert torch.all((total.cpu().double() - s).abs() <= U * s.abs())
    # s is rounded once where a residual is added, and v is proportional to it
    tol = NORM_SLACK + U
    assert torch.all((y.cpu().double() - v).abs() <= (tol + HALF[kind]) * v.abs())
    check_codes(q, scale, v, tol)


@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (16, 8), (3, 0), (5, 1)])
def test_norm_strides_and_each_output_alone(pad, shift):
    rows, hidden = 9, 1024
    g = gen(pad)
    x, r, w = torch.randn(rows, hidden, generator=g), torch.randn(rows, hidden, generator=g).bfloat16(), torch.rand(hidden, generator=g)
    s, v = norm_ref(x, r, w)
    xs, rs = strided(x, pad, shift), strided(r, pad, shift)
    y = strided(torch.zeros(rows, hidden, dtype=torch.bfloat16), pad, shift)
    qm.qs_rmsnorm_residual(xs, rs, w.cuda(), EPS, y=y)
    assert torch.all((y.cpu().double() - v).abs() <= (NORM_SLACK + U + 2.0 ** -8) * v.abs())
    q, scale = codes(rows, hidden, pad)
    qm.qs_rmsnorm_residual(xs, rs, w.cuda(), EPS, q=q, q_scale=scale)
    check_codes(q, scale, v, NORM_SLACK + U)
    qm.qs_rmsnorm_residual(xs, rs, w.cuda(), EPS, sum_out=rs)  # in place
    assert torch.equal(rs.cpu(), s.float().bfloat16())
    assert torch.equal(xs.cpu(), x)


def test_norm_rows_that_are_zero_infinite_or_nan():
    x = torch.randn(5, 512, generator=gen(1))
    x[0] = 0
    x[1, 200] = float("inf")
    x[2, 300] = float("nan")
    x[3] = 1e-30
    q, scale = codes(5, 512)
    y = torch.empty(5, 512, device="cuda")
    qm.qs_rmsnorm_residual(x.cuda(), None, torch.ones(512, device="cuda"), EPS, y=y, q=q, q_scale=scale)
    assert torch.all(y[0] == 0) and torch.all(q[0].float() == 0) and torch.all(torch.isfinite(scale[0]) & (scale[0] > 0))
    assert torch.isnan(y[1, 200]) and torch.all(y[1, :200] == 0) and torch.isnan(q[1].float()[200])
    assert torch.all(torch.isnan(y[2])) and torch.all(torch.isnan(q[2].float()))
    assert torch.all(torch.isfinite(q[3].float())) and torch.all(torch.isfinite(y[4]))


def bwd_ref(s, w, dy, dsum):
    s, w, dy = s.double(), w.double(), dy.double()
    n = s.shape[1]
    rho = 1 / torch.sqrt(s.pow(2).mean(1, keepdim=True) + EPS)
    g = w * dy
    dx = rho * g - s * rho ** 3 * (g * s).sum(1, keepdim=True) / n
    size = (rho * g).abs() + s.abs() * rho ** 3 * (g * s).abs().sum(1, keepdim=True) / n
    if dsum is not None:
        dx, size = dx + dsum.double(), size + dsum.double().abs()
    return dx, size, (dy * s * rho).sum(0), (dy * s * rho).abs().sum(0)


@pytest.mark.parametrize("hidden", [1, 8, 100, 256, 264, 1000, 1024, 2048, 4096, 4104, 8192, 16384])
@pytest.mark.parametrize("rows,kind,with_dsum", [(1, torch.bfloat16, True), (37, torch.float32, False), (1500, torch.bfloat16, True)])
def test_norm_backward(hidden, rows, kind, with_dsum):
    g = gen(hidden * 3 + rows)
    s = (2 * torch.randn(rows, hidden, generator=g)).to(kind)
    dy, dsum = torch.randn(rows, hidden, generator=g).to(kind), torch.randn(rows, hidden, generator=g).to(kind)
    w = 1 + 0.2 * torch.randn(hidden, generator=g)
    dx, dw = torch.empty(rows, hidden, dtype=kind, device="cuda"), torch.empty(hidden, device="cuda")
    ws = qm.alloc_rmsnorm_backward_workspace(hidden)
    ws.fill_(0xFF)  # needs no initialisation
    call = lambda: qm.qs_rmsnorm_residual_backward(s.cuda(), w.cuda(), EPS, dy.cuda(), dsum.cuda() if with_dsum else None, dx, dw, ws)  # noqa: E731
    call()
    want, size, dwant, dsize = bwd_ref(s, w, dy, dsum if with_dsum else None)
    # rho^3 carries three times rho's error, the mean over the row its own 48 U
    assert torch.all((dx.cpu().double() - want).abs() <= 160 * U * size + HALF[kind] * want.abs())
    # a column's chain: rho, two products, a group's rows (at most 3 here), the groups of a CTA, 32 slices of CTAs
    assert torch.all((dw.cpu().double() - dwant).abs() <= 160 * U * dsize)
    first = (dx.clone(), dw.clone())
    call()
    assert torch.equal(dx, first[0]) and torch.equal(dw, first[1])


def test_norm_backward_against_differences():
    rows, hidden = 3, 264
    g = gen(4)
    x, dy, w, d = (torch.randn(*n, generator=g) for n in ((rows, hidden), (rows, hidden), (hidden,), (rows, hidden)))
    dw_dir = torch.randn(hidden, generator=g)

    def loss(xx, ww):
        y = torch.empty(rows, hidden, device="cuda")
        qm.qs_rmsnorm_residual(xx.cuda(), None, ww.cuda(), EPS, y=y)
        return float((y.cpu().double() * dy.double()).sum())

    dx, dw = torch.empty(rows, hidden, device="cuda"), torch.empty(hidden, device="cuda")
    qm.qs_rmsnorm_residual_backward(x.cuda(), w.cuda(), EPS, dy.cuda(), None, dx, dw, qm.alloc_rmsnorm_backward_workspace(hidden))
    h = 1e-2  # truncation h^2 and rounding 1e-7 * size / h are both near 1e-4 of the gradient's size here
    for slope, grad in (((loss(x + h * d, w) - loss(x - h * d, w)) / (2 * h), float((dx.cpu().double() * d.double()).sum())),
                        ((loss(x, w + h * dw_dir) - loss(x, w - h * dw_dir)) / (2 * h), float((dw.cpu().double() * dw_dir.double()).sum()))):
        scale = float(dx.cpu().double().norm() * d.double().norm())
        assert abs(slope - grad) <= 2e-3 * scale


def test_norm_backward_in_place_without_dweight_and_without_rows():
    g = gen(6)
    s, dy, w = torch.randn(8, 512, generator=g), torch.randn(8, 512, generator=g), torch.rand(512, generator=g)
    want, size, _, _ = bwd_ref(s, w, dy, None)
    buf = dy.cuda()
    qm.qs_rmsnorm_residual_backward(s.cuda(), w.cuda(), EPS, buf, None, buf)
    assert torch.all((buf.cpu().double() - want).abs() <= 160 * U * size)
    dw = torch.full((512,), 7.0, device="cuda")
    none = torch.empty(0, 512, device="cuda")
    qm.qs_rmsnorm_residual_backward(none, w.cuda(), EPS, none, None, none, dw, qm.alloc_rmsnorm_backward_workspace(512))
    assert torch.all(dw == 0)


@pytest.mark.parametrize("ffn", [1, 5, 8, 64, 128, 136, 200, 512, 1000, 2048])
@pytest.mark.parametrize("rows,kind", [(1, torch.bfloat16), (3, torch.float32), (130, torch.bfloat16)])
def test_silu(ffn, rows, kind):
    gu = (3 * torch.randn(rows, 2 * ffn, generator=gen(ffn))).to(kind)
    q, scale = codes(rows, ffn, pad=(-ffn) % 16)
    qm.qs_silu_mul_quant(gu.cuda(), q, scale)
    gate, up = gu.double().chunk(2, 1)
    # exp within 2 units, sum, division, two products; the sum's error is relative to 1 + exp(-gate) itself
    check_codes(q, scale, gate / (1 + torch.exp(-gate)) * up, 10 * U)


def test_silu_row_limit_and_large_gates():
    gu = torch.zeros(6, 256, device="cuda")
    gu[:, :128] = torch.tensor([-200.0, -20.0, 0.0, 20.0, 200.0, 1.0], device="cuda")[:, None]
    gu[:, 128:] = 2.0
    q, scale = codes(6, 128)
    qm.qs_silu_mul_quant(gu, q, scale, torch.tensor([5], dtype=torch.int32, device="cuda"))
    v = (q.float() * scale)[:, 0].cpu()
    assert abs(float(v[0])) == 0 and float(v[2]) == 0 and abs(float(v[3]) - 40) < 1e-3 and abs(float(v[4]) - 400) < 1e-3
    assert torch.all(scale[5] == -1) and torch.all(q[5].view(torch.uint8) == 0x55)  # beyond the limit: left alone
    qm.qs_silu_mul_quant(gu, q, scale, torch.tensor([-3], dtype=torch.int32, device="cuda"))
    qm.qs_silu_mul_quant(gu, q, scale, torch.tensor([100], dtype=torch.int32, device="cuda"))
    assert torch.all(scale[5] > 0)


# ------------------------------------------------------------------ dispatch and combine

def plan(ids, experts):
    flat = ids.flatten().tolist()
    lists = [[i for i, e in enumerate(flat) if e == x] for x in range(experts)]
    perm = [i for part in lists for i in part]
    pos = [-1] * len(flat)
    for p, i in enumerate(perm):
        pos[i] = p
    counts = [len(part) for part in lists]
    return (torch.tensor(counts, dtype=torch.int32), torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32),
            torch.tensor(perm + [-1] * (len(flat) - len(perm)), dtype=torch.int32), torch.tensor(pos, dtype=torch.int32).view(ids.shape))


def outputs(tokens, k, experts):
    i32 = dict(dtype=torch.int32, device="cuda")
    return torch.full((experts,), 99, **i32), torch.full((experts + 1,), 99, **i32), torch.full((tokens * k,), 99, **i32), torch.full((tokens, k), 99, **i32)


def routed(tokens, k, experts, g, how):
    if how == "one":
        return torch.full((tokens, k), experts - 1, dtype=torch.int32)
    if how == "none":
        return torch.full((tokens, k), -1, dtype=torch.int32)
    ids = torch.randint(0, experts, (tokens, k), generator=g, dtype=torch.int32)
    if how == "drop":
        bad = torch.tensor([-1, experts, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
        ids = torch.where(torch.rand(tokens, k, generator=g) < 0.3, bad[torch.randint(0, 4, (tokens, k), generator=g)], ids)
    return ids


@pytest.mark.parametrize("tokens,k,experts,hidden,kind,how", [
    (1, 1, 1, 16, torch.float32, "random"), (8, 8, 256, 2048, F8, "random"), (5, 3, 7, 100, F8, "drop"),
    (5, 2, 4, 1, F8, "random"), (33, 8, 64, 520, torch.bfloat16, "drop"), (7, 32, 1024, 24, torch.bfloat16, "random"),
    (256, 8, 16, 64, torch.bfloat16, "drop"), (257, 8, 16, 64, torch.bfloat16, "random"), (1000, 5, 100, 33, torch.bfloat16, "drop"),
    (512, 8, 16, 64, torch.bfloat16, "drop"), (513, 8, 300, 64, torch.bfloat16, "random"), (600, 8, 256, 128, torch.float32, "one"),
    (600, 8, 256, 129, torch.float32, "none"), (300, 8, 256, 128, torch.float32, "one"), (300, 8, 256, 129, torch.float32, "none"), (40, 2, 3, 7, torch.float32, "none"),
    (4099, 32, 1024, 8, F8, "drop"), (0, 4, 16, 64, torch.bfloat16, "random")])
def test_dispatch(tokens, k, experts, hidden, kind, how):
    g = gen(tokens + experts)
    ids = routed(tokens, k, experts, g, how)
    x = (torch.randn(tokens, hidden, generator=g) * 2).to(kind)
    scale = torch.rand(tokens, (hidden + 127) // 128, generator=g)
    xs = torch.full((tokens * k, hidden), 3.0, device="cuda").to(kind)
    ss = torch.full((tokens * k, scale.shape[1]), 3.0, device="cuda")
    out = outputs(tokens, k, experts)
    ws = qm.alloc_dispatch_workspace(tokens, k, experts)
    ws.fill_(0xFF)
    fp8 = kind is F8
    qm.qs_dispatch_tokens(ids.cuda(), x.cuda(), scale.cuda() if fp8 else None, *out, xs, ss if fp8 else None, ws)
    want = plan(ids, experts)
    for got, ref in zip(out, want):
        assert torch.equal(got.cpu(), ref)
    total = int(want[1][-1])
    token = want[2][:total].long() // k
    size = {F8: torch.uint8, torch.bfloat16: torch.int16, torch.float32: torch.int32}[kind]
    assert torch.equal(xs.cpu()[:total].view(size), x.view(size)[token])
    assert torch.all(xs[total:].float() == 3.0)
    if fp8:
        assert torch.equal(ss.cpu()[:total], scale[token]) and torch.all(ss[total:] == 3.0)
    alone = outputs(tokens, k, experts)  # the plan without rows
    qm.qs_dispatch_tokens(ids.cuda(), None, None, *alone, None, None, ws)
    assert all(torch.equal(a, b) for a, b in zip(alone, out))


@pytest.mark.parametrize("pad,shift", [(0, 0), (2, 0), (1, 1), (8, 8)])
def test_dispatch_strides(pad, shift):
    ids = routed(70, 4, 9, gen(2), "drop")
    x = torch.randn(70, 48, generator=gen(3)).bfloat16()
    xs = strided(torch.zeros(280, 48, dtype=torch.bfloat16), pad, shift)
    qm.qs_dispatch_tokens(ids.cuda(), strided(x, pad, shift), None, *outputs(70, 4, 9), xs, None, qm.alloc_dispatch_workspace(70, 4, 9))
    _, off, perm, _ = plan(ids, 9)
    n = int(off[-1])
    assert torch.equal(xs.cpu()[:n], x[perm[:n].long() // 4])


@pytest.mark.parametrize("tokens,k,hidden,kind,out_kind,how,weighted", [
    (1, 1, 8, torch.float32, torch.float32, "random", True), (8, 8, 2048, torch.bfloat16, torch.float32, "random", True),
    (33, 8, 100, torch.bfloat16, torch.bfloat16, "drop", True), (300, 5, 1000, torch.float32, torch.bfloat16, "drop", False),
    (20, 32, 4096, torch.bfloat16, torch.bfloat16, "drop", True), (9, 9, 3, torch.float32, torch.float32, "none", True),
    (400, 2, 5000, torch.bfloat16, torch.float32, "one", True)])
def test_combine_and_backward(tokens, k, hidden, kind, out_kind, how, weighted):
    g = gen(hidden)
    ids = routed(tokens, k, 11, g, how)
    _, off, _, pos = plan(ids, 11)
    n = tokens * k
    y, dout = torch.randn(n, hidden, generator=g).to(kind), torch.randn(tokens, hidden, generator=g).to(out_kind)
    y[int(off[-1]):] = float("nan")  # rows that no entry has
    w = torch.rand(tokens, k, generator=g)
    w[pos < 0] = float("inf")  # and weights of dropped entries
    out = torch.empty(tokens, hidden, dtype=out_kind, device="cuda")
    wc = w.cuda() if weighted else None
    qm.qs_combine_tokens(y.cuda(), pos.cuda(), wc, out)
    on = (pos >= 0)[..., None]
    rows = torch.where(on, y.double()[pos.clamp_min(0).long()], 0.0)
    wd = torch.where(pos >= 0, w.double(), 0.0) if weighted else (pos >= 0).double()
    want, size = (rows * wd[..., None]).sum(1), (rows * wd[..., None]).abs().sum(1)
    assert torch.all((out.cpu().double() - want).abs() <= (k + 1) * U * size + HALF[out_kind] * want.abs())
    dy, dw = torch.full((n, hidden), 5.0, dtype=kind, device="cuda"), torch.full((tokens, k), 5.0, device="cuda")
    qm.qs_combine_tokens_backward(dout.cuda(), y.cuda(), pos.cuda(), wc, dy, dw)
    dyw = wd[..., None] * dout.double()[:, None, :]
    got = dy.cpu().double()
    assert torch.all(((got[pos.clamp_min(0).long()] - dyw).abs() <= (U + HALF[kind]) * dyw.abs()) | ~on)
    assert torch.all(got[int(off[-1]):] == 5.0)
    prod = rows * dout.double()[:, None, :]
    # a thread's chain is at most 8 * ceil(hidden / 2048) products, then 5 shuffles and 8 warps
    assert torch.all((dw.cpu().double() - prod.sum(2)).abs() <= (8 * -(-hidden // 2048) + 14) * U * prod.abs().sum(2))
    assert torch.all(dw.cpu()[pos < 0] == 0)
    only = torch.full((n, hidden), 5.0, dtype=kind, device="cuda")
    qm.qs_combine_tokens_backward(dout.cuda(), None, pos.cuda(), wc, only)
    assert torch.equal(only, dy)


def test_combine_backward_against_differences():
    tokens, k, hidden = 4, 3, 40
    g = gen(8)
    ids = routed(tokens, k, 5, g, "drop")
    pos = plan(ids, 5)[3].cuda()
    y, w, dout = torch.randn(12, hidden, generator=g).cuda(), torch.rand(tokens, k, generator=g).cuda(), torch.randn(tokens, hidden, generator=g).cuda()

    def loss(yy, ww):
        out = torch.empty(tokens, hidden, device="cuda")
        qm.qs_combine_tokens(yy, pos, ww, out)
        return float((out.double() * dout.double()).sum())

    dy, dw = torch.zeros(12, hidden, device="cuda"), torch.empty(tokens, k, device="cuda")
    qm.qs_combine_tokens_backward(dout, y, pos, w, dy, dw)
    a, b = torch.randn(12, hidden, generator=g).cuda(), torch.randn(tokens, k, generator=g).cuda()
    # the loss is linear in each: the difference has rounding errors alone, U * size / h
    for slope, grad in ((loss(y + a, w) - loss(y - a, w), (dy * a).double().sum()), (loss(y, w + b) - loss(y, w - b), (dw * b).double().sum())):
        assert abs(slope / 2 - float(grad)) <= 1e-4 * float(dout.double().norm()) * 10


def test_matrices_without_rows():
    none, f8 = torch.empty(0, 256, device="cuda"), torch.empty(0, 256, device="cuda").to(F8)
    scale = torch.empty(0, 2, device="cuda")
    qm.qs_rmsnorm_residual(none, none, torch.ones(256, device="cuda"), EPS, none, none, f8, scale)
    qm.qs_silu_mul_quant(torch.empty(0, 512, device="cuda"), f8, scale)
    pos = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    qm.qs_combine_tokens(none, pos, None, none)
    qm.qs_combine_tokens_backward(none, none, pos, None, none, torch.empty(0, 3, device="cuda"))
    w = torch.zeros(64, 256, device="cuda").to(F8)
    qm.qs_fp8_matmul(f8, scale, w, torch.ones(1, 2, device="cuda"), torch.empty(0, 64, device="cuda"), qm.alloc_fp8_matmul_workspace(0, 64, 256))


def test_positions_outside_the_rows_are_not_read():
    y = torch.ones(4, 16, device="cuda")
    pos = torch.tensor([[0, 4], [2 ** 31 - 1, -7]], dtype=torch.int32, device="cuda")
    out = torch.empty(2, 16, device="cuda")
    qm.qs_combine_tokens(y, pos, None, out)
    assert torch.all(out[0] == 1) and torch.all(out[1] == 0)
    dy, dw = torch.zeros(4, 16, device="cuda"), torch.empty(2, 2, device="cuda")
    qm.qs_combine_tokens_backward(out, y, pos, None, dy, dw)
    assert torch.all(dy[0] == 1) and torch.all(dy[1:] == 0) and dw.flatten().tolist() == [16, 0, 0, 0]


def test_offsets_past_32_bits():
    """Rows whose element offsets pass 2^31: the last rows are written and read where they belong."""
    tokens, k, hidden, experts = 66000, 8, 4096, 16
    ids = torch.arange(tokens * k, dtype=torch.int32, device="cuda").view(tokens, k) % experts
    x = (torch.arange(tokens, device="cuda") % 251).to(torch.bfloat16)[:, None].expand(tokens, hidden).contiguous()
    xs = torch.empty(tokens * k, hidden, dtype=torch.bfloat16, device="cuda")
    counts, offsets, perm, pos = outputs(tokens, k, experts)
    qm.qs_dispatch_tokens(ids, x, None, counts, offsets, perm, pos, xs, None, qm.alloc_dispatch_workspace(tokens, k, experts))
    assert torch.equal(xs[:, 0].float(), (perm // k % 251).float()) and torch.equal(xs[:, -1], xs[:, 0])
    out = torch.empty_like(x)
    qm.qs_combine_tokens(xs, pos, None, out)
    assert torch.equal(out, (x.float() * k).bfloat16())


def test_on_another_stream_and_in_a_graph():
    """The chain norm -> dispatch -> combine on a side stream and replayed from a graph gives the same bits."""
    g = gen(12)
    tokens, k, hidden = 6, 4, 256
    x, r, w = torch.randn(tokens, hidden, generator=g).cuda(), torch.randn(tokens, hidden, generator=g).cuda(), torch.rand(hidden, generator=g).cuda()
    ids, wt = routed(tokens, k, 9, g, "random").cuda(), torch.rand(tokens, k, generator=g).cuda()
    q, scale = codes(tokens, hidden)
    xs, ss = codes(tokens * k, hidden)
    total, back = torch.empty_like(x), torch.empty_like(x)
    out = outputs(tokens, k, 9)
    ws = qm.alloc_dispatch_workspace(tokens, k, 9)
    y = torch.randn(tokens * k, hidden, generator=g).cuda()

    def chain():
        qm.qs_rmsnorm_residual(x, r, w, EPS, total, None, q, scale)
        qm.qs_dispatch_tokens(ids, q, scale, *out, xs, ss, ws)
        qm.qs_combine_tokens(y, out[3], wt, back)

    chain()
    torch.cuda.synchronize()
    want = [t.clone() for t in (total, xs.view(torch.uint8), ss, back, *out)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for t in (total, ss, back):
            t.fill_(-5)
        chain()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (total, xs.view(torch.uint8), ss, back, *out)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for t in (total, ss, back):
        t.fill_(-5)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (total, xs.view(torch.uint8), ss, back, *out)))


def test_infinities_and_nans_in_a_silu_block():
    gu = torch.ones(3, 512, device="cuda")
    gu[0, 300] = float("inf")   # up of column 44: block 0
    gu[1, 5] = float("nan")
    q, scale = codes(3, 256)
    qm.qs_silu_mul_quant(gu, q, scale)
    v = q.float() * scale.repeat_interleave(128, 1)
    one = 1 / (1 + np.exp(-1.0))
    assert torch.all(torch.isnan(v[0, :128])) and torch.all((v[0, 128:] - one).abs() <= one * 2.0 ** -4)
    assert torch.isnan(v[1, 5]) and int(torch.isnan(v[1]).sum()) == 1 and torch.all((v[2] - one).abs() <= one * 2.0 ** -4)


@pytest.mark.parametrize("size", [1e-37, 1e-30, 1e-20, 1e-8, 1e8, 1e15])
@pytest.mark.parametrize("eps", [1e-12, 1e-5])
def test_norm_codes_of_tiny_and_huge_rows(size, eps):
    """The codes do not depend on how far the row's factor is from one."""
    x, w = torch.randn(4, 640, generator=gen(3)) * size, torch.rand(640, generator=gen(4)) + 0.5
    q, scale = codes(4, 640)
    qm.qs_rmsnorm_residual(x.cuda(), None, w.cuda(), eps, q=q, q_scale=scale)
    v = x.double() / torch.sqrt(x.double().pow(2).mean(1, keepdim=True) + float(np.float32(eps))) * w.double()
    check_codes(q, scale, v, NORM_SLACK + U)


def test_binding_refuses_wrong_types_shapes_and_strides():
    x, w = torch.zeros(4, 256, device="cuda"), torch.ones(256, device="cuda")
    q, scale = codes(4, 256)
    for call, text in [
            (lambda: qm.qs_rmsnorm_residual(x.half(), None, w, EPS, y=x), "x: torch.float16"),
            (lambda: qm.qs_rmsnorm_residual(x, x[:3], w, EPS, y=x), "residual: shape"),
            (lambda: qm.qs_rmsnorm_residual(x, None, w[:255], EPS, y=x), "weight: shape"),
            (lambda: qm.qs_rmsnorm_residual(x, None, w.double(), EPS, y=x), "weight: torch.float64"),
            (lambda: qm.qs_rmsnorm_residual(x, None, w, EPS, y=torch.zeros(256, 4, device="cuda").t()), "y: expected contiguous columns"),
            (lambda: qm.qs_rmsnorm_residual(x, None, w, EPS, q=q), "come with scales"),
            (lambda: qm.qs_rmsnorm_residual(x, None, w, EPS, q=q, q_scale=scale[:, :1]), "q scale: shape"),
            (lambda: qm.qs_silu_mul_quant(x, q, scale), "gate_up: shape"),
            (lambda: qm.qs_fp8_matmul(q, scale, q, scale, torch.zeros(4, 4, device="cuda"), qm.alloc_fp8_matmul_workspace(4, 4, 256)), "w scale: shape"),
            (lambda: qm.qs_combine_tokens(x, torch.zeros(2, 2, device="cuda"), None, x[:2]), "pos: torch.float32"),
            (lambda: qm.qs_dispatch_tokens(torch.zeros(2, 2, dtype=torch.int32, device="cuda"), x[:2], None, *outputs(2, 2, 4)[:3], x, x, None,
                                           qm.alloc_dispatch_workspace(2, 2, 4)), "pos: torch.float32")]:
        with pytest.raises(ValueError, match=text):
            call()
    flat = torch.zeros(8 * 256 + 8, dtype=torch.uint8, device="cuda")
    off = flat[8:8 + 4 * 256].view(4, 256).view(F8)  # not at 16 bytes
    with pytest.raises(qm.QsError):
        qm.qs_fp8_matmul(off, scale, q, torch.ones(1, 2, device="cuda"), torch.zeros(4, 4, device="cuda"), qm.alloc_fp8_matmul_workspace(4, 4, 256))
    with pytest.raises(qm.QsError):  # a broadcast row
        qm.qs_rmsnorm_residual(x[:1].expand(4, 256), None, w, EPS, y=x)
    with pytest.raises(qm.QsError):
        qm.qs_rmsnorm_residual(x, None, w, EPS)
    torch.cuda.synchronize()
