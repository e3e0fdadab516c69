"""Row operators at the ends of fp32's range, on the GPU against 64-bit forms.

Tolerances: 2^-24 (U) of the value a rounding, 2^-4 of the value or 2^-10 of the scale for a code, as the operators'
other tests count them.
"""
import pytest
import torch

from bit_quantized_moe_router_gb300 import qs_moe as qm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F8 = torch.float8_e4m3fn
LEAST = 2.0 ** -100 / 448  # the scale of a block of zeros


def gen(seed):
    return torch.Generator().manual_seed(seed)


def codes(rows, cols):
    q = torch.full((rows, cols), 0x55, dtype=torch.uint8, device="cuda").view(F8)
    return q, torch.full((rows, (cols + 127) // 128), -1.0, device="cuda")


@pytest.mark.parametrize("hidden", [128, 640, 641, 2048, 4096, 8192, 16384])
def test_codes_of_rows_whose_sum_of_squares_is_infinite(hidden):
    """Codes are made of v: an infinity's own v is a NaN (infinity times the factor 0), all others are 0, as y has them."""
    x = torch.randn(5, hidden, generator=gen(hidden))
    x[1, 100] = float("inf")
    x[2, 3] = -float("inf")
    x[3, 7] = 1e25  # finite; its square is not
    w = 0.5 + torch.rand(hidden, generator=gen(1))
    q, scale = codes(5, hidden)
    y = torch.empty(5, hidden, device="cuda")
    qm.qs_rmsnorm_residual(x.cuda(), None, w.cuda(), 1e-5, y=y, q=q, q_scale=scale)
    nan = torch.zeros(5, hidden, dtype=torch.bool)
    nan[1, 100] = nan[2, 3] = True
    got, y, scale = q.float().cpu(), y.cpu(), scale.cpu()
    assert torch.equal(torch.isnan(y), nan) and torch.equal(torch.isnan(got), nan)
    flat = torch.zeros(5, 1, dtype=torch.bool)
    flat[1:4] = True
    assert torch.all(y[(flat & ~nan)] == 0) and torch.all(got[(flat & ~nan)] == 0)
    # 448 goes in as its rounded reciprocal: two roundings
    assert torch.all((scale[1:4].double() - LEAST).abs() <= 2 * U * LEAST)
    assert torch.all(torch.isfinite(scale[[0, 4]])) and torch.all(got[[0, 4]].abs().amax(1) == 448)
    alone = codes(5, hidden)
    qm.qs_rmsnorm_residual(x.cuda(), None, w.cuda(), 1e-5, q=alone[0], q_scale=alone[1])
    assert torch.equal(alone[0].view(torch.uint8), q.view(torch.uint8)) and torch.equal(alone[1].cpu(), scale)


@pytest.mark.parametrize("hidden", [264, 1001, 2048, 4096, 16384])
@pytest.mark.parametrize("size,eps", [(1e-13, 0.0), (1e-17, 0.0), (1e-13, 1e-30), (1e-8, 1e-20), (1e8, 1e-5), (1e14, 1e-5), (1e15, 1e-5), (1e16, 1e-5)])
def test_norm_gradient_of_tiny_and_huge_rows(hidden, size, eps):
    """dx and dweight hold where 1 / rms cubed leaves fp32 (the sum of squares does not, at these sizes)."""
    rows, g = 5, gen(hidden)
    s, w = torch.randn(rows, hidden, generator=g) * size, 0.5 + torch.rand(hidden, generator=g)
    dy = torch.randn(rows, hidden, generator=g) + 0.1 * s / size  # a part along s, so that the mean of dy * s counts
    dsum = torch.randn(rows, hidden, generator=g) / size
    dx, dw = torch.empty(rows, hidden, device="cuda"), torch.empty(hidden, device="cuda")
    qm.qs_rmsnorm_residual_backward(s.cuda(), w.cuda(), eps, dy.cuda(), dsum.cuda(), dx, dw, qm.alloc_rmsnorm_backward_workspace(hidden))
    eps = float(torch.tensor(eps, dtype=torch.float32))
    s, w, dy, dsum = s.double(), w.double(), dy.double(), dsum.double()
    rho = 1 / torch.sqrt(s.pow(2).mean(1, keepdim=True) + eps)
    unit = s * rho
    along = (w * dy * unit).mean(1, keepdim=True)
    want = rho * (w * dy - unit * along) + dsum
    terms = rho * ((w * dy).abs() + unit.abs() * (w * dy * unit).abs().mean(1, keepdim=True)) + dsum.abs()
    # the row's two sums at most 48 U each, the first under a root; rho three times, a rounding a product
    assert torch.all((dx.cpu().double() - want).abs() <= 160 * U * terms)
    assert torch.all((dw.cpu().double() - (dy * unit).sum(0)).abs() <= 160 * U * (dy * unit).abs().sum(0))


@pytest.mark.parametrize("ffn", [5, 128, 512, 1001])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate", [-1.0, -9.0, -20.0, -40.0, -80.0, -86.0])
def test_silu_of_gates_far_below_zero(ffn, kind, gate):
    """A block's scale and codes are as near where all gates are far below zero as elsewhere.

    Units in the last place (2 U): the exponential 2 and its argument's remainder half of one; 1 + exp, product with the
    gate and product with up half each; quotient 2: under 12 U together, and the scale's own two roundings.
    """
    rows = 40
    g = gen(ffn)
    gu = torch.empty(rows, 2 * ffn)
    gu[:, :ffn] = gate + 0.5 * torch.rand(rows, ffn, generator=g)
    gu[:, ffn:] = torch.randn(rows, ffn, generator=g) * 1e12  # so that no block's largest value is below 2^-100
    gu = gu.to(kind)
    q, scale = codes(rows, ffn)
    qm.qs_silu_mul_quant(gu.cuda(), q, scale)
    a, b = gu.double().chunk(2, 1)
    v = a / (1 + torch.exp(-a)) * b
    nb = scale.shape[1]
    wide = torch.zeros(rows, nb * 128, dtype=torch.float64)
    wide[:, :ffn] = v
    amax = wide.abs().view(rows, nb, 128).amax(2)
    got = scale.cpu().double()
    assert float(amax.min()) > 2.0 ** -100
    assert torch.all((got - amax / 448).abs() <= 14 * U * amax / 448)
    per = got.repeat_interleave(128, 1)[:, :ffn]
    assert torch.all((q.cpu().float().double() * per - v).abs() <= v.abs() * (2.0 ** -4 + 16 * U) + per * 2.0 ** -10)


def test_silu_of_infinite_and_nan_gates():
    inf, nan = float("inf"), float("nan")
    gu = torch.zeros(5, 256)
    gu[:, :128] = torch.tensor([200.0, inf, -inf, nan, -1e30])[:, None]
    gu[:, 128:] = 2.0
    q, scale = codes(5, 128)
    qm.qs_silu_mul_quant(gu.cuda(), q, scale)
    v = (q.float() * scale).cpu()
    assert torch.all((v[0] - 400).abs() <= 400 * 4 * U) and torch.all(torch.isnan(v[1:4])) and torch.all(v[4] == 0)


def test_dispatch_with_a_workspace_made_for_more_tokens():
    """Calls on both sides of the size from which chunks of the sort grow (262144 entries), in one workspace."""
    k, experts = 8, 256
    ws = qm.alloc_dispatch_workspace(33000, k, experts)
    for tokens in (33000, 32769, 32768, 32700, 600, 512, 1):
        ids = torch.randint(-1, experts, (tokens, k), generator=gen(tokens), dtype=torch.int32).cuda()
        i32 = dict(dtype=torch.int32, device="cuda")
        counts, offsets, perm, pos = torch.empty(experts, **i32), torch.empty(experts + 1, **i32), torch.empty(tokens * k, **i32), torch.empty(tokens, k, **i32)
        qm.qs_dispatch_tokens(ids, None, None, counts, offsets, perm, pos, None, None, ws)
        flat = torch.where(ids < 0, experts, ids).flatten().long()
        order, total = torch.sort(flat, stable=True).indices, int((flat < experts).sum())
        assert torch.equal(counts.long(), torch.bincount(flat, minlength=experts + 1)[:experts])
        assert torch.equal(offsets[1:].long(), counts.long().cumsum(0)) and int(offsets[0]) == 0
        assert torch.equal(perm[:total].long(), order[:total]) and torch.all(perm[total:] == -1)
        assert torch.equal(pos.flatten()[order[:total]].long(), torch.arange(total, device="cuda")) and torch.all(pos[ids < 0] == -1)
