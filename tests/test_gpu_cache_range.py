"""Attention over the paged cache at the ends of its ranges: value scales of any size, infinities, offsets that are none.

Tolerances are a row's own (a token and head), from its own scores and scales.  A score is off by delta = (d + 8) 2^-23 scale
sum |q k| + 2^-22 |s|, a weight by 2 delta + 2^-21 of itself, a sum over n positions by n 2^-23, and the 16-bit parts of a
weight leave out u_p: 2^-22 with fp32 rows or codes, else 2^-16 (bf16 cache) or 2^-11 (e4m3).  Over e4m3 the argument of a weight's
exponential has the value scale's logarithm in it, up to |log2 scale| + 16 of a rounding of 2^-24; and the smallest step of an
fp16 weight is 2^-24 where the row's largest is 2^3 at least, so each position is off by up to 2^-28 of the largest weighted scale:
    |out - exact| <= u |exact| + (2 delta + n 2^-23 + u_p + 2^-21 + 2^-23 (max |log2 scale| + 16)) sum w |v| + 2^-28 max(w scale) sum |code|
"""
import math

import pytest
import torch

from bit_quantized_moe_router_gb300 import qs_moe as qm
from test_gpu_cache import BF16, E4M3, F32, U, Paged

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def rows64(c, q, scale, window=0):
    """A dict of what is exact and what the tolerances are made of, each per token and head, in 64 bits."""
    heads, group, eight = q.shape[1], q.shape[1] // c.kv, c.kind is E4M3
    r = {n: torch.zeros(q.shape, dtype=torch.float64, device="cuda") for n in ("out", "mass", "floor")}
    r.update({n: torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda") for n in ("size", "most", "lv")})
    r["lse"] = torch.full(q.shape[:2], -INF, dtype=torch.float64, device="cuda")
    for i in range(len(c.lens)):
        k, v, there = c.rows("k", i), c.rows("v", i), c.there(i)
        if eight:
            pages = self_pages(c, i)
            codes = c.v.view(torch.uint8)[pages].view(E4M3).double().flatten(0, 1)
            scales = c.v_scale[pages].double().flatten(0, 1)
        for j in range(c.new[i]):
            t, p = int(c.offsets[i]) + j, int(c.starts[i]) + j
            at = torch.arange(k.shape[0], device="cuda")
            seen = (there & (at >= (max(0, p + 1 - window) if window else 0)) & (at <= p)).nonzero().flatten()
            if not seen.numel():
                continue
            kk, vv = k[seen].repeat_interleave(group, 1), v[seen].repeat_interleave(group, 1)
            x = q[t].double()
            s = torch.einsum("hd,lhd->hl", x, kk) * scale
            w = torch.softmax(s, 1)
            r["out"][t], r["lse"][t] = torch.einsum("hl,lhd->hd", w, vv), torch.logsumexp(s, 1)
            r["mass"][t] = torch.einsum("hl,lhd->hd", w, vv.abs())
            r["size"][t] = (torch.einsum("hd,lhd->hl", x.abs(), kk.abs()) * abs(scale)).amax(1)
            r["most"][t] = s.abs().amax(1)
            if eight:
                u = scales[seen].repeat_interleave(group, 1).T  # [heads, positions]
                r["lv"][t] = torch.log2(u).abs().clamp_max(150.0).amax(1)
                r["floor"][t] = (w * u).amax(1)[:, None] * codes[seen].repeat_interleave(group, 1).abs().sum(0)
    return r


def self_pages(c, i):
    there = c.there_pages(i)
    return torch.where(there, c.table[i].long(), torch.zeros_like(c.table[i].long()))


def tolerances(c, r, out_type, wide):
    """(of the output, of the log-sum)"""
    eight, n = c.kind is E4M3, max(c.lens)
    delta = (c.d + 8) * 2.0 ** -23 * r["size"] + 2.0 ** -22 * r["most"]
    args = 2.0 ** -23 * (r["lv"] + 16) if eight else torch.zeros_like(delta)
    each = 2 * delta + n * 2.0 ** -23 + (2.0 ** -22 if wide else 2.0 ** -11 if eight else 2.0 ** -16) + 2.0 ** -21 + args
    out = U[out_type] * r["out"].abs() + each[..., None] * r["mass"] + 2.0 ** -28 * r["floor"] + 2.0 ** -133
    return out, delta + n * 2.0 ** -23 + 2.0 ** -20 + args + 2.0 ** -22 * r["lse"].abs()


def attend(c, q, scale, out_type, window=0, codes=False):
    """(out or None, lse, codes or None, their scales) of every token of c."""
    heads, most_new = q.shape[1], max(c.new)
    out = None if codes else torch.full(q.shape, 7.0, dtype=out_type, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    q8 = torch.zeros(q.shape[0], heads * c.d, dtype=E4M3, device="cuda") if codes else None
    s8 = torch.zeros(q.shape[0], heads * c.d // 128, device="cuda") if codes else None
    qm.qs_cache_attention(c.cache, c.seqs, q, scale, out, qm.alloc_cache_attention_workspace(heads, c.kv, c.d, most_new), max_new=most_new,
                          window=window, lse=lse, codes=q8, codes_scale=s8)
    return out, lse, q8, s8


def check_rows(c, q, out_type=None, window=0, scale=None, codes=False):
    out_type = F32 if codes else out_type or q.dtype
    scale = 1.3 / math.sqrt(c.d) if scale is None else scale
    out, lse, q8, s8 = attend(c, q, scale, out_type, window, codes)
    r = rows64(c, q, scale, window)
    tol, tol_lse = tolerances(c, r, out_type, codes or q.dtype is F32 or out_type is F32)
    if codes:  # a code's rounding, or half of the smallest step
        n = q.shape[0]
        scales = s8.double().repeat_interleave(128, 1).view(q.shape)
        out = q8.double().view(q.shape) * scales
        tol = 1.07 * tol + 2.0 ** -4 * r["out"].abs() + 2.0 ** -10 * scales
        assert n == out.shape[0]
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    worst = ((out.double() - r["out"]).abs() / tol).max().item()
    assert worst <= 1.0, f"out: {worst:.3g} of the tolerance"
    worst = ((lse.double() - r["lse"]).abs() / tol_lse).max().item()
    assert worst <= 1.0, f"lse: {worst:.3g} of the tolerance"


FORMS = [(BF16, BF16, False), (F32, F32, False), (BF16, F32, False), (F32, BF16, False), (BF16, BF16, True)]
IDS = ["bf16", "f32", "bf16-f32", "f32-bf16", "codes"]


def queries(c, heads, kind=BF16, seed=1):
    return torch.randn(c.tokens, heads, c.d, generator=torch.Generator().manual_seed(seed)).to(kind).cuda()


# ------------------------------------------------------------------ value scales

@pytest.mark.parametrize("form", FORMS, ids=IDS)
@pytest.mark.parametrize("group", [1, 4, 16])
@pytest.mark.parametrize("new,window", [(1, 0), (4, 0), (4, 57), (1, 57), (4, 2)])
@pytest.mark.parametrize("power", [-100, -60, -40, -16, 0, 60, 90, "any"])
def test_value_scales_of_any_size(power, new, window, group, form):
    """Positions that only some of an item's rows see count for the running maximum as the others do."""
    q_type, out_type, codes = form
    c = Paged([200, new, 60, 33], [new, new, new, max(new - 1, 1)], E4M3, kv=2, d=128, page=16)
    if power == "any":
        c.v_scale *= torch.exp2(torch.randint(-40, 40, c.v_scale.shape, generator=torch.Generator().manual_seed(5)).cuda().float())
    else:
        c.v_scale *= 2.0 ** power * 16.0
        c.v_scale.clamp_(2.0 ** (power - 2), 2.0 ** (power + 2))  # (a NaN of a slot that nobody has stays)
    check_rows(c, queries(c, 2 * group, q_type), out_type, window, codes=codes)


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("form", FORMS[:4], ids=IDS[:4])
def test_quiet_rows_beside_loud_ones(kind, form):
    """A row of zeros and rows next to them have their own tolerance, whatever the others' scores are."""
    c = Paged([200, 100], [1, 1], kind, kv=2, d=64, page=16)
    q = 50.0 * torch.randn(2, 8, 64, generator=torch.Generator().manual_seed(3))
    q[0, 0] = 0.0
    q[0, 1] *= 2.0 ** -60
    q[1, 1] *= 2.0 ** -120
    q[1, 2] *= 0.01
    check_rows(c, q.to(form[0]).cuda(), form[1])
    check_rows(c, q.to(form[0]).cuda(), form[1], scale=-0.2)


@pytest.mark.parametrize("new", [1, 3])
@pytest.mark.parametrize("value", [0.0, 2.0 ** -100])
def test_log_sums_of_many_small_values(value, new):
    """2^22 positions whose values are all zero, or as small as scales get: 64 of them, over and over."""
    n, d, page = 1 << 22, 16, 64
    k, v = torch.zeros(1, page, 1, d, device="cuda"), torch.full((1, page, 1, d), value, device="cuda")
    k8, v8 = torch.zeros(1, page, 1, d, dtype=E4M3, device="cuda"), torch.zeros(1, page, 1, d, dtype=E4M3, device="cuda")
    ks, vs = torch.zeros(1, page, 1, device="cuda"), torch.zeros(1, page, 1, device="cuda")
    cache = qm.make_cache(k8, v8, ks, vs)
    qm.qs_cache_write(cache, qm.make_seqs(torch.zeros(1, 1, dtype=torch.int32, device="cuda"), None, torch.tensor([0, page], dtype=torch.int32, device="cuda")), k[0], v[0])
    seqs = qm.make_seqs(torch.zeros(1, n // page, dtype=torch.int32, device="cuda"), torch.tensor([n - new], dtype=torch.int32, device="cuda"),
                        torch.tensor([0, new], dtype=torch.int32, device="cuda"))
    q = torch.ones(new, 4, d, device="cuda").to(BF16)
    out, lse = torch.full((new, 4, d), 7.0, dtype=BF16, device="cuda"), torch.empty(new, 4, device="cuda")
    qm.qs_cache_attention(cache, seqs, q, 0.25, out, qm.alloc_cache_attention_workspace(4, 1, d, new), max_new=new, lse=lse)
    # every weight is the same power of two, and sums of them have few bits: what is left is the logarithm's own
    want = torch.log(torch.arange(n - new + 1, n + 1, dtype=torch.float64, device="cuda"))
    assert ((lse.double() - want[:, None]).abs() <= 2.0 ** -16 * want[:, None]).all(), lse
    assert ((out.double() - value).abs() <= 2.0 ** -4 * value).all()


# ------------------------------------------------------------------ infinities

def special(c, i, p, name, value):
    """Position p of sequence i gets this value in every head."""
    getattr(c, name)[int(c.table[i, p // c.page]), p % c.page] = value


@pytest.mark.parametrize("form", FORMS, ids=IDS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group,new", [(1, 1), (4, 1), (12, 1), (20, 1), (3, 4), (8, 8)])
def test_scores_of_minus_infinity(group, new, d, form):
    """Where every score is -infinity a row is zeros, and its log-sum -infinity; one such position among others counts nothing."""
    q_type, out_type, codes = form
    if codes and d < 128:
        d = 128
    c = Paged([30, 70, 25], [new, new, new], BF16, kv=2, d=d, page=16, garbage=False)
    c.k[c.table[0].long()[c.table[0] >= 0]] = -INF
    special(c, 1, 5, "k", -INF)
    special(c, 2, 25 - new, "k", -INF)   # the first new token's own
    q = (torch.rand(c.tokens, 2 * group, d, generator=torch.Generator().manual_seed(2)) + 0.5).to(q_type)
    q[:, :, 1] = 1.0  # held by one part
    q = q.cuda()
    scale = 1.0 / d
    out, lse, q8, s8 = attend(c, q, scale, out_type, codes=codes)
    if codes:
        out = q8.double().view(q.shape) * s8.double().repeat_interleave(128, 1).view(q.shape)
    assert out[:new].double().count_nonzero() == 0 and (lse[:new] == -INF).all()
    # the others' as if the position were not there: one key that no row sees a difference of
    finite = Paged([30, 70, 25], [new, new, new], BF16, kv=2, d=d, page=16, garbage=False)
    special(finite, 1, 5, "k", -1.0e30)
    special(finite, 2, 25 - new, "k", -1.0e30)
    want, want_lse, w8, t8 = attend(finite, q, scale, out_type, codes=codes)
    if codes:
        want = w8.double().view(q.shape) * t8.double().repeat_interleave(128, 1).view(q.shape)
    assert torch.equal(out[new:], want[new:]) and torch.equal(lse[new:], want_lse[new:])
    assert torch.isfinite(out[new:]).all() and torch.isfinite(lse[new:]).all()


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("form", FORMS[:4], ids=IDS[:4])
def test_queries_of_minus_infinity(kind, form):
    """Queries of -infinity over positive keys: every score is -infinity."""
    c = Paged([30, 20], [1, 1], kind, kv=2, d=64, page=16, garbage=False)
    c.k.copy_(c.k.float().abs().clamp_min(0.25).to(kind))
    q = queries(c, 8, form[0])
    q[0, 3] = -INF
    q[0, 5, 7] = -INF
    out, lse, _, _ = attend(c, q, 0.1, form[1])
    want, want_lse, _, _ = attend(c, queries(c, 8, form[0]), 0.1, form[1])
    quiet = torch.zeros(2, 8, dtype=torch.bool, device="cuda")
    quiet[0, 3] = quiet[0, 5] = True
    assert out[quiet].count_nonzero() == 0 and (lse[quiet] == -INF).all()
    assert torch.equal(out[~quiet], want[~quiet]) and torch.equal(lse[~quiet], want_lse[~quiet])


@pytest.mark.parametrize("form", FORMS[:4], ids=IDS[:4])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group,new", [(1, 1), (4, 1), (12, 1), (20, 1), (3, 4), (8, 8)])
def test_values_that_are_infinite(group, new, d, form):
    """An infinite value makes its column infinite for the rows that see it (a NaN where both signs are seen), and no other column."""
    c = Paged([30, 70, 5000], [new, new, new], BF16, kv=2, d=d, page=16, garbage=False)
    places = [(1, 5, 3, INF), (1, 69, 4, -INF), (1, 20, 8, INF), (1, 40, 8, -INF), (2, 1, d - 1, -INF), (2, 4999, 0, INF), (2, 2500, 1, INF)]
    q = queries(c, 2 * group, form[0])
    clean, clean_lse, _, _ = attend(c, q, 1.0 / math.sqrt(d), form[1])
    expect = clean.double().clone()
    for i, p, col, value in places:
        c.v[int(c.table[i, p // 16]), p % 16, :, col] = value
        first = max(0, p - (c.lens[i] - new))   # the first of the sequence's tokens that sees it
        t0, t1 = int(c.offsets[i]) + first, int(c.offsets[i + 1])
        expect[t0:t1, :, col] = torch.where(torch.isinf(expect[t0:t1, :, col]), NAN, value)
    out, lse, _, _ = attend(c, q, 1.0 / math.sqrt(d), form[1])
    assert torch.equal(lse, clean_lse)
    assert torch.equal(torch.isnan(out), torch.isnan(expect))
    assert torch.equal(out.double().nan_to_num(0.0), expect.nan_to_num(0.0))


@pytest.mark.parametrize("power", [100, 113, 116, 120, 124])
@pytest.mark.parametrize("form", FORMS, ids=IDS)
def test_large_queries_over_small_keys(power, form):
    """Queries next to fp32's end over e4m3 keys next to its beginning: scores as anywhere."""
    q_type, out_type, codes = form
    c = Paged([60, 33], [1, 1], E4M3, kv=2, d=128, page=16)
    c.k_scale.copy_(torch.where(torch.isnan(c.k_scale), NAN, 2.0 ** -(power - 1)))
    q = queries(c, 8, F32)
    check_rows(c, (q / q.abs().max() * 2.0 ** power * 7.9).to(q_type), out_type, codes=codes, scale=0.02)


# ------------------------------------------------------------------ offsets from device memory

@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("offsets", [[-5, 2, 1, 900], [1, -2 ** 31, 2 ** 31 - 1, 3], [2 ** 31 - 1, -2 ** 31, 0, 3], [3, 2, 1, 0], [-2 ** 31, -2 ** 31, -2 ** 31, -2 ** 31],
                                     [3, -2 ** 31 + 2, 5, -2 ** 31], [0, 1, -2 ** 31 + 1, -1], [2 ** 31 - 1] * 4], ids=str)
def test_offsets_that_are_no_offsets(offsets, kind):
    """Offsets outside the rows and not ascending: nothing outside the rows is read or written, and what is written is finite."""
    c = Paged([40, 40, 40], [1, 1, 1], kind, kv=2, d=64, page=16, garbage=False)
    if kind is E4M3:  # what lies behind the 40 may be seen
        c.k_scale.nan_to_num_(0.05), c.v_scale.nan_to_num_(0.05)
    c.offsets.copy_(torch.tensor(offsets, dtype=torch.int32))
    room, n, heads = 300, 3, 4
    q = torch.full((n + 2 * room, heads, 64), NAN, device="cuda").to(BF16)  # beside the rows NaN, which no row may have seen
    q[room:room + n] = torch.randn(n, heads, 64, device="cuda").to(BF16)
    out, lse = torch.full(q.shape, 7.0, dtype=BF16, device="cuda"), torch.full(q.shape[:2], 7.0, device="cuda")
    inside = slice(room, room + n)
    for most_new in (1, 4, 256):
        qm.qs_cache_attention(c.cache, c.seqs, q[inside], 0.1, out[inside], qm.alloc_cache_attention_workspace(heads, 2, 64, most_new), max_new=most_new, lse=lse[inside])
        assert torch.isfinite(out).all() and torch.isfinite(lse[inside]).logical_or(lse[inside] == -INF).all()
        for x in (out, lse):
            assert (x[:room] == 7.0).all() and (x[room + n:] == 7.0).all()
    # reading leaves the same rows alone, writing stores no NaN
    rows = torch.full((n + 2 * room, 2, 64), 7.0, device="cuda"), torch.full((n + 2 * room, 2, 64), 7.0, device="cuda")
    before = c.k.view(torch.uint8).clone()
    qm.qs_cache_read(c.cache, c.seqs, rows[0][inside], rows[1][inside])
    for x in rows:
        assert (x[:room] == 7.0).all() and (x[room + n:] == 7.0).all()
    new = torch.full((n + 2 * room, 2, 64), NAN, device="cuda")
    new[inside] = 1.0
    qm.qs_cache_write(c.cache, c.seqs, new[inside], new[inside])
    changed = (before != c.k.view(torch.uint8)).flatten(2).any(2)
    assert changed.sum() <= n and torch.isfinite(c.k.float()[changed]).all()


# ------------------------------------------------------------------ layouts

@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("one", [0, 1, 2])
def test_strides_of_dimensions_of_one_do_not_count(one, kind):
    """Keys and values, and their scales, that differ in such a stride alone are one layout: what is written comes back."""
    shape = [3, 16, 2, 64]
    shape[one] = 1

    def odd(t):  # the same elements, with another stride where the size is one
        strides = list(t.stride())
        strides[one] = 7 * strides[one] + 5
        return t.as_strided(t.shape, strides)

    k, v = torch.zeros(shape, device="cuda").to(kind), odd(torch.zeros(shape, device="cuda").to(kind))
    scales = (torch.zeros(shape[:3], device="cuda"), odd(torch.zeros(shape[:3], device="cuda"))) if kind is E4M3 else ()
    assert k.stride() != v.stride()
    n = shape[0] * shape[1]
    seqs = qm.make_seqs(torch.arange(shape[0], dtype=torch.int32, device="cuda")[None], None, torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    rows = [torch.randint(-8, 9, (n, shape[2], 64), device="cuda").float() for _ in range(2)]
    for x in rows:
        x[:, :, 0] = 448.0 if kind is E4M3 else 1.0  # a scale of one
    for pair in ((k, v, *scales), (v, k, *scales[::-1])):
        cache = qm.make_cache(*pair)
        back = [torch.empty_like(x) for x in rows]
        qm.qs_cache_write(cache, seqs, *rows)
        qm.qs_cache_read(cache, seqs, *back)
        for x, y in zip(rows, back):
            assert ((x - y).abs() <= 2.0 ** -20 * x.abs()).all()
    with pytest.raises(ValueError, match="strides"):  # strides that count
        qm.make_cache(k, torch.zeros([2 * x for x in shape], device="cuda").to(kind)[:shape[0], :shape[1], :shape[2], :64], *scales)
