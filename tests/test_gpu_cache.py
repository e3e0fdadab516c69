"""The paged key-value cache: writing, reading back and attention against plain forms in 64 bits.

Tolerances.  A rounding to a type is off by at most u = eps / 2 of the value.  Attention, per output column, with w the
softmax's weights: the score is a sum of d products and one or two scales, each fp32 step off by at most 2^-23 of the sum
of magnitudes (tensor cores cut rather than round), so a score is off by delta = (d + 8) 2^-23 max_i scale sum |q k_i| plus
2^-22 |s| for the base-2 argument, and a weight by 2 delta + 2^-21 (two exponentials) of itself; a sum over n positions
adds n 2^-23; the 16-bit parts of a weight leave out u_p of it.  Altogether
    |out - exact| <= u |exact| + (2 delta + n 2^-23 + u_p + 2^-21) sum w |v|
with u_p = 2^-16 (bf16 cache) or 2^-11 (e4m3) for bf16 queries and output, 2^-22 with any in fp32.
"""
import math

import pytest
import torch

from bit_quantized_moe_router_gb300 import qs_moe as qm

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = {t: torch.finfo(t).eps / 2 for t in (BF16, F32)}


class Paged:
    """A cache of random values, sequences of these lengths on shuffled pages, and garbage (NaN and infinities) in
    every slot that no sequence has."""

    def __init__(self, lens, new, kind=BF16, kv=2, d=64, page=16, seed=0, layout="slots", spare_pages=2, shared=False, garbage=True):
        g = torch.Generator().manual_seed(seed)
        n = len(lens)
        self.lens, self.new, self.kind, self.kv, self.d, self.page = list(lens), list(new), kind, kv, d, page
        each = [-(-x // page) for x in lens]
        width = max(max(each), 1)
        total = sum(each) + spare_pages
        order = torch.randperm(total, generator=g)
        table, at = torch.full((n, width + 3), -1, dtype=torch.int32), 0
        for i, e in enumerate(each):
            table[i, :e] = order[at:at + e].int()
            at += e
        self.table = table.cuda()[:, :width]  # rows of a wider table
        self.starts = torch.tensor([x - m for x, m in zip(lens, new)], dtype=torch.int32).cuda()
        self.offsets = torch.tensor([0] + list(new), dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
        self.tokens = sum(new)
        shape = (total, page, kv, d)
        k, v = torch.randn(shape, generator=g), torch.randn(shape, generator=g)
        used = torch.zeros(total, page, dtype=torch.bool)
        for i, x in enumerate(lens):
            for p in range(each[i]):
                used[table[i, p].long(), : max(0, min(page, x - p * page))] = True
        if garbage:
            junk = torch.tensor([float("nan"), float("inf"), -float("inf")])[torch.randint(0, 3, shape, generator=g)]
            k, v = torch.where(used[..., None, None], k, junk), torch.where(used[..., None, None], v, junk)
        self.k_scale = self.v_scale = None
        if kind is E4M3:
            ks, vs = torch.exp(torch.randn(shape[:3], generator=g)) * 0.05, torch.exp(torch.randn(shape[:3], generator=g)) * 0.05
            self.k_scale, self.v_scale = (torch.where(used[..., None], s, torch.full((), float("nan"))).cuda() for s in (ks, vs))
            k, v = k * 20, v * 20
        if layout == "both":  # halves of one buffer
            both = torch.stack([k, v], 1).to(kind).cuda()
            self.k, self.v = both[:, 0], both[:, 1]
        elif layout == "heads":  # a head's slots side by side
            self.k, self.v = (x.transpose(1, 2).contiguous().to(kind).cuda().transpose(1, 2) for x in (k, v))
        else:
            self.k, self.v = k.to(kind).cuda(), v.to(kind).cuda()
        self.cache = qm.make_cache(self.k, self.v, self.k_scale, self.v_scale)
        self.seqs = qm.make_seqs(self.table, self.starts, self.offsets)

    def rows(self, name, i):
        """Sequence i's cached values in 64 bits, [positions, heads, columns]; a position whose page is not there is NaN."""
        there, pages = self.there_pages(i), self.table[i].long()
        pages = torch.where(there, pages, torch.zeros_like(pages))
        x = getattr(self, name)
        all_rows = x.view(torch.uint8)[pages].view(E4M3).double() if self.kind is E4M3 else x[pages].double()
        if self.kind is E4M3:
            all_rows = all_rows * getattr(self, name + "_scale")[pages].double()[..., None]
        all_rows = torch.where(there[:, None, None, None], all_rows, torch.full((), float("nan"), dtype=torch.float64, device="cuda"))
        return all_rows.flatten(0, 1)

    def there_pages(self, i):
        return (self.table[i] >= 0) & (self.table[i] < self.k.shape[0])

    def there(self, i):
        return self.there_pages(i).repeat_interleave(self.page)


def attend64(c, q, scale, window=0):
    """(out, lse, sum of w |v|, largest scale * sum |q k|, largest |score|) in 64 bits, token by token."""
    heads, group = q.shape[1], q.shape[1] // c.kv
    out, mass = (torch.zeros(q.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    size, most = 0.0, 0.0
    for i in range(len(c.lens)):
        k, v, there = c.rows("k", i), c.rows("v", i), c.there(i)
        for j in range(c.new[i]):
            t, p = int(c.offsets[i]) + j, int(c.starts[i]) + j
            lo = max(0, p + 1 - window) if window else 0
            at = torch.arange(k.shape[0], device="cuda")
            seen = (there & (at >= lo) & (at <= p)).nonzero().flatten()
            if not seen.numel():
                continue
            kk, vv = k[seen].repeat_interleave(group, 1), v[seen].repeat_interleave(group, 1)
            x = q[t].double()
            s = torch.einsum("hd,lhd->hl", x, kk) * scale
            w = torch.softmax(s, 1)
            out[t], mass[t], lse[t] = torch.einsum("hl,lhd->hd", w, vv), torch.einsum("hl,lhd->hd", w, vv.abs()), torch.logsumexp(s, 1)
            size = max(size, float((torch.einsum("hd,lhd->hl", x.abs(), kk.abs()) * abs(scale)).max()))
            most = max(most, float(s.abs().max()))
    return out, lse, mass, size, most


def bounds(c, q, out_type, wide, exact, mass, size, most):
    u_p = 2.0 ** -22 if wide else 2.0 ** -11 if c.kind is E4M3 else 2.0 ** -16
    delta = (c.d + 8) * 2.0 ** -23 * size + 2.0 ** -22 * most
    each = 2 * delta + max(c.lens) * 2.0 ** -23 + u_p + 2.0 ** -21
    return U[out_type] * exact.abs() + each * mass + 1e-30, delta + max(c.lens) * 2.0 ** -23 + 2.0 ** -20


def check(c, heads, q_type=BF16, out_type=None, window=0, scale=None, seed=1, max_new=None, codes=False, workspace=None, q=None, spare=0):
    out_type = out_type or q_type
    g = torch.Generator().manual_seed(seed)
    scale = 1.3 / math.sqrt(c.d) if scale is None else scale
    q = torch.randn(c.tokens + spare, heads, c.d, generator=g).to(q_type).cuda() if q is None else q
    out = torch.full(q.shape, 7.0, dtype=out_type, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    most_new = max_new or max(c.new)
    ws = workspace if workspace is not None else qm.alloc_cache_attention_workspace(heads, c.kv, c.d, most_new)
    qm.qs_cache_attention(c.cache, c.seqs, q, scale, out, ws, max_new=most_new, window=window, lse=lse)
    exact, exact_lse, mass, size, most = attend64(c, q, scale, window)
    tol, tol_lse = bounds(c, q, out_type, q_type is F32 or out_type is F32, exact, mass, size, most)
    done = torch.zeros(q.shape[0], dtype=torch.bool)
    for i, m in enumerate(c.new):
        done[int(c.offsets[i]): int(c.offsets[i]) + min(m, most_new)] = True
    done = done.cuda()
    err = (out.double() - exact).abs()
    assert not torch.isnan(out[done]).any()
    worst = (err[done] / tol[done]).max().item() if done.any() else 0.0
    assert worst <= 1.0, f"out: {worst:.3g} of the tolerance"
    assert (out[~done] == 7.0).all() and (lse[~done] == 7.0).all()
    empty = torch.isinf(exact_lse)
    assert (torch.isinf(lse[done]) == empty[done]).all() and (lse[done][empty[done]] < 0).all()
    ok = done[:, None] & ~empty
    assert ((lse.double() - exact_lse).abs()[ok] <= tol_lse + 2.0 ** -22 * exact_lse.abs()[ok]).all()
    assert ws[256:256 + 1920].count_nonzero() == 0  # the counters are zero between calls
    return q, out, lse


# ------------------------------------------------------------------ attention

LENS = [[1], [2], [15], [16], [17], [33], [130], [513], [1, 40, 0, 7], [300, 1, 64, 65, 129, 16]]


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_attention_lengths(kind, lens):
    new = [min(1, x) for x in lens]
    check(Paged(lens, new, kind, kv=2, d=128, page=16), 8)


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [16, 32, 48, 64, 80, 112, 128, 144, 192, 240, 256])
@pytest.mark.parametrize("q_type", [BF16, F32], ids=["q16", "q32"])
def test_attention_head_sizes(kind, d, q_type):
    check(Paged([70, 5, 200], [1, 1, 1], kind, kv=2, d=d, page=16), 6, q_type)


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group,new", [(1, 1), (8, 1), (9, 1), (16, 1), (17, 1), (40, 1), (65, 1), (1, 8), (3, 5), (2, 8), (8, 8), (5, 13), (1, 70)])
def test_attention_groups_and_drafted_tokens(kind, d, group, new):
    c = Paged([new + 90, new, new + 1], [new, max(new - 1, 1), new], kind, kv=2, d=d, page=16)
    check(c, 2 * group, spare=3)
    if group * new <= 64:
        check(c, 2 * group, F32, BF16)
        check(c, 2 * group, BF16, F32)


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("page", [1, 3, 7, 16, 17, 64, 100, 1000])
def test_attention_page_sizes(kind, page):
    check(Paged([121, 33, 250], [2, 1, 3], kind, kv=3, d=64, page=page), 6)


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 50, 129, 100000])
@pytest.mark.parametrize("heads,d", [(2, 128), (16, 64), (24, 256)])
def test_attention_windows(kind, window, heads, d):
    check(Paged([121, 3, 250, 16], [5, 3, 1, 4], kind, kv=2, d=d, page=8), heads, window=window)


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_attention_pages_that_are_not_there(kind):
    c = Paged([100, 100, 100, 20], [3, 3, 3, 2], kind, kv=2, d=64, page=10)
    c.table[0, 2] = -1                # in the middle
    c.table[1, :] = 2 ** 31 - 1       # none at all: zeros and -inf
    c.table[2, 9] = c.k.shape[0]      # the last one, and the new tokens with it
    c.table[3, 0] = -2 ** 31
    _, out, lse = check(c, 8)
    assert out[3:6].count_nonzero() == 0 and (lse[3:6] == -math.inf).all()


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("layout", ["slots", "heads", "both"])
def test_attention_layouts(kind, layout):
    check(Paged([77, 130], [2, 1], kind, kv=4, d=80, page=16, layout=layout), 8)


@pytest.mark.parametrize("kind,d", [(BF16, 256), (E4M3, 256), (E4M3, 128), (BF16, 64)])
@pytest.mark.parametrize("lens", [[5000], [9001, 3], [20000], [1] * 300, [300] * 40 + [0, 1, 2]], ids=lambda x: f"{len(x)}x{max(x)}")
def test_attention_is_split_and_joined(kind, d, lens):
    c = Paged(lens, [min(1, x) for x in lens], kind, kv=2, d=d, page=64)
    q, out, lse = check(c, 8)
    again, lse2 = torch.empty_like(out), torch.empty_like(lse)
    qm.qs_cache_attention(c.cache, c.seqs, q, 1.3 / math.sqrt(d), again, qm.alloc_cache_attention_workspace(8, 2, d), lse=lse2)
    assert torch.equal(out, again) and torch.equal(lse, lse2)  # the same bits every run


def test_attention_many_rows_split_and_joined():
    check(Paged([4000, 2000], [8, 5], BF16, kv=2, d=128, page=32), 16)
    check(Paged([4000, 2000], [8, 5], E4M3, kv=2, d=256, page=32), 16)
    check(Paged([4000, 2000], [8, 5], E4M3, kv=1, d=64, page=32), 16, F32)


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("group", [1, 4, 16])
def test_what_a_token_does_not_see_does_not_touch_it(kind, group):
    """The last drafted token's own key and value are NaN or infinite: the tokens before it keep their values."""
    c = Paged([60, 16, 49], [4, 4, 4], kind, kv=2, d=64, page=16)
    q, clean, _ = check(c, 2 * group)
    for i, bad in enumerate((float("nan"), float("inf"), float("nan"))):
        p = c.lens[i] - 1
        page, slot = int(c.table[i, p // 16]), p % 16
        c.v[page, slot] = torch.full((2, 64), float("nan"), device="cuda").to(kind)
        c.k[page, slot] = torch.full((2, 64), bad, device="cuda").to(kind)
        if kind is E4M3:
            c.v_scale[page, slot] = float("nan")
    out = torch.empty_like(clean)
    ws = qm.alloc_cache_attention_workspace(2 * group, 2, 64, 4)
    qm.qs_cache_attention(c.cache, c.seqs, q, 1.3 / 8, out, ws, max_new=4)
    for i in range(3):
        assert torch.equal(out[4 * i: 4 * i + 3], clean[4 * i: 4 * i + 3])
        assert torch.isnan(out[4 * i + 3]).all()
    # and behind a window: the first position is seen by the first token alone
    c = Paged([60], [4], kind, kv=2, d=64, page=16)
    q, clean, _ = check(c, 2 * group, window=57)
    c.v[int(c.table[0, 0]), 0] = torch.full((2, 64), float("nan"), device="cuda").to(kind)
    qm.qs_cache_attention(c.cache, c.seqs, q, 1.3 / 8, out[:4], ws, max_new=4, window=57)
    assert torch.isnan(out[0]).all() and torch.equal(out[1:4], clean[1:4])


def test_attention_fewer_tokens_than_a_sequence_has():
    """max_new bounds the tokens attended: the others' rows stay, and the positions are the sequences' own."""
    check(Paged([50, 20], [5, 2], BF16, kv=2, d=64), 8, max_new=3)


def test_attention_positions_outside_the_table():
    """Starts below zero and past the table: what is there is seen, and nothing else."""
    c = Paged([40, 40], [2, 2], BF16, kv=2, d=64, page=16)
    c.starts.copy_(torch.tensor([-2, 1000], dtype=torch.int32))
    q = torch.randn(4, 4, 64, device="cuda").to(BF16)
    out, lse = torch.empty_like(q), torch.empty(4, 4, device="cuda")
    c.k.nan_to_num_(0, 0, 0), c.v.nan_to_num_(0, 0, 0)  # slots behind the 40 are seen now
    qm.qs_cache_attention(c.cache, c.seqs, q, 0.1, out, qm.alloc_cache_attention_workspace(4, 2, 64, 2), max_new=2, lse=lse)
    assert out[:2].count_nonzero() == 0 and (lse[:2] == -math.inf).all()
    k, v = c.rows("k", 1).repeat_interleave(2, 1), c.rows("v", 1).repeat_interleave(2, 1)
    s = torch.einsum("thd,lhd->thl", q[2:].double(), k) * 0.1
    want = torch.einsum("thl,lhd->thd", torch.softmax(s, 2), v)
    assert (out[2:].double() - want).abs().max() <= 2.0 ** -7 * want.abs().max()
    for bad in (-2 ** 31, 2 ** 31 - 1):
        c.starts.fill_(bad)
        qm.qs_cache_attention(c.cache, c.seqs, q, 0.1, out, qm.alloc_cache_attention_workspace(4, 2, 64, 2), max_new=2, lse=lse)
        assert torch.isfinite(out).all()


def test_attention_offsets_that_are_no_offsets():
    """Offsets outside the rows and not ascending are clipped: nothing outside is read or written."""
    c = Paged([40, 40, 40], [1, 1, 1], BF16, kv=2, d=64, page=16)
    c.offsets.copy_(torch.tensor([-5, 2, 1, 900], dtype=torch.int32))
    q = torch.randn(3, 4, 64, device="cuda").to(BF16)
    out = torch.empty_like(q)
    qm.qs_cache_attention(c.cache, c.seqs, q, 0.1, out, qm.alloc_cache_attention_workspace(4, 2, 64, 4), max_new=4)
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_attention_extremes(kind):
    """Scores far apart and far from zero, scales far apart: the formula's values, no overflow."""
    c = Paged([200, 100], [1, 1], kind, kv=2, d=64, page=16)
    q = (50.0 * torch.randn(2, 8, 64, generator=torch.Generator().manual_seed(3))).to(BF16).cuda()
    q[0, 0] = 0.0          # a row of zeros: an even mean
    q[0, 1] *= 2.0 ** -60  # next to it
    q[1, 1] *= 2.0 ** -120
    check(c, 8, q=q)
    check(c, 8, q=q, scale=-0.2)
    check(c, 8, q=q.float() * (1 + 2.0 ** -10), q_type=F32)
    if kind is E4M3:
        c.v_scale *= torch.exp2(torch.randint(-40, 40, c.v_scale.shape, device="cuda").float())
        check(c, 8)
        c.v_scale.fill_(2.0 ** -100)
        check(c, 8)
        c.v_scale.fill_(2.0 ** 90)
        check(c, 8, out_type=F32)
        c.v_scale.zero_()
        check(c, 8)


def test_attention_scores_of_minus_infinity():
    c = Paged([30, 30], [1, 1], BF16, kv=1, d=64, page=16, garbage=False)
    c.k[c.table[0].long()] = -float("inf")
    q = torch.ones(2, 2, 64, device="cuda").to(BF16)
    out, lse = torch.empty_like(q), torch.empty(2, 2, device="cuda")
    qm.qs_cache_attention(c.cache, c.seqs, q, 0.1, out, qm.alloc_cache_attention_workspace(2, 1, 64), lse=lse)
    assert out[0].count_nonzero() == 0 and (lse[0] == -math.inf).all() and torch.isfinite(out[1]).all()


@pytest.mark.parametrize("out", [True, False])
@pytest.mark.parametrize("kind,d,heads", [(BF16, 128, 8), (E4M3, 128, 6), (E4M3, 256, 4), (BF16, 256, 40)])
def test_attention_codes(kind, d, heads, out):
    """The codes are those of the row operators for the exact rows: a code is off by one step at most, where the exact
    value is within the row's tolerance of a border; scales by the tolerance of the block's largest."""
    c = Paged([100, 40, 500], [2, 1, 3], kind, kv=2, d=d, page=16)
    q = torch.randn(c.tokens + 2, heads, d, generator=torch.Generator().manual_seed(5)).to(BF16).cuda()
    o = torch.empty_like(q) if out else None
    codes = torch.zeros(c.tokens + 2, heads * d, dtype=E4M3, device="cuda")
    scale = torch.full((c.tokens + 2, heads * d // 128), 7.0, device="cuda")
    sm = 1.0 / math.sqrt(d)
    qm.qs_cache_attention(c.cache, c.seqs, q, sm, o, qm.alloc_cache_attention_workspace(heads, 2, d, 3), max_new=3, codes=codes, codes_scale=scale)
    exact, _, mass, size, most = attend64(c, q, sm)
    n = c.tokens
    tol, _ = bounds(c, q, F32, True, exact, mass, size, most)
    exact, tol = exact[:n].reshape(n, -1, 128), tol[:n].reshape(n, -1, 128)
    amax = exact.abs().amax(2)
    assert ((scale[:n].double() * 448 - amax).abs() <= tol.amax(2) + 2.0 ** -22 * amax).all()
    got = codes[:n].double().reshape(n, -1, 128) * scale[:n].double()[..., None]
    # a code's rounding: 2^-4 of the value, or half of the smallest step; then what the row and its scale were off by
    room = 2.0 ** -4 * exact.abs() + 2.0 ** -10 * scale[:n].double()[..., None] + 1.07 * tol
    assert ((got - exact).abs() <= room).all()
    assert (scale[n:] == 7.0).all() and codes[n:].float().count_nonzero() == 0
    if out:
        assert ((o[:n].double().reshape(n, -1, 128) - exact).abs() <= U[BF16] * exact.abs() + 1.01 * tol).all()


@pytest.mark.parametrize("q_type,out_type", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
def test_attention_strides_and_alignment(q_type, out_type):
    """Queries and output as slices of wider rows at 16-byte boundaries, other heads left as they are; others are refused."""
    c = Paged([70, 33], [2, 1], BF16, kv=2, d=64, page=16)
    ws = qm.alloc_cache_attention_workspace(8, 2, 64, 2)
    for pad in (0, 8, 24):
        q_all = torch.randn(3, 9, 64 + 8 + pad, device="cuda").to(q_type)
        q = q_all[:, 1:9, pad:pad + 64]
        o_all = torch.full((3, 9, 64 + 8 + pad), 3.0, dtype=out_type, device="cuda")
        o = o_all[:, :8, pad:pad + 64]
        qm.qs_cache_attention(c.cache, c.seqs, q, 0.2, o, ws, max_new=2)
        want = torch.empty(3, 8, 64, dtype=out_type, device="cuda")
        qm.qs_cache_attention(c.cache, c.seqs, q.contiguous(), 0.2, want, ws, max_new=2)
        assert torch.equal(o, want)
        o.fill_(3.0)
        assert (o_all == 3.0).all()
        for odd in (q_all[:, 1:9, pad + 1:pad + 65], torch.randn(3, 8, 65, device="cuda").to(q_type)[:, :, :64]):
            with pytest.raises(qm.QsError):
                qm.qs_cache_attention(c.cache, c.seqs, odd, 0.2, o, ws, max_new=2)
        with pytest.raises(qm.QsError):
            qm.qs_cache_attention(c.cache, c.seqs, q, 0.2, o_all[:, :8, pad + 1:pad + 65], ws, max_new=2)


def test_attention_one_token_each_without_offsets_or_starts():
    c = Paged([1, 1, 1], [1, 1, 1], BF16, kv=2, d=64, page=16)
    q, out, _ = check(c, 4)
    again = torch.empty_like(out)
    qm.qs_cache_attention(c.cache, qm.make_seqs(c.table), q, 1.3 / 8, again, qm.alloc_cache_attention_workspace(4, 2, 64))
    assert torch.equal(out, again)


def test_attention_in_a_graph_follows_lengths_and_tables():
    c = Paged([400, 30], [1, 1], E4M3, kv=2, d=128, page=16)
    q = torch.randn(2, 8, 128, device="cuda").to(BF16)
    out, want, ws = torch.empty_like(q), torch.empty_like(q), qm.alloc_cache_attention_workspace(8, 2, 128)
    qm.qs_cache_attention(c.cache, c.seqs, q, 0.1, out, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qm.qs_cache_attention(c.cache, c.seqs, q, 0.1, out, ws)
    for starts in ([399, 29], [17, 3], [0, 0], [250, 29]):
        c.starts.copy_(torch.tensor(starts, dtype=torch.int32))
        q.copy_(torch.randn(2, 8, 128, device="cuda"))
        graph.replay()
        qm.qs_cache_attention(c.cache, c.seqs, q, 0.1, want, qm.alloc_cache_attention_workspace(8, 2, 128))
        assert torch.equal(out, want)


def test_attention_on_two_streams_at_once():
    """Each call has a workspace of its own."""
    c = Paged([6000, 100], [1, 1], BF16, kv=2, d=128, page=64)
    q = torch.randn(2, 8, 128, device="cuda").to(BF16)
    want = torch.empty_like(q)
    qm.qs_cache_attention(c.cache, c.seqs, q, 0.1, want, qm.alloc_cache_attention_workspace(8, 2, 128))
    torch.cuda.synchronize()
    sides = []
    for _ in range(2):
        stream, out, ws = torch.cuda.Stream(), torch.empty_like(q), qm.alloc_cache_attention_workspace(8, 2, 128)
        stream.wait_stream(torch.cuda.current_stream())
        sides.append((stream, out, ws))
    for _ in range(20):
        for stream, out, ws in sides:
            qm.qs_cache_attention(c.cache, c.seqs, q, 0.1, out, ws, stream=stream.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for _, out, _ in sides)


def test_attention_over_a_cache_past_32_bits():
    """Byte offsets and element offsets past 2^32; keys and values are one buffer, of which few pages are written."""
    pages, page = 70_000, 256
    k = torch.zeros(pages, page, 1, 256, dtype=E4M3, device="cuda")  # 4.6 GB
    scale = torch.ones(pages, page, 1, device="cuda")
    last = torch.randn(2, page, 1, 256, device="cuda")
    k[-1], k[-2] = last[0].to(E4M3), last[1].to(E4M3)
    cache = qm.make_cache(k, k, scale, scale)
    table = torch.tensor([[pages - 2, pages - 1]], dtype=torch.int32, device="cuda")
    seqs = qm.make_seqs(table, torch.tensor([2 * page - 1], dtype=torch.int32, device="cuda"))
    q = torch.randn(1, 4, 256, device="cuda")
    out = torch.empty_like(q)
    qm.qs_cache_attention(cache, seqs, q, 0.1, out, qm.alloc_cache_attention_workspace(4, 1, 256))
    x = torch.cat([k[-2].double(), k[-1].double()])[:, 0]
    want = torch.softmax(q[0].double() @ x.T * 0.1, 1) @ x
    assert (out[0].double() - want).abs().max() <= 1e-4 * want.abs().max()
    back = torch.empty(2 * page, 1, 256, device="cuda"), torch.empty(2 * page, 1, 256, device="cuda")
    qm.qs_cache_read(cache, qm.make_seqs(table, None, torch.tensor([0, 2 * page], dtype=torch.int32, device="cuda")), *back)
    assert torch.equal(back[0][:, 0].double(), x)


# ------------------------------------------------------------------ writing and reading

def written64(rows, kind):
    """(values in 64 bits, scales) that a row's writing should give before its rounding."""
    if kind is not E4M3:
        return rows.double(), None
    scale = rows.double().abs().amax(-1).clamp_min(2.0 ** -100) / 448
    return rows.double() / scale[..., None], scale


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [16, 48, 64, 80, 128, 208, 256])
@pytest.mark.parametrize("rows_type", [BF16, F32], ids=["r16", "r32"])
@pytest.mark.parametrize("kv", [1, 3, 8])
def test_write_then_read(kind, d, rows_type, kv):
    lens, new = [40, 7, 100, 0, 64, 1], [5, 7, 33, 0, 64, 1]
    c = Paged(lens, new, kind, kv=kv, d=d, page=16, garbage=False)
    k, v = (torch.randn(c.tokens + 4, kv, d, device="cuda").to(rows_type) for _ in range(2))
    k[0] = 0.0
    v[1] *= 2.0 ** -110
    before = {n: getattr(c, n).clone() for n in ("k", "v")}
    scales_before = None if kind is not E4M3 else {n: getattr(c, n + "_scale").clone() for n in ("k", "v")}
    qm.qs_cache_write(c.cache, c.seqs, k, v)
    back = {n: torch.full((c.tokens + 4, kv, d), 9.0, dtype=F32, device="cuda") for n in ("k", "v")}
    qm.qs_cache_read(c.cache, c.seqs, back["k"], back["v"])
    for name, rows in (("k", k), ("v", v)):
        touched = torch.zeros(getattr(c, name).shape[:2], dtype=torch.bool, device="cuda")
        value, scale = written64(rows, kind)
        for i in range(len(lens)):
            for j in range(new[i]):
                t, p = int(c.offsets[i]) + j, int(c.starts[i]) + j
                page, slot = int(c.table[i, p // 16]), p % 16
                touched[page, slot] = True
                got = getattr(c, name)[page, slot].double()
                if kind is E4M3:
                    s = getattr(c, name + "_scale")[page, slot].double()
                    assert ((s - scale[t]).abs() <= 2.0 ** -22 * scale[t]).all()
                    # rounded to the nearest code, of a value off by 2^-22: half a step (2^-4, or 2^-10 among the smallest)
                    assert ((got - value[t]).abs() <= (2.0 ** -4 + 2.0 ** -21) * value[t].abs() + 2.0 ** -10).all()
                    stored = got.float() * getattr(c, name + "_scale")[page, slot][:, None]
                else:
                    assert torch.equal(got, rows[t].to(BF16).double())
                    stored = got.float()
                assert torch.equal(back[name][t], stored)
        same = getattr(c, name).view(torch.uint8)[~touched] == before[name].view(torch.uint8)[~touched]
        assert same.all()
        if kind is E4M3:
            assert torch.equal(getattr(c, name + "_scale")[~touched].view(torch.int32), scales_before[name][~touched].view(torch.int32))
        assert (back[name][c.tokens:] == 9.0).all()


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [16, 32, 48, 64, 80, 128, 208, 256])
@pytest.mark.parametrize("rows_type", [BF16, F32], ids=["r16", "r32"])
@pytest.mark.parametrize("kv,aligned", [(1, True), (3, True), (8, True), (5, False)])
def test_many_rows_are_written_and_read_as_few(kind, d, rows_type, kv, aligned):
    """The bytes of one call with 6001 tokens and of calls with 250 are the same, both ways."""
    n, each, page = 6001, 250, 16
    pages = -(-n // page) + 1
    table = torch.randperm(pages, device="cuda", dtype=torch.int32)[None, :-1].contiguous()

    def rows():
        pad = 0 if aligned else 1
        return torch.randn(n, kv, d + pad, device="cuda").to(rows_type)[:, :, pad:]

    k, v = rows(), rows()
    k[0] = 0.0
    k[1, 0, 3], k[1, 0, 4], k[2, 0, d - 1] = float("nan"), 7.0, float("inf")
    v[3] = float("nan")
    v[4] *= 2.0 ** -110
    v[5, kv - 1, d - 1] = -1000.0

    def cache():
        t = [torch.zeros(pages, page, kv, d, device="cuda").to(kind) for _ in range(2)]
        return t + ([torch.zeros(pages, page, kv, device="cuda") for _ in range(2)] if kind is E4M3 else [])

    def seqs(lo, m):
        return qm.make_seqs(table, torch.tensor([lo], dtype=torch.int32, device="cuda"), torch.tensor([0, m], dtype=torch.int32, device="cuda"))

    one, few = cache(), cache()
    qm.qs_cache_write(qm.make_cache(*one), seqs(0, n), k, v)
    for lo in range(0, n, each):
        m = min(each, n - lo)
        qm.qs_cache_write(qm.make_cache(*few), seqs(lo, m), k[lo:lo + m], v[lo:lo + m])
    for x, y in zip(one, few):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    back, pieces = [rows() for _ in range(2)], [rows() for _ in range(2)]
    qm.qs_cache_read(qm.make_cache(*one), seqs(0, n), *back)
    for lo in range(0, n, each):
        m = min(each, n - lo)
        qm.qs_cache_read(qm.make_cache(*one), seqs(lo, m), *(x[lo:lo + m] for x in pieces))
    bits = torch.int16 if rows_type is BF16 else torch.int32
    for x, y in zip(back, pieces):
        assert torch.equal(x.contiguous().view(bits), y.contiguous().view(bits))


def test_codes_are_the_nearest_and_ties_go_to_even():
    c = Paged([300], [300], E4M3, kv=1, d=256, page=32, garbage=False)
    # scale 1: every code's value, the middles between neighbours, and values beside these
    codes = torch.arange(0, 127, dtype=torch.uint8).view(E4M3).float()
    mid = (codes[1:] + codes[:-1]) / 2
    grid = torch.cat([codes, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)])
    k = torch.zeros(300, 1, 256)
    flat = k.view(300, 256)
    for i in range(0, len(grid), 255):
        part = grid[i:i + 255]
        flat[2 * (i // 255), : len(part)], flat[2 * (i // 255) + 1, : len(part)] = part, -part
    flat[:, 255] = 448.0
    qm.qs_cache_write(c.cache, c.seqs, k.cuda(), k.cuda())
    want = k.to(E4M3)
    for p in range(300):
        page, slot = int(c.table[0, p // 32]), p % 32
        assert abs(float(c.k_scale[page, slot, 0]) - 1.0) <= 2.0 ** -23
        assert torch.equal(c.k[page, slot].cpu().view(torch.uint8), want[p].view(torch.uint8))


def test_write_not_finite():
    c = Paged([4], [4], E4M3, kv=1, d=64, page=16, garbage=False)
    k = torch.randn(4, 1, 64, device="cuda")
    k[0, 0, 3] = float("nan")
    k[1, 0, 5] = float("inf")
    k[2, 0, 6] = 3.0e38
    qm.qs_cache_write(c.cache, c.seqs, k, k)
    rows = c.rows("k", 0)[:4, 0]
    assert torch.isnan(rows[0, 3]) and torch.isfinite(rows[0]).sum() == 63 and torch.isnan(rows[1]).all()
    assert (rows[2, 6] - 3.0e38).abs() <= 2.0 ** -4 * 3.0e38 and torch.isfinite(rows[2:]).all()
    b = Paged([4], [4], BF16, kv=1, d=64, page=16, garbage=False)
    qm.qs_cache_write(b.cache, b.seqs, k, k)
    assert torch.equal(b.rows("k", 0)[:4, 0].isfinite(), k[:, 0].to(BF16).isfinite())


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("layout", ["slots", "heads", "both"])
@pytest.mark.parametrize("pad", [0, 1, 5])
def test_rows_strides_and_alignment(kind, layout, pad):
    c = Paged([40, 33], [3, 4], kind, kv=4, d=80, page=8, layout=layout, garbage=False)
    wide = torch.randn(7, 8, 80 + 8 + pad, device="cuda").to(BF16)
    k, v = wide[:, :4, pad:pad + 80], wide[:, 4:, pad:pad + 80]
    qm.qs_cache_write(c.cache, c.seqs, k, v)
    o_all = torch.full((7, 8, 80 + 8 + pad), 3.0, device="cuda")
    ko, vo = o_all[:, :4, pad:pad + 80], o_all[:, 4:, pad:pad + 80]
    qm.qs_cache_read(c.cache, c.seqs, ko, vo)
    for rows, got in ((k, ko), (v, vo)):
        value, scale = written64(rows, kind)
        tol = 2.0 ** -4 * rows.double().abs() + 2.0 ** -10 * scale[..., None] if kind is E4M3 else 0.0
        assert ((got.double() - rows.double()).abs() <= 1.0001 * tol).all() if kind is E4M3 else torch.equal(got.double(), rows.double())
    ko.fill_(3.0), vo.fill_(3.0)
    assert (o_all == 3.0).all()


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_tokens_without_a_place(kind):
    """Pages that are not there, positions outside the table, rows of no sequence: dropped in writing, zeros in reading
    (rows of no sequence stay)."""
    c = Paged([32, 32, 32], [32, 4, 4], kind, kv=2, d=64, page=8, garbage=False)
    c.table[0, 1] = -1
    c.table[0, 2] = c.k.shape[0]
    c.starts.copy_(torch.tensor([0, -2, 30], dtype=torch.int32))
    k = torch.randn(45, 2, 64, device="cuda")
    before = c.k.clone()
    qm.qs_cache_write(c.cache, c.seqs, k, k)
    back = torch.full((45, 2, 64), 9.0, device="cuda"), torch.full((45, 2, 64), 9.0, device="cuda")
    qm.qs_cache_read(c.cache, c.seqs, *back)
    lost = list(range(8, 24)) + [32, 33] + [38, 39]
    kept = [t for t in range(40) if t not in lost]
    for rows in back:
        assert rows[lost].count_nonzero() == 0 and (rows[40:] == 9.0).all()
        assert ((rows[kept] - k[kept]).abs() <= 2.0 ** -4 * k[kept].abs() + 0.01).all()
    changed = (c.k.view(torch.uint8) != before.view(torch.uint8)).flatten(2).any(2).sum()
    assert changed == len(kept)
    empty = qm.make_seqs(torch.empty(0, 4, dtype=torch.int32, device="cuda"), None, torch.zeros(1, dtype=torch.int32, device="cuda"))
    qm.qs_cache_write(c.cache, empty, k, k)  # no sequences: nothing


@pytest.mark.parametrize("n", [31, 32, 33, 1024, 1025, 3000])
def test_many_sequences_are_found(n):
    """A token's sequence among many, empty ones among them."""
    new = [(i * 7) % 3 for i in range(n)]
    lens = [x + i % 5 for i, x in enumerate(new)]
    c = Paged(lens, new, BF16, kv=1, d=16, page=4, garbage=False)
    k, v = (torch.randn(c.tokens, 1, 16, device="cuda").to(BF16) for _ in range(2))
    qm.qs_cache_write(c.cache, c.seqs, k, v)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    qm.qs_cache_read(c.cache, c.seqs, ko, vo)
    assert torch.equal(ko, k) and torch.equal(vo, v)
    seq = torch.repeat_interleave(torch.arange(n), torch.tensor(new)).cuda()
    at = torch.cat([torch.arange(m) + x - m for x, m in zip(lens, new)]).cuda()
    assert torch.equal(c.k[c.table[seq, at // 4].long(), at % 4], k)
    check(c, 2)


def test_a_decode_step_in_a_graph():
    """Write, attend, as a program's step: a captured step is replayed as the sequences grow, and agrees with 64 bits."""
    d, kv, heads, page, n = 128, 2, 8, 16, 3
    pool = 64
    cache_k, cache_v = (torch.zeros(pool, page, kv, d, dtype=E4M3, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(pool, page, kv, device="cuda") for _ in range(2))
    cache = qm.make_cache(cache_k, cache_v, ks, vs)
    table = torch.randperm(pool)[: n * 8].int().view(n, 8).cuda()
    starts = torch.tensor([0, 3, 14], dtype=torch.int32, device="cuda")
    seqs = qm.make_seqs(table, starts)
    k, v, q = (torch.zeros(n, h, d, dtype=BF16, device="cuda") for h in (kv, kv, heads))
    out, ws = torch.empty_like(q), qm.alloc_cache_attention_workspace(heads, kv, d)
    history = [[] for _ in range(n)]

    def step():
        qm.qs_cache_write(cache, seqs, k, v)
        qm.qs_cache_attention(cache, seqs, q, 0.1, out, ws)

    # what the sequences have before the first step
    first = torch.randn(17, kv, d, device="cuda").to(BF16), torch.randn(17, kv, d, device="cuda").to(BF16)
    qm.qs_cache_write(cache, qm.make_seqs(table, None, torch.tensor([0, 0, 3, 17], dtype=torch.int32, device="cuda")), *first)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(20):
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape, device="cuda"))
        graph.replay()
        for i in range(n):
            at = torch.arange(int(starts[i]) + 1, device="cuda")
            where = table[i, at // page].long(), at % page
            kk = (cache_k.view(torch.uint8)[where].view(E4M3).double() * ks[where].double()[..., None]).repeat_interleave(heads // kv, 1)
            vv = (cache_v.view(torch.uint8)[where].view(E4M3).double() * vs[where].double()[..., None]).repeat_interleave(heads // kv, 1)
            w = torch.softmax(torch.einsum("hd,lhd->hl", q[i].double(), kk) * 0.1, 1)
            want, mass = torch.einsum("hl,lhd->hd", w, vv), torch.einsum("hl,lhd->hd", w, vv.abs())
            assert ((out[i].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * mass).all()
            # the newest position is this step's row
            assert ((kk[-1, :: heads // kv] - k[i].double()).abs() <= 2.0 ** -4 * k[i].double().abs() + 0.01).all()
        starts += 1


def test_prompt_prefix_decode_and_projection():
    """As a program uses them: a prompt's rows into the cache, its prefix back as rows, one more token's row, attention over
    all of it to codes, and the 8-bit projection of these."""
    heads, kv, d, page, hidden = 8, 2, 128, 32, 384
    lens, new = [75, 130], [75, 130]
    c = Paged(lens, new, E4M3, kv=kv, d=d, page=page, seed=11, garbage=False)
    wide = torch.randn(c.tokens, heads + 2 * kv, d, device="cuda").to(BF16)  # a projection's output: queries, keys, values
    k, v = wide[:, heads:heads + kv], wide[:, heads + kv:]
    qm.qs_cache_write(c.cache, c.seqs, k, v)
    back = torch.empty(c.tokens, kv, d, device="cuda"), torch.empty(c.tokens, kv, d, device="cuda")
    qm.qs_cache_read(c.cache, c.seqs, *back)
    for rows, got in ((k, back[0]), (v, back[1])):
        scale = rows.double().abs().amax(2) / 448
        assert ((got.double() - rows.double()).abs() <= (2.0 ** -4 + 2.0 ** -20) * rows.double().abs() + 2.0 ** -9 * scale[..., None]).all()
    # the next token overwrites the last prompt position of each sequence
    seqs = qm.make_seqs(c.table, torch.tensor([x - 1 for x in lens], dtype=torch.int32, device="cuda"))
    one = torch.randn(2, heads + 2 * kv, d, device="cuda").to(BF16)
    qm.qs_cache_write(c.cache, seqs, one[:, heads:heads + kv], one[:, heads + kv:])
    c.starts, c.offsets, c.new, c.tokens = torch.tensor([x - 1 for x in lens], dtype=torch.int32).cuda(), torch.tensor([0, 1, 2], dtype=torch.int32).cuda(), [1, 1], 2
    codes, scale = torch.empty(2, heads * d, dtype=E4M3, device="cuda"), torch.empty(2, heads * d // 128, device="cuda")
    qm.qs_cache_attention(c.cache, seqs, one[:, :heads], d ** -0.5, None, qm.alloc_cache_attention_workspace(heads, kv, d), codes=codes, codes_scale=scale)
    exact, _, mass, size, most = attend64(c, one[:, :heads], d ** -0.5)
    tol, _ = bounds(c, one[:, :heads], F32, True, exact, mass, size, most)
    exact, tol = exact.reshape(2, -1), tol.reshape(2, -1)
    w = (0.02 * torch.randn(hidden, heads * d, device="cuda")).to(E4M3)
    ws = torch.rand(hidden // 128, heads * d // 128, device="cuda") + 0.5
    out = torch.empty(2, hidden, device="cuda")
    qm.qs_fp8_matmul(codes, scale, w, ws, out, qm.alloc_fp8_matmul_workspace(2, hidden, heads * d))
    wide_w = w.double() * ws.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    # each code is off by 2^-4 of its value and half of the smallest step, the row by its tolerance; the product's sums by 2^-12 in all
    room = (2.0 ** -4 * exact.abs() + 2.0 ** -9 * scale.double().repeat_interleave(128, 1) + 1.07 * tol + 2.0 ** -12 * exact.abs()) @ wide_w.abs().T
    assert ((out.double() - exact @ wide_w.T).abs() <= room).all()


def test_attention_of_many_tokens_and_heads():
    """The largest counts of rows: 256 heads to a key-value head, 256 new tokens of a sequence."""
    check(Paged([300], [3], BF16, kv=1, d=16, page=16), 256)
    check(Paged([300, 256], [256, 200], E4M3, kv=1, d=64, page=32), 2, max_new=256)


@pytest.mark.parametrize("page", [2, 127, 128, 129, 255, 1023, 65535, 65536])
def test_attention_more_page_sizes(page):
    check(Paged([400, 3], [2, 1], BF16, kv=1, d=16, page=page, spare_pages=1), 2)


def test_bindings_refusals():
    c = Paged([20], [1], BF16, kv=2, d=64)
    q = torch.zeros(1, 4, 64, dtype=BF16, device="cuda")
    ws = qm.alloc_cache_attention_workspace(4, 2, 64)
    ok = dict(cache=c.cache, seqs=c.seqs, q=q, scale=0.1, out=torch.empty_like(q), workspace=ws)
    qm.qs_cache_attention(**ok)
    for bad in (dict(q=q.cpu()), dict(q=q[:, :, :32]), dict(q=q[0]), dict(q=q.half()), dict(out=torch.empty(2, 4, 64, dtype=BF16, device="cuda")),
                dict(lse=torch.empty(1, 4, dtype=BF16, device="cuda")), dict(lse=torch.empty(4, 1, device="cuda")), dict(workspace=ws.cpu()),
                dict(codes=torch.empty(1, 256, dtype=E4M3, device="cuda")), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            qm.qs_cache_attention(**{**ok, **bad})
    for bad in (dict(workspace=ws[:1024]), dict(out=None), dict(max_new=0), dict(window=-1), dict(scale=float("nan")), dict(max_new=9),
                dict(codes=torch.empty(1, 256, dtype=E4M3, device="cuda"), codes_scale=torch.empty(1, 2, device="cuda"))):
        with pytest.raises(qm.QsError):
            qm.qs_cache_attention(**{**ok, **bad})
    kv = torch.zeros(1, 2, 64, dtype=BF16, device="cuda")
    for bad in (kv.cpu(), kv[:, :1], kv[0], kv.half()):
        with pytest.raises(ValueError):
            qm.qs_cache_write(c.cache, c.seqs, bad, kv)
        with pytest.raises(ValueError):
            qm.qs_cache_read(c.cache, c.seqs, kv, bad)
    with pytest.raises(ValueError, match="no offsets"):
        qm.qs_cache_write(c.cache, qm.make_seqs(c.table, c.starts), kv.expand(2, 2, 64).contiguous(), kv)
    with pytest.raises(qm.QsError):  # one row for all heads
        qm.qs_cache_read(c.cache, c.seqs, kv[:, :1].expand(1, 2, 64), kv)
    one = c.k[:, :, :1].expand_as(c.k)
    qm.qs_cache_read(qm.make_cache(one, one), c.seqs, kv, kv.clone())
    with pytest.raises(qm.QsError):
        qm.qs_cache_write(qm.make_cache(one, one), c.seqs, kv, kv)
    k8, s8 = torch.zeros(2, 16, 2, 64, dtype=E4M3, device="cuda"), torch.zeros(2, 16, 2, device="cuda")
    for bad in ((c.k, c.v[:1]), (c.k, c.v.float()), (c.k, c.v.cpu()), (c.k, c.v, s8, s8), (k8, k8), (k8, k8, s8, None), (k8, k8, s8, s8[:1]), (k8, k8, s8, s8.double()),
                (k8.half(), k8.half()), (c.k, c.v.transpose(1, 2).contiguous().transpose(1, 2)), (k8, k8, s8, s8.transpose(1, 2).contiguous().transpose(1, 2)),
                (c.k.transpose(2, 3), c.v.transpose(2, 3))):
        with pytest.raises(ValueError):
            qm.make_cache(*bad)
    for bad in ((c.table.long(),), (c.table, c.starts.long()), (c.table, c.starts[:0]), (c.table, c.starts, c.offsets[:1]), (c.table, c.starts.cpu()), (c.table.t().contiguous().t(),) if c.table.shape[0] > 1 else (c.table[0],)):
        with pytest.raises(ValueError):
            qm.make_seqs(*bad)
