"""Attention over the paged cache at the ends of its ranges."""
import pytest
import torch

from bit_quantized_moe_router_gb300 import qs_moe as qm
from test_gpu_cache import BF16, E4M3, Paged

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


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
