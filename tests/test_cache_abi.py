"""Refusals of the paged cache's operators: every bad argument is answered on the host, before a GPU is touched."""
import pytest
import torch

from bit_quantized_moe_router_gb300 import qs_moe as qm

FAKE = 1 << 40   # an address that is never read: the checks come first
INV, WS = qm.QS_ERR_INVALID, qm.QS_ERR_WORKSPACE
F32, BF16, E4M3 = qm.QS_F32, qm.QS_BF16, qm.QS_E4M3

# 10 pages of 16 slots, 4 heads of 128 columns; two sequences of five pages
CACHE = dict(ck=FAKE, cv=FAKE, cks=FAKE, cvs=FAKE, page=16 * 512, slot=512, head=128, spage=64, sslot=4, shead=1, dtype=E4M3, n_pages=10, page_size=16, kv=4, d=128)
SEQS = dict(table=FAKE, table_stride=5, starts=FAKE, offsets=FAKE, n_seqs=2, n_seq_pages=5)


def heads(name, n_heads=4, dtype=BF16):
    return {name: FAKE, name + "_token": n_heads * 128, name + "_head": 128, name + "_dtype": dtype}


ROWS = {**CACHE, **SEQS, **heads("k"), **heads("v"), "n": 3}
ATTN = {**CACHE, **SEQS, **heads("q", 8), **heads("out", 8), "codes": FAKE, "codes_stride": 1024, "codes_scale": FAKE, "codes_scale_stride": 8,
        "lse": FAKE, "ws": FAKE, "bytes": 1 << 40, "scale": 0.1, "n": 3, "h": 8, "max_new": 2, "window": 0}


def call(name, base, over):
    """The entry point on the packed struct of base's fields with some of them changed."""
    assert set(over) <= set(base)
    return getattr(qm.load(), name)(qm.ARGS[name].pack(*{**base, **over}.values()), None)


BAD_CACHE = [
    dict(ck=0), dict(cv=0), dict(cks=0), dict(cvs=0), dict(ck=FAKE + 8), dict(cv=FAKE + 1), dict(cks=FAKE + 2), dict(dtype=F32), dict(dtype=9),
    dict(page=-16), dict(slot=8), dict(head=100), dict(page=1 << 41), dict(spage=-1), dict(n_pages=-1), dict(page_size=0), dict(kv=0), dict(kv=257),
    dict(d=0), dict(d=120), dict(d=272), dict(page_size=(1 << 30) + 1)]
BAD_SEQS = [
    dict(table=0), dict(table=FAKE + 2), dict(starts=FAKE + 1), dict(offsets=FAKE + 2), dict(table_stride=4), dict(n_seqs=-1), dict(n_seqs=(1 << 16) + 1),
    dict(n_seq_pages=-1), dict(n_seq_pages=1 << 27, table_stride=1 << 27), dict(offsets=0), dict(n=-1), dict(n=(1 << 24) + 1)]


@pytest.mark.parametrize("name", ["qs_cache_write", "qs_cache_read"])
@pytest.mark.parametrize("over", BAD_CACHE + BAD_SEQS + [
    dict(k=0), dict(v=0), dict(k=FAKE + 1), dict(k_dtype=E4M3), dict(v_dtype=5), dict(v_dtype=F32), dict(k_token=-1), dict(v_head=-128), dict(k_token=1 << 41)], ids=str)
def test_rows_refusals(name, over):
    assert call(name, ROWS, over) == INV
    assert getattr(qm.load(), name)(None, None) == INV


# places of the cache that coincide: fine to read, not to write
@pytest.mark.parametrize("over", [dict(head=0), dict(slot=0), dict(page=0), dict(head=112), dict(page=16 * 512 - 16), dict(shead=0), dict(sslot=3), dict(spage=60)], ids=str)
def test_write_refuses_places_that_coincide(over):
    assert call("qs_cache_write", ROWS, over) == INV


# extents past 2^60 elements, whose product of stride and size passes 64 bits (2^64 exactly, and beside it)
@pytest.mark.parametrize("over", [dict(page=1 << 40, n_pages=(1 << 24) + 1), dict(page=1 << 40, n_pages=1 << 24), dict(page=1 << 40, n_pages=(1 << 31) - 1),
                                  dict(page=3 << 38, n_pages=(1 << 24) + 1), dict(spage=1 << 40, n_pages=(1 << 24) + 1)], ids=str)
def test_write_refuses_extents_past_64_bits(over):
    assert call("qs_cache_write", ROWS, {**over, "n": 0}) == INV
    assert call("qs_cache_write", ROWS, {**over, "n_pages": 1 << 20, "n": 0}) == qm.QS_OK  # 2^60


def test_read_refuses_rows_whose_extents_pass_64_bits():
    assert call("qs_cache_read", ROWS, dict(k_token=1 << 40, n=1 << 24)) == INV


# rows that coincide: fine to write from, not to read into
@pytest.mark.parametrize("over", [dict(k_head=0), dict(v_token=0), dict(v_head=64), dict(k_token=500)], ids=str)
def test_read_refuses_rows_that_coincide(over):
    assert call("qs_cache_read", ROWS, over) == INV


@pytest.mark.parametrize("over,code", [(o, INV) for o in BAD_CACHE + BAD_SEQS] + [
    (dict(q=0), INV), (dict(q=FAKE + 1), INV), (dict(q=FAKE + 2), INV), (dict(q_head=132), INV), (dict(q_token=1028), INV), (dict(out=FAKE + 8), INV), (dict(out_head=132, out_token=1100), INV), (dict(q_dtype=E4M3), INV), (dict(out=0, codes=0, codes_scale=0), INV), (dict(out=FAKE + 1), INV), (dict(out_dtype=E4M3), INV),
    (dict(out_head=0), INV), (dict(out_token=1000), INV), (dict(codes=0), INV), (dict(codes_scale=0), INV), (dict(codes=FAKE + 8), INV),
    (dict(codes_stride=1032), INV), (dict(codes_stride=1008), INV), (dict(codes_scale_stride=7), INV), (dict(codes_scale=FAKE + 1), INV),
    (dict(d=64, head=64, slot=256, page=4096), INV),                     # codes of rows whose heads share a scale
    (dict(lse=FAKE + 2), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(scale=2e38), INV), (dict(window=-1), INV), (dict(max_new=0), INV),
    (dict(max_new=257), INV), (dict(h=9), INV), (dict(h=0), INV), (dict(h=2), INV), (dict(ws=0), WS), (dict(ws=FAKE + 16), WS), (dict(bytes=1000), WS)], ids=str)
def test_attention_refusals(over, code):
    assert call("qs_cache_attention", ATTN, over) == code
    assert qm.load().qs_cache_attention(None, None) == INV


def test_attention_refuses_places_past_32_bits():
    """Places are counted in the largest power of two that divides the pages' and slots' strides: 2^31 of them at most."""
    odd = dict(page=16 * (1 << 21) + 16, n_pages=1 << 11)      # 16 bytes: 34 GB of them are more
    assert call("qs_cache_attention", ATTN, odd) == qm.QS_ERR_UNSUPPORTED
    assert call("qs_cache_attention", ATTN, dict(page=1 << 25, n_pages=1 << 11, n=0)) == qm.QS_OK


def test_attention_refuses_more_tiles_than_a_cta_counts():
    """2e10 tiles of 16 positions and 8 rows: a CTA's share of the places that these take is a 32-bit number."""
    room = dict(n=0, n_seqs=1 << 16, n_seq_pages=1 << 13, table_stride=1 << 13)   # 2^16 sequences of 2^17 positions: 3.2e9
    assert call("qs_cache_attention", ATTN, room) == qm.QS_OK
    for more in (dict(n_seq_pages=1 << 16, table_stride=1 << 16), dict(n_seq_pages=1 << 26, table_stride=1 << 26), dict(max_new=256, h=256)):
        assert call("qs_cache_attention", ATTN, {**room, **more}) == qm.QS_ERR_UNSUPPORTED


def test_calls_without_tokens_launch_nothing():
    for name, base in (("qs_cache_write", ROWS), ("qs_cache_read", ROWS), ("qs_cache_attention", ATTN)):
        assert call(name, base, dict(n=0)) == qm.QS_OK
        assert call(name, base, dict(n=0, offsets=0, n_seqs=0, table=0, starts=0)) == qm.QS_OK


def test_attention_workspace_sizes():
    size = qm.load().qs_cache_attention_workspace_bytes
    assert size(16, 2, 256, 1) > 256 and size(16, 2, 256, 8) > size(16, 2, 256, 2) > size(16, 2, 256, 1) > size(16, 2, 64, 1)
    for bad in [(0, 1, 128, 1), (8, 0, 128, 1), (9, 2, 128, 1), (8, 2, 100, 1), (8, 2, 272, 1), (8, 2, 128, 0), (8, 2, 128, 257), (2, 4, 128, 1), (257, 1, 128, 1)]:
        assert size(*bad) == 0
    for heads, kv, d in [(16, 2, 256), (32, 8, 128), (6, 2, 80), (5, 5, 16)]:  # one made for more new tokens does for fewer
        assert [size(heads, kv, d, n) for n in range(1, 20)] == sorted(size(heads, kv, d, n) for n in range(1, 20))


def test_bindings_refusals_without_a_gpu():
    k = torch.zeros(2, 16, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device memory"):
        qm.make_cache(k, k)
    with pytest.raises(ValueError, match="4|dimensions"):
        qm.make_cache(k[0], k[0])
    with pytest.raises(ValueError, match="device memory"):
        qm.make_seqs(torch.zeros(2, 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="matrix"):
        qm.make_seqs(torch.zeros(2, dtype=torch.int32))
    with pytest.raises(qm.QsError):
        qm.alloc_cache_attention_workspace(8, 3, 128)
