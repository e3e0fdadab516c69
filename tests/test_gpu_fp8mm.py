"""The e4m3 product with block scales on the GPU against the sum in 64 bits.

An output is a sum of n products with magnitudes |a||w|.  Products of e4m3 codes are exact in fp32; the sums inside a
block take 128 additions, the sum over blocks ceil(K / 128), the scales two roundings a block; with 2^-23 for an addition
(the tensor cores may cut where fp32 rounds) the error is at most (128 + blocks + 4) 2^-23 sum(|a||w|), and storing adds half
a step of the output's type.
"""
import pytest
import torch

from bit_quantized_moe_router_gb300 import qs_moe as qm

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def operand(shape, scale_shape, g, pad=0):
    """Codes (rows 16 bytes apart at least, `pad` bytes more) and scales over several orders of magnitude."""
    k = shape[-1]
    buf = torch.randn(*shape[:-1], -(-k // 16) * 16 + pad, generator=g).mul_(8).to(F8).cuda()
    return buf[..., :k], torch.exp2(torch.randint(-6, 3, scale_shape, generator=g).float() + torch.rand(scale_shape, generator=g)).cuda()


def blocks(n):
    return (n + 127) // 128


def values(q, scale, weights):
    v = q.cpu().float().double()
    s = scale.cpu().double().repeat_interleave(128, -1)[..., : v.shape[-1]]
    if weights:
        s = s.repeat_interleave(128, -2)[..., : v.shape[-2], :]
    return v * s


def check(out, a, w, kind):
    want, size = a @ w.T, a.abs() @ w.abs().T
    got = out.cpu().double()
    assert torch.all((got - want).abs() <= (128 + blocks(a.shape[1]) + 4) * 2.0 ** -23 * size + HALF[kind] * want.abs())


@pytest.mark.parametrize("rows,cols,inner,kind", [
    (1, 1, 1, torch.float32), (1, 16, 16, torch.bfloat16), (1, 4096, 2048, torch.bfloat16), (2, 100, 129, torch.float32),
    (15, 256, 128, torch.bfloat16), (16, 17, 384, torch.float32), (17, 1000, 1000, torch.bfloat16), (64, 2049, 250, torch.float32),
    (65, 128, 2048, torch.float32), (127, 300, 72, torch.bfloat16), (128, 256, 4096, torch.float32), (129, 257, 640, torch.bfloat16),
    (333, 1000, 1200, torch.float32), (1024, 2048, 512, torch.bfloat16), (2500, 4104, 384, torch.bfloat16), (5000, 130, 90, torch.float32)])
def test_matmul(rows, cols, inner, kind):
    g = torch.Generator().manual_seed(rows + cols + inner)
    a, sa = operand((rows, inner), (rows, blocks(inner)), g)
    w, sw = operand((cols, inner), (blocks(cols), blocks(inner)), g)
    out = torch.full((rows, cols), float("nan"), dtype=kind, device="cuda")
    ws = qm.alloc_fp8_matmul_workspace(rows, cols, inner)
    qm.qs_fp8_matmul(a, sa, w, sw, out, ws)
    assert qm.qs_read_device_status(ws) == qm.QS_OK
    check(out, values(a, sa, False), values(w, sw, True), kind)


@pytest.mark.parametrize("rows", [3, 200])
def test_matmul_strides(rows):
    g = torch.Generator().manual_seed(5)
    a, sa = operand((rows, 300), (rows, 8), g, pad=64)
    sa = sa[:, :3]
    w, sw = operand((70, 300), (1, 3), g, pad=16)
    wide = torch.full((rows, 99), 7.0, device="cuda")
    out = wide[:, 1:71]  # rows that start off every boundary
    ws = qm.alloc_fp8_matmul_workspace(rows, 70, 300)
    qm.qs_fp8_matmul(a, sa, w, sw, out, ws)
    check(out, values(a, sa, False), values(w, sw, True), torch.float32)
    assert torch.all(wide[:, 0] == 7) and torch.all(wide[:, 71:] == 7)


COUNTS = {
    "one row each": [1] * 12, "empty and full": [0, 0, 5, 0, 128, 1, 0, 129, 64, 65, 0, 300, 0], "all in one": [0, 0, 700, 0],
    "none": [0, 0, 0], "many": [(7 * e) % 23 for e in range(256)], "last alone": [0] * 31 + [17], "sixty-four": [64] * 9, "one expert": [40], "seven": [2, 0, 5, 0], "fifty-five": [20, 1, 0, 34],
    "few each": [(5 * e) % 7 for e in range(128)], "few but one": [1] * 60 + [100] + [0] * 67}


@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("cols,inner,kind", [(256, 256, torch.bfloat16), (100, 200, torch.float32), (1024, 512, torch.bfloat16)])
def test_grouped(name, cols, inner, kind):
    counts = COUNTS[name]
    experts, total = len(counts), sum(counts)
    rows = total + 9  # rows after the last group are left alone
    g = torch.Generator().manual_seed(total + cols)
    a, sa = operand((rows, inner), (rows, blocks(inner)), g)
    w, sw = operand((experts, cols, inner), (experts, blocks(cols), blocks(inner)), g)
    off = torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    out = torch.full((rows, cols), 5.0, dtype=kind, device="cuda")
    ws = qm.alloc_fp8_matmul_workspace(rows, cols, inner, experts)
    qm.qs_fp8_matmul(a, sa, w, sw, out, ws, off)
    assert qm.qs_read_device_status(ws) == qm.QS_OK
    av, wv = values(a, sa, False), values(w, sw, True)
    at = 0
    for e, c in enumerate(counts):
        if c:
            check(out[at:at + c], av[at:at + c], wv[e], kind)
        at += c
    assert torch.all(out[total:] == 5.0)


def test_grouped_offsets_are_clipped():
    g = torch.Generator().manual_seed(3)
    a, sa = operand((20, 128), (20, 1), g)
    w, sw = operand((3, 64, 128), (3, 1, 1), g)
    ws = qm.alloc_fp8_matmul_workspace(20, 64, 128, 3)
    av, wv = values(a, sa, False), values(w, sw, True)
    for off in ([-5, 10, 15, 1000], [4, 4, 2, 2 ** 31 - 1], [30, 40, 50, 60]):
        out = torch.full((20, 64), 5.0, device="cuda")
        qm.qs_fp8_matmul(a, sa, w, sw, out, ws, torch.tensor(off, dtype=torch.int32, device="cuda"))
        cut = [min(max(o, 0), 20) for o in off]
        untouched = torch.ones(20, dtype=torch.bool)
        for e in range(3):
            if cut[e + 1] > cut[e]:
                check(out[cut[e]:cut[e + 1]], av[cut[e]:cut[e + 1]], wv[e], torch.float32)
                untouched[cut[e]:cut[e + 1]] = False
        assert torch.all(out.cpu()[untouched] == 5.0)
    assert qm.qs_read_device_status(ws) == qm.QS_OK


def test_nan_and_infinite_scales_stay_in_their_rows():
    g = torch.Generator().manual_seed(9)
    a, sa = operand((40, 256), (40, 2), g)
    w, sw = operand((96, 256), (1, 2), g)
    ref = torch.empty(40, 96, device="cuda")
    ws = qm.alloc_fp8_matmul_workspace(40, 96, 256)
    qm.qs_fp8_matmul(a, sa, w, sw, ref, ws)
    a.view(torch.uint8)[3, 17] = 0x7F  # NaN code
    sa[5, 1] = float("inf")
    w.view(torch.uint8)[11, 200] = 0xFF
    out = torch.empty_like(ref)
    qm.qs_fp8_matmul(a, sa, w, sw, out, ws)
    assert torch.all(torch.isnan(out[3])) and torch.all(torch.isnan(out[:, 11])) and not torch.any(torch.isfinite(out[5]))
    rows = [r for r in range(40) if r not in (3, 5)]
    cols = [c for c in range(96) if c != 11]
    assert torch.equal(out[rows][:, cols], ref[rows][:, cols])


def test_same_bits_alone_and_in_a_batch_and_in_a_graph():
    """A row's result does not depend on the rows beside it, nor on the run."""
    g = torch.Generator().manual_seed(11)
    a, sa = operand((150, 1024), (150, 8), g)
    w, sw = operand((512, 1024), (4, 8), g)
    ws = qm.alloc_fp8_matmul_workspace(150, 512, 1024)
    full, one = torch.empty(150, 512, device="cuda"), torch.empty(1, 512, device="cuda")
    qm.qs_fp8_matmul(a, sa, w, sw, full, ws)
    for r in (0, 77, 149):
        qm.qs_fp8_matmul(a[r:r + 1], sa[r:r + 1], w, sw, one, ws)
        assert torch.equal(one[0], full[r])
    graph, again = torch.cuda.CUDAGraph(), torch.empty_like(full)
    with torch.cuda.graph(graph):
        qm.qs_fp8_matmul(a, sa, w, sw, again, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, full)


@pytest.mark.parametrize("rows,cols,inner,kind", [
    (2304, 2560, 128, torch.float32), (2500, 2600, 700, torch.bfloat16), (5121, 1030, 200, torch.float32), (8192, 1024, 2048, torch.bfloat16),
    (300, 9984, 130, torch.float32)])
def test_matmul_with_tiles_of_two_ctas(rows, cols, inner, kind):
    test_matmul(rows, cols, inner, kind)


@pytest.mark.parametrize("counts", [[300, 0, 129, 700, 1, 256, 2, 512], [2000] + [0] * 4 + [1] * 3, [513] * 8])
@pytest.mark.parametrize("cols,inner,kind", [(2560, 384, torch.bfloat16), (2100, 100, torch.float32)])
def test_grouped_with_tiles_of_two_ctas(counts, cols, inner, kind):
    COUNTS["wide"] = counts
    try:
        test_grouped("wide", cols, inner, kind)
    finally:
        del COUNTS["wide"]


@pytest.mark.parametrize("rows,cols,inner", [(128, 8192, 4096), (300, 4104, 4096), (512, 8192, 1024), (1, 8192, 4096), (40, 2048, 4096), (100, 1000, 2000)])
def test_same_bits_every_time(rows, cols, inner):
    """Copies that land in another order, as they do when memory is busy, change nothing."""
    g = torch.Generator().manual_seed(rows)
    a, sa = operand((rows, inner), (rows, blocks(inner)), g)
    w, sw = operand((cols, inner), (blocks(cols), blocks(inner)), g)
    ws = qm.alloc_fp8_matmul_workspace(rows, cols, inner)
    first = torch.empty(rows, cols, device="cuda")
    qm.qs_fp8_matmul(a, sa, w, sw, first, ws)
    check(first, values(a, sa, False), values(w, sw, True), torch.float32)
    src = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    dst, side, out = torch.empty_like(src), torch.cuda.Stream(), torch.empty_like(first)
    for _ in range(20):
        with torch.cuda.stream(side):
            dst.copy_(src)
        out.fill_(7)
        qm.qs_fp8_matmul(a, sa, w, sw, out, ws)
        assert torch.equal(out, first)
    assert qm.qs_read_device_status(ws) == qm.QS_OK


@pytest.mark.parametrize("rows,cols,kind", [(3, 70, torch.float32), (200, 70, torch.float32), (200, 131, torch.bfloat16), (2600, 2500, torch.bfloat16), (129, 257, torch.float32)])
def test_columns_past_the_last_are_left_alone(rows, cols, kind):
    """Aligned rows wider than the result: copies out are cut at its edge."""
    g = torch.Generator().manual_seed(rows)
    a, sa = operand((rows, 256), (rows, 2), g)
    w, sw = operand((cols, 256), (blocks(cols), 2), g)
    wide = torch.full((rows + 1, (cols + 63) // 16 * 16), 7.0, dtype=kind, device="cuda")
    out = wide[:rows, :cols]
    qm.qs_fp8_matmul(a, sa, w, sw, out, qm.alloc_fp8_matmul_workspace(rows, cols, 256))
    check(out, values(a, sa, False), values(w, sw, True), kind)
    assert torch.all(wide[:, cols:] == 7) and torch.all(wide[rows] == 7)


def test_experts_and_scales_inside_wider_buffers():
    g = torch.Generator().manual_seed(21)
    counts, cols, inner = [5, 0, 70, 33], 200, 300
    rows = sum(counts)
    a, sa = operand((rows, inner), (rows, 5), g, pad=32)
    big, sw = operand((4, cols + 9, inner), (4, blocks(cols), blocks(inner)), g, pad=48)
    w = big[:, :cols]  # nine rows between experts that are another's
    off = torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    out = torch.empty(rows, cols, device="cuda")
    qm.qs_fp8_matmul(a, sa[:, 1:4], w, sw, out, qm.alloc_fp8_matmul_workspace(rows, cols, inner, 4), off)
    av, wv, at = values(a, sa[:, 1:4], False), values(w, sw, True), 0
    for e, c in enumerate(counts):
        if c:
            check(out[at:at + c], av[at:at + c], wv[e], torch.float32)
        at += c


def test_first_call_of_a_process_may_be_captured():
    import subprocess
    import sys
    code = """
import torch
from bit_quantized_moe_router_gb300 import qs_moe as qm
F8 = torch.float8_e4m3fn
a, w = torch.ones(5, 256, device="cuda").to(F8), torch.ones(64, 256, device="cuda").to(F8)
sa, sw, out = torch.ones(5, 2, device="cuda"), torch.ones(1, 2, device="cuda"), torch.zeros(5, 64, device="cuda")
ws = qm.alloc_fp8_matmul_workspace(5, 64, 256)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    qm.qs_fp8_matmul(a, sa, w, sw, out, ws)
g.replay()
torch.cuda.synchronize()
assert torch.all(out == 256), out
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("rows,cols,inner", [(13, 300, 384), (30, 130, 200), (60, 256, 640)])
def test_groups_of_few_rows_have_the_bits_that_they_have_in_a_longer_call(rows, cols, inner):
    g = torch.Generator().manual_seed(rows)
    a, sa = operand((300, inner), (300, blocks(inner)), g)
    w, sw = operand((5, cols, inner), (5, blocks(cols), blocks(inner)), g)
    off = torch.tensor([0, 0, 3, 4, rows - 2, rows], dtype=torch.int32, device="cuda")
    ws = qm.alloc_fp8_matmul_workspace(300, cols, inner, 5)
    out = [torch.zeros(n, cols, device="cuda") for n in (300, rows, rows)]
    qm.qs_fp8_matmul(a, sa, w, sw, out[0], ws, off)
    qm.qs_fp8_matmul(a[:rows], sa[:rows], w, sw, out[1], ws, off)
    assert torch.equal(out[1], out[0][:rows]) and out[1].abs().amax(1).min() > 0
    # a row of NaN codes, and an expert with a NaN scale, stay where they are
    a.view(torch.uint8)[3] = 0x7F
    sw[4] = float("nan")
    qm.qs_fp8_matmul(a[:rows], sa[:rows], w, sw, out[2], ws, off)
    keep = [r for r in range(rows - 2) if r != 3]
    assert torch.equal(out[2][keep], out[1][keep])
    assert torch.isnan(out[2][3]).all() and torch.isnan(out[2][rows - 2:]).all()


@pytest.mark.parametrize("rows,cols,inner,kind", [(1, 20000, 256, torch.bfloat16), (7, 19999, 200, torch.float32), (16, 20001, 640, torch.bfloat16)])
def test_few_rows_by_many_columns(rows, cols, inner, kind):
    test_matmul(rows, cols, inner, kind)
    g = torch.Generator().manual_seed(rows)
    a, sa = operand((100, inner), (100, blocks(inner)), g)
    w, sw = operand((cols, inner), (blocks(cols), blocks(inner)), g)
    out = [torch.zeros(n, cols, dtype=kind, device="cuda") for n in (100, rows)]
    ws = qm.alloc_fp8_matmul_workspace(100, cols, inner)
    qm.qs_fp8_matmul(a, sa, w, sw, out[0], ws)
    qm.qs_fp8_matmul(a[:rows], sa[:rows], w, sw, out[1], ws)
    assert torch.equal(out[0][:rows], out[1])


@pytest.mark.parametrize("rows,cols,inner,kind", [
    (1, 4096, 2048, torch.bfloat16), (9, 63, 129, torch.float32), (33, 65, 1000, torch.bfloat16), (100, 1000, 640, torch.float32),
    (16, 9728, 130, torch.bfloat16), (17, 9728, 130, torch.bfloat16), (64, 4864, 200, torch.float32), (65, 3201, 1100, torch.bfloat16), (500, 511, 640, torch.bfloat16), (16, 9729, 256, torch.float32), (2000, 64, 300, torch.float32)])
def test_tiles_of_few_rows(rows, cols, inner, kind):
    test_matmul(rows, cols, inner, kind)


@pytest.mark.parametrize("cols", [100, 512])
def test_one_group_of_few_tiles(cols):
    test_grouped("seven", cols, 520, torch.bfloat16)
    test_grouped("one expert", cols, 1024, torch.float32)


@pytest.mark.parametrize("cols,inner", [(4096, 512), (900, 1100)])
def test_a_row_has_the_same_bits_in_calls_of_any_length(cols, inner):
    g = torch.Generator().manual_seed(cols)
    a, sa = operand((2600, inner), (2600, blocks(inner)), g)
    w, sw = operand((cols, inner), (blocks(cols), blocks(inner)), g)
    ws = qm.alloc_fp8_matmul_workspace(2600, cols, inner)
    full = torch.empty(2600, cols, device="cuda")
    qm.qs_fp8_matmul(a, sa, w, sw, full, ws)
    for rows in (1, 16, 17, 33, 64, 65, 100, 129, 333, 1000):
        out = torch.empty(rows, cols, device="cuda")
        qm.qs_fp8_matmul(a[:rows], sa[:rows], w, sw, out, ws)
        assert torch.equal(out, full[:rows])


@pytest.mark.parametrize("counts", [[0] * 5 + [990] + [1] * 24 + [0] * 226, [700, 0, 250] + [0] * 253])
def test_long_groups_in_tiles_of_few_rows(counts):
    """Four rows an expert on average, nearly all of them one expert's."""
    COUNTS["long"] = counts
    try:
        test_grouped("long", 200, 384, torch.bfloat16)
    finally:
        del COUNTS["long"]
