"""Refusals of the row operators: every bad argument is answered on the host, before a GPU is touched."""
import pytest
import torch

from bit_quantized_moe_router_gb300 import qs_moe as qm

FAKE = 1 << 40   # an address that is never read: the checks come first
INV, WS = qm.QS_ERR_INVALID, qm.QS_ERR_WORKSPACE
F32, BF16, E4M3 = qm.QS_F32, qm.QS_BF16, qm.QS_E4M3
BIG = 1 << 40


def change(base, **over):
    d = dict(base)
    assert set(over) <= set(d)
    d.update(over)
    return list(d.values())


NORM = dict(x=FAKE, x_stride=256, x_dtype=BF16, r=FAKE, r_stride=256, r_dtype=BF16, w=FAKE, eps=1e-6, n=4, h=256, s=FAKE,
            s_stride=256, s_dtype=BF16, y=FAKE, y_stride=256, y_dtype=BF16, q=FAKE, q_stride=256, qs=FAKE, qs_stride=2, st=None)


@pytest.mark.parametrize("over", [
    dict(x=None), dict(x_dtype=E4M3), dict(x_dtype=7), dict(x_stride=255), dict(x=FAKE + 1), dict(w=None), dict(w=FAKE + 2),
    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(n=-1), dict(h=0), dict(h=16385), dict(r_stride=0),
    dict(r_dtype=-1), dict(s_stride=10), dict(y_dtype=E4M3), dict(y=FAKE + 1), dict(q_stride=255), dict(qs=None), dict(q=None),
    dict(qs_stride=1), dict(qs=FAKE + 2), dict(s=None, y=None, q=None, qs=None)], ids=str)
def test_norm_refusals(over):
    assert qm.load().qs_rmsnorm_residual(*change(NORM, **over)) == INV


BWD = dict(s=FAKE, s_stride=256, s_dtype=F32, w=FAKE, eps=1e-6, dy=FAKE, dy_stride=256, dy_dtype=F32, ds=FAKE, ds_stride=256,
           ds_dtype=F32, n=4, h=256, dx=FAKE, dx_stride=256, dx_dtype=F32, dw=FAKE, ws=FAKE, bytes=BIG, st=None)


@pytest.mark.parametrize("over,code", [
    (dict(s=None), INV), (dict(dy=None), INV), (dict(dx=None), INV), (dict(w=None), INV), (dict(h=20000), INV),
    (dict(n=-2), INV), (dict(dy_stride=1), INV), (dict(ds_dtype=E4M3), INV), (dict(dx=FAKE + 2), INV), (dict(dw=FAKE + 1), INV),
    (dict(ws=None), WS), (dict(ws=FAKE + 8), WS), (dict(bytes=1000), WS)], ids=str)
def test_norm_backward_refusals(over, code):
    assert qm.load().qs_rmsnorm_residual_backward(*change(BWD, **over)) == code


SILU = dict(g=FAKE, g_stride=512, g_dtype=BF16, n=4, nd=None, f=256, q=FAKE, q_stride=256, qs=FAKE, qs_stride=2, st=None)


@pytest.mark.parametrize("over", [dict(g=None), dict(g_stride=511), dict(g_dtype=E4M3), dict(n=-1), dict(f=0), dict(q=None),
                                  dict(qs=None), dict(q_stride=1), dict(qs_stride=1), dict(nd=FAKE + 1)], ids=str)
def test_silu_refusals(over):
    assert qm.load().qs_silu_mul_quant(*change(SILU, **over)) == INV


MM = dict(a=FAKE, a_stride=256, sa=FAKE, sa_stride=2, w=FAKE, w_stride=256, we=256 * 64, sw=FAKE, off=FAKE, e=4, m=8, n=64, k=256,
          out=FAKE, o_stride=64, o_dtype=BF16, ws=FAKE, bytes=BIG, st=None)


@pytest.mark.parametrize("over,code", [
    (dict(a=None), INV), (dict(a=FAKE + 8), INV), (dict(a_stride=264), INV), (dict(a_stride=240), INV), (dict(sa=None), INV),
    (dict(sa_stride=1), INV), (dict(w=None), INV), (dict(w=FAKE + 4), INV), (dict(w_stride=250), INV), (dict(w_stride=128), INV),
    (dict(we=256 * 63), INV), (dict(we=256 * 64 + 8), INV), (dict(sw=None), INV), (dict(off=None), INV), (dict(off=FAKE + 2), INV),
    (dict(e=0), INV), (dict(e=1025), INV), (dict(m=-1), INV), (dict(n=0), INV), (dict(k=0), INV), (dict(out=None), INV),
    (dict(o_stride=63), INV), (dict(o_dtype=E4M3), INV), (dict(out=FAKE + 1), INV), (dict(ws=None), WS), (dict(ws=FAKE + 16), WS),
    (dict(bytes=16), WS)], ids=str)
def test_matmul_refusals(over, code):
    assert qm.load().qs_fp8_matmul(*change(MM, **over)) == code


DISPATCH = dict(ids=FAKE, t=8, k=2, e=16, c=FAKE, o=FAKE, p=FAKE, pos=FAKE, x=FAKE, x_stride=256, x_dtype=E4M3, sx=FAKE, sx_stride=2,
                h=256, xs=FAKE, xs_stride=256, sxs=FAKE, sxs_stride=2, ws=FAKE, bytes=BIG, st=None)


@pytest.mark.parametrize("over,code", [
    (dict(ids=None), INV), (dict(t=-1), INV), (dict(k=0), INV), (dict(k=33), INV), (dict(e=0), INV), (dict(e=1025), INV),
    (dict(t=1 << 30), INV), (dict(c=None), INV), (dict(o=None), INV), (dict(p=None), INV), (dict(pos=None), INV),
    (dict(pos=FAKE + 2), INV), (dict(x=None), INV), (dict(x_stride=1), INV), (dict(x_dtype=9), INV), (dict(sx=None), INV),
    (dict(sxs=None), INV), (dict(sxs_stride=1), INV), (dict(xs_stride=255), INV), (dict(h=0), INV), (dict(ws=None), WS),
    (dict(ws=FAKE + 128), WS), (dict(bytes=8), WS)], ids=str)
def test_dispatch_refusals(over, code):
    assert qm.load().qs_dispatch_tokens(*change(DISPATCH, **over)) == code


COMBINE = dict(y=FAKE, y_stride=256, y_dtype=BF16, pos=FAKE, w=FAKE, t=8, k=2, h=256, out=FAKE, o_stride=256, o_dtype=F32, st=None)


@pytest.mark.parametrize("over", [dict(y=None), dict(y_dtype=E4M3), dict(y_stride=0), dict(pos=None), dict(pos=FAKE + 1), dict(w=FAKE + 2),
                                  dict(t=-1), dict(k=0), dict(k=40), dict(h=0), dict(out=None), dict(o_stride=255), dict(o_dtype=5)], ids=str)
def test_combine_refusals(over):
    assert qm.load().qs_combine_tokens(*change(COMBINE, **over)) == INV


COMBINE_BWD = dict(d=FAKE, d_stride=256, d_dtype=BF16, y=FAKE, y_stride=256, y_dtype=BF16, pos=FAKE, w=FAKE, t=8, k=2, h=256, dy=FAKE,
                   dy_stride=256, dy_dtype=BF16, dw=FAKE, st=None)


@pytest.mark.parametrize("over", [dict(d=None), dict(y=None), dict(y_stride=7), dict(pos=None), dict(dy=None), dict(dy_dtype=E4M3),
                                  dict(dw=FAKE + 2), dict(k=0), dict(h=-5), dict(dy_stride=0)], ids=str)
def test_combine_backward_refusals(over):
    assert qm.load().qs_combine_tokens_backward(*change(COMBINE_BWD, **over)) == INV


def test_workspace_sizes():
    L = qm.load()
    assert L.qs_rmsnorm_backward_workspace_bytes(2048) >= 2048 * 4
    assert L.qs_rmsnorm_backward_workspace_bytes(0) == 0 and L.qs_rmsnorm_backward_workspace_bytes(16385) == 0
    assert L.qs_fp8_matmul_workspace_bytes(8, 64, 256, 1) >= 256
    for bad in [(-1, 64, 256, 1), (8, 0, 256, 1), (8, 64, 0, 1), (8, 64, 256, 0), (8, 64, 256, 1025)]:
        assert L.qs_fp8_matmul_workspace_bytes(*bad) == 0
    assert L.qs_dispatch_workspace_bytes(0, 8, 256) >= 256
    assert L.qs_dispatch_workspace_bytes(65536, 8, 256) > L.qs_dispatch_workspace_bytes(1, 8, 256)
    for bad in [(-1, 8, 256), (8, 0, 256), (8, 33, 256), (8, 8, 0), (8, 8, 2000), (1 << 28, 8, 256)]:
        assert L.qs_dispatch_workspace_bytes(*bad) == 0


def test_nothing_is_launched_for_no_rows():
    L = qm.load()
    assert L.qs_rmsnorm_residual(*change(NORM, n=0)) == qm.QS_OK
    assert L.qs_silu_mul_quant(*change(SILU, n=0)) == qm.QS_OK
    assert L.qs_fp8_matmul(*change(MM, m=0)) == qm.QS_OK
    assert L.qs_combine_tokens(*change(COMBINE, t=0)) == qm.QS_OK
    assert L.qs_combine_tokens_backward(*change(COMBINE_BWD, t=0)) == qm.QS_OK


def test_binding_refuses_wrong_tensors():
    host = torch.zeros(2, 256)
    with pytest.raises(ValueError, match="device memory"):
        qm.qs_rmsnorm_residual(host, None, torch.ones(256), 1e-6, y=host)
    with pytest.raises(ValueError, match="device memory"):
        qm.qs_silu_mul_quant(torch.zeros(2, 512), torch.zeros(2, 256, dtype=torch.float8_e4m3fn), torch.zeros(2, 2))
    with pytest.raises(ValueError, match="matrix"):
        qm.qs_rmsnorm_residual(torch.zeros(256), None, torch.ones(256), 1e-6, y=host)
    with pytest.raises(ValueError, match="workspace"):
        qm.qs_rmsnorm_residual_backward(host, host, 1e-6, host, None, host, dweight=host)
    with pytest.raises(ValueError, match="come together"):
        qm.qs_dispatch_tokens(torch.zeros(2, 2, dtype=torch.int32), host, None, torch.zeros(4), None, None, None, None, None, host)
    with pytest.raises(ValueError, match="needs y"):
        qm.qs_combine_tokens_backward(host, None, torch.zeros(2, 2, dtype=torch.int32), None, host, dtopk_w=host)
    with pytest.raises(ValueError, match="experts, cols, inner"):
        qm.qs_fp8_matmul(host, host, host, host, host, host, offsets=host)
