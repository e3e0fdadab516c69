"""Refusals of the row operators: every bad argument is answered on the host, before a GPU is touched."""
import pytest
import torch

from bit_quantized_moe_router_gb300 import qs_moe as qm

FAKE = 1 << 40   # an address that is never read: the checks come first
INV, WS = qm.QS_ERR_INVALID, qm.QS_ERR_WORKSPACE
F32, BF16, E4M3 = qm.QS_F32, qm.QS_BF16, qm.QS_E4M3
BIG = 1 << 40


def call(name, base, over):
    """The entry point on the packed struct of base's fields with some of them changed."""
    assert set(over) <= set(base)
    return getattr(qm.load(), name)(qm.ARGS[name].pack(*{**base, **over}.values()), None)


def rows(name, stride=256, dtype=BF16):
    return {name: FAKE, name + "_stride": stride, name + "_dtype": dtype}


def codes(name, stride=256):
    return {name: FAKE, name + "_stride": stride, name + "_scale": FAKE, name + "_scale_stride": 2}


NORM = {**rows("x"), **rows("r"), **rows("s"), **rows("y"), **codes("q"), "w": FAKE, "eps": 1e-6, "n": 4, "h": 256}


@pytest.mark.parametrize("over", [
    dict(x=0), dict(x_dtype=E4M3), dict(x_dtype=7), dict(x_stride=255), dict(x=FAKE + 1), dict(w=0), dict(w=FAKE + 2),
    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(n=-1), dict(h=0), dict(h=16385), dict(r_stride=0),
    dict(r_dtype=-1), dict(s_stride=10), dict(y_dtype=E4M3), dict(y=FAKE + 1), dict(q_stride=255), dict(q_scale=0), dict(q=0),
    dict(q_scale_stride=1), dict(q_scale=FAKE + 2), dict(s=0, y=0, q=0, q_scale=0)], ids=str)
def test_norm_refusals(over):
    assert call("qs_rmsnorm_residual", NORM, over) == INV


BWD = {**rows("s", 256, F32), **rows("dy", 256, F32), **rows("ds", 256, F32), **rows("dx", 256, F32), "w": FAKE, "dw": FAKE, "ws": FAKE,
       "bytes": BIG, "eps": 1e-6, "n": 4, "h": 256}


@pytest.mark.parametrize("over,code", [
    (dict(s=0), INV), (dict(dy=0), INV), (dict(dx=0), INV), (dict(w=0), INV), (dict(h=20000), INV),
    (dict(n=-2), INV), (dict(dy_stride=1), INV), (dict(ds_dtype=E4M3), INV), (dict(dx=FAKE + 2), INV), (dict(dw=FAKE + 1), INV),
    (dict(ws=0), WS), (dict(ws=FAKE + 8), WS), (dict(bytes=1000), WS)], ids=str)
def test_norm_backward_refusals(over, code):
    assert call("qs_rmsnorm_residual_backward", BWD, over) == code


SILU = {**rows("g", 512), **codes("q"), "nd": 0, "n": 4, "f": 256}


@pytest.mark.parametrize("over", [dict(g=0), dict(g_stride=511), dict(g_dtype=E4M3), dict(n=-1), dict(f=0), dict(q=0),
                                  dict(q_scale=0), dict(q_stride=1), dict(q_scale_stride=1), dict(nd=FAKE + 1)], ids=str)
def test_silu_refusals(over):
    assert call("qs_silu_mul_quant", SILU, over) == INV


MM = {**codes("a"), "w": FAKE, "w_stride": 256, "we": 256 * 64, "sw": FAKE, "off": FAKE, **rows("out", 64), "ws": FAKE, "bytes": BIG,
      "e": 4, "m": 8, "n": 64, "k": 256}


@pytest.mark.parametrize("over,code", [
    (dict(a=0), INV), (dict(a=FAKE + 8), INV), (dict(a_stride=264), INV), (dict(a_stride=240), INV), (dict(a_scale=0), INV),
    (dict(a_scale_stride=1), INV), (dict(w=0), INV), (dict(w=FAKE + 4), INV), (dict(w_stride=250), INV), (dict(w_stride=128), INV),
    (dict(we=256 * 63), INV), (dict(we=256 * 64 + 8), INV), (dict(sw=0), INV), (dict(off=0), INV), (dict(off=FAKE + 2), INV),
    (dict(e=0), INV), (dict(e=1025), INV), (dict(m=-1), INV), (dict(n=0), INV), (dict(k=0), INV), (dict(out=0), INV),
    (dict(out_stride=63), INV), (dict(out_dtype=E4M3), INV), (dict(out=FAKE + 1), INV), (dict(ws=0), WS), (dict(ws=FAKE + 16), WS),
    (dict(bytes=16), WS)], ids=str)
def test_matmul_refusals(over, code):
    assert call("qs_fp8_matmul", MM, over) == code


DISPATCH = {"ids": FAKE, "c": FAKE, "o": FAKE, "p": FAKE, "pos": FAKE, **rows("x", 256, E4M3), **rows("xs", 256, E4M3), "sx": FAKE,
            "sx_stride": 2, "sxs": FAKE, "sxs_stride": 2, "ws": FAKE, "bytes": BIG, "t": 8, "k": 2, "e": 16, "h": 256}


@pytest.mark.parametrize("over,code", [
    (dict(ids=0), INV), (dict(t=-1), INV), (dict(k=0), INV), (dict(k=33), INV), (dict(e=0), INV), (dict(e=1025), INV),
    (dict(t=1 << 30), INV), (dict(c=0), INV), (dict(o=0), INV), (dict(p=0), INV), (dict(pos=0), INV),
    (dict(pos=FAKE + 2), INV), (dict(x=0), INV), (dict(x_stride=1), INV), (dict(x_dtype=9, xs_dtype=9), INV), (dict(x_dtype=BF16), INV),
    (dict(sx=0), INV), (dict(sxs=0), INV), (dict(sxs_stride=1), INV), (dict(xs_stride=255), INV), (dict(h=0), INV), (dict(ws=0), WS),
    (dict(ws=FAKE + 128), WS), (dict(bytes=8), WS)], ids=str)
def test_dispatch_refusals(over, code):
    assert call("qs_dispatch_tokens", DISPATCH, over) == code


COMBINE = {**rows("y"), **rows("out", 256, F32), "pos": FAKE, "w": FAKE, "t": 8, "k": 2, "h": 256}


@pytest.mark.parametrize("over", [dict(y=0), dict(y_dtype=E4M3), dict(y_stride=0), dict(pos=0), dict(pos=FAKE + 1), dict(w=FAKE + 2),
                                  dict(t=-1), dict(k=0), dict(k=40), dict(h=0), dict(out=0), dict(out_stride=255), dict(out_dtype=5)], ids=str)
def test_combine_refusals(over):
    assert call("qs_combine_tokens", COMBINE, over) == INV


COMBINE_BWD = {**rows("d"), **rows("y"), **rows("dy"), "pos": FAKE, "w": FAKE, "dw": FAKE, "t": 8, "k": 2, "h": 256}


@pytest.mark.parametrize("over", [dict(d=0), dict(y=0), dict(y_stride=7), dict(pos=0), dict(dy=0), dict(dy_dtype=E4M3),
                                  dict(dw=FAKE + 2), dict(k=0), dict(h=-5), dict(dy_stride=0)], ids=str)
def test_combine_backward_refusals(over):
    assert call("qs_combine_tokens_backward", COMBINE_BWD, over) == INV


@pytest.mark.parametrize("name", list(qm.ARGS))
def test_missing_arguments_are_refused(name):
    assert getattr(qm.load(), name)(None, None) == INV


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
    assert call("qs_rmsnorm_residual", NORM, dict(n=0)) == qm.QS_OK
    assert call("qs_silu_mul_quant", SILU, dict(n=0)) == qm.QS_OK
    assert call("qs_fp8_matmul", MM, dict(m=0)) == qm.QS_OK
    assert call("qs_combine_tokens", COMBINE, dict(t=0)) == qm.QS_OK
    assert call("qs_combine_tokens_backward", COMBINE_BWD, dict(t=0)) == qm.QS_OK


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


@pytest.mark.parametrize("top_k", [1, 2, 3, 8, 32])
@pytest.mark.parametrize("experts", [1, 7, 256, 1024])
def test_a_dispatch_workspace_is_enough_for_every_smaller_call(top_k, experts):
    size = qm.load().qs_dispatch_workspace_bytes
    entries = [*range(1, 9000, 61), *range(260000, 273000, 32), *range(300000, 1200000, 7919), 1 << 24, (1 << 24) + 1, 1 << 30]
    tokens = sorted({max(1, n // top_k + d) for n in entries for d in (-1, 0, 1)} - {(1 << 30) // top_k + 1})
    sizes = [size(t, top_k, experts) for t in tokens]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    assert all(size(t, k, e) <= size(t, top_k, experts) for t in tokens[::50] for k, e in ((1, experts), (top_k, 1)))
    # a chunk of at least 1024 entries has its histogram
    assert all(s >= 4 * experts * min(256, t * top_k // 1024) for s, t in zip(sizes, tokens) if t * top_k > 4096)


class OnDevice:
    """What the binding reads of a CUDA tensor, for a device that need not be there."""

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.device, self.is_cuda = torch.Size(shape), dtype, f"cuda:{device}", True
        self._device = device

    def dim(self):
        return len(self.shape)

    def stride(self, d=None):
        strides = [1]
        for n in self.shape[:0:-1]:
            strides.insert(0, strides[0] * n)
        return tuple(strides) if d is None else strides[d]

    def numel(self):
        return self.shape.numel()

    @property
    def nbytes(self):
        return self.numel() * self.dtype.itemsize

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return FAKE

    def get_device(self):
        return self._device


F8, I32, BF, FP = torch.float8_e4m3fn, torch.int32, torch.bfloat16, torch.float32
OPERANDS = {  # entry point: its tensors by argument, the first operand first
    "qs_rmsnorm_residual": dict(x=((4, 256), BF), residual=((4, 256), BF), weight=((256,), FP), sum_out=((4, 256), BF),
                                y=((4, 256), BF), q=((4, 256), F8), q_scale=((4, 2), FP)),
    "qs_rmsnorm_residual_backward": dict(sum=((4, 256), FP), weight=((256,), FP), dy=((4, 256), FP), dsum=((4, 256), FP),
                                         dx=((4, 256), FP), dweight=((256,), FP), workspace=((1 << 22,), torch.uint8)),
    "qs_silu_mul_quant": dict(q=((4, 256), F8), gate_up=((4, 512), BF), q_scale=((4, 2), FP), n_rows=((1,), I32)),
    "qs_fp8_matmul": dict(a=((8, 256), F8), a_scale=((8, 2), FP), w=((3, 64, 256), F8), w_scale=((3, 1, 2), FP), out=((8, 64), FP),
                          workspace=((4096,), torch.uint8), offsets=((4,), I32)),
    "qs_dispatch_tokens": dict(topk_ids=((8, 2), I32), x=((8, 256), F8), x_scale=((8, 2), FP), counts=((16,), I32), offsets=((17,), I32),
                               perm=((16,), I32), pos=((8, 2), I32), xs=((16, 256), F8), xs_scale=((16, 2), FP), workspace=((4096,), torch.uint8)),
    "qs_combine_tokens": dict(pos=((8, 2), I32), y=((16, 256), BF), topk_w=((8, 2), FP), out=((8, 256), FP)),
    "qs_combine_tokens_backward": dict(pos=((8, 2), I32), dout=((8, 256), BF), y=((16, 256), BF), topk_w=((8, 2), FP), dy=((16, 256), BF),
                                       dtopk_w=((8, 2), FP)),
}


@pytest.fixture
def no_launch(monkeypatch):
    """Device 0 is current, and an entry point that is reached after all says so instead of running."""
    monkeypatch.setattr(qm, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0)

    class Library:
        def __getattr__(self, name):
            def entry(*args):
                raise RuntimeError(f"{name} reached")
            return entry

    monkeypatch.setattr(qm, "_lib", Library())


def on_devices(name, device, other=None):
    """The entry point's call with its operands on `device`, those in `other` on theirs."""
    at = other or {}
    operands = {k: OnDevice(shape, dtype, at.get(k, device)) for k, (shape, dtype) in OPERANDS[name].items()}
    return lambda: getattr(qm, name)(**operands, **({"eps": 1e-6} if "norm" in name else {}))


@pytest.mark.parametrize("name,operand", [(n, k) for n in OPERANDS for k in OPERANDS[n]])
def test_operands_of_two_devices_are_refused(no_launch, name, operand):
    with pytest.raises(ValueError, match="cuda:1"):
        on_devices(name, 0, {operand: 1})()


@pytest.mark.parametrize("name", list(OPERANDS))
def test_operands_on_a_device_that_is_not_current_are_refused(no_launch, name):
    with pytest.raises(ValueError, match="on cuda:1, but cuda:0 is the current device"):
        on_devices(name, 1)()
    with pytest.raises(RuntimeError, match=f"{name} reached"):  # those on the current one are not
        on_devices(name, 0)()


def test_a_row_limit_without_an_element_is_refused(no_launch, monkeypatch):
    """It has no address, and none means no limit: rows past the limit that was meant would be overwritten."""
    monkeypatch.setitem(OPERANDS["qs_silu_mul_quant"], "n_rows", ((0,), I32))
    with pytest.raises(ValueError, match="n_rows: expected an element"):
        on_devices("qs_silu_mul_quant", 0)()


@pytest.mark.parametrize("stride,cols", [(1 << 39, (1 << 25) + 1), (1 << 39, 1 << 29), (1 << 36, (1 << 28) + 1), ((1 << 40) - 16, 1 << 30)])
def test_strides_whose_product_passes_64_bits_are_refused(stride, cols):
    """An expert's rows would reach past the next expert's, by more than 64 bits count."""
    assert call("qs_fp8_matmul", MM, dict(w_stride=stride, n=cols, we=512, out_stride=cols)) == INV


@pytest.mark.parametrize("expert_stride,code", [(256 * 64, INV), (256 * 63 + 272, INV), (256 * 63 + 256, INV), (240, INV), (0, INV), (-16, INV),
                                                (272 * 63 + 240, INV), (272 * 63 + 256, WS)])
def test_experts_that_overlap_are_refused(expert_stride, code):
    """63 strides of 272 bytes and a last row of 256 is the least (without a workspace, so that nothing is launched)."""
    assert call("qs_fp8_matmul", MM, dict(w_stride=272, we=expert_stride, ws=0)) == code
