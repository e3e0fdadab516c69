"""An 8-bit mixture-of-experts FFN block from the row operators, next to the 2-bit layer's own routing.

Per token: the residual's addition and root-mean-square norm (the router reads the norm in bf16, the experts in
e4m3), router top-k, rows sorted to their experts, the gate/up product of every expert's rows, SwiGLU back to e4m3,
the down product, and the rows weighted and summed back.  Eight launches:

    python examples/fp8_moe_block.py --tokens 8

prints the time of a step and how far the block is from the same formulas in plain fp32 torch.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_quantized_moe_router_gb300 import qs_moe as qm  # noqa: E402

F8 = torch.float8_e4m3fn
EPS = 1e-6


def quantize_weights(w):
    """e4m3 codes and scales of fp32 weights [experts, cols, inner], one scale per 128 x 128 block."""
    e, n, k = w.shape
    p = torch.nn.functional.pad(w, (0, -k % 128, 0, -n % 128)).view(e, -(-n // 128), 128, -(-k // 128), 128)
    scale = p.abs().amax((2, 4)).clamp_min(2.0 ** -100) / 448
    codes = (p / scale[:, :, None, :, None]).reshape(e, -(-n // 128) * 128, -1)[:, :n, :k].to(F8)
    return codes.contiguous(), scale.contiguous()


class Fp8MoeBlock:
    """The block's weights, its buffers for up to max_tokens, and one step of it."""

    def __init__(self, hidden, ffn, experts, top_k, max_tokens, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.hidden, self.ffn, self.experts, self.top_k = hidden, ffn, experts, top_k
        self.norm = 1 + 0.1 * randn(hidden)
        self.router = randn(experts, hidden) / hidden ** 0.5
        self.gate_up = quantize_weights(randn(experts, 2 * ffn, hidden) / hidden ** 0.5)
        self.down = quantize_weights(randn(experts, hidden, ffn) / ffn ** 0.5)
        self.shape = qm.make_shape(hidden, experts, top_k, ffn, 0, qm.QS_BF16)
        t, n, blocks = max_tokens, max_tokens * top_k, lambda c: (c + 127) // 128
        buf = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device=device)  # noqa: E731
        i32 = torch.int32
        self.y, self.q, self.qs = buf(t, hidden, dtype=torch.bfloat16), buf(t, hidden, dtype=F8), buf(t, blocks(hidden))
        self.ids, self.weights = buf(t, top_k, dtype=i32), buf(t, top_k)
        self.counts, self.offsets = buf(experts, dtype=i32), buf(experts + 1, dtype=i32)
        self.perm, self.pos = buf(n, dtype=i32), buf(t, top_k, dtype=i32)
        self.xs, self.xss = buf(n, hidden, dtype=F8), buf(n, blocks(hidden))
        self.h, self.hq, self.hs = buf(n, 2 * ffn, dtype=torch.bfloat16), buf(n, ffn, dtype=F8), buf(n, blocks(ffn))
        self.ye = buf(n, hidden, dtype=torch.bfloat16)
        self.route_ws = qm.alloc_workspace(self.shape, t)
        self.dispatch_ws = qm.alloc_dispatch_workspace(t, top_k, experts)
        self.matmul_ws = qm.alloc_fp8_matmul_workspace(n, max(2 * ffn, hidden), max(hidden, ffn), experts)

    def step(self, x, residual, total, out):
        """out [tokens, hidden] of x and residual; total gets their sum, the next block's residual."""
        t = x.shape[0]
        n = t * self.top_k
        y, q, qs, ids, weights, pos = (b[:t] for b in (self.y, self.q, self.qs, self.ids, self.weights, self.pos))
        perm, xs, xss, h, hq, hs, ye = (b[:n] for b in (self.perm, self.xs, self.xss, self.h, self.hq, self.hs, self.ye))
        qm.qs_rmsnorm_residual(x, residual, self.norm, EPS, total, y, q, qs)
        qm.qs_route_topk(self.shape, y, self.router, None, t, ids, weights, self.route_ws)
        qm.qs_dispatch_tokens(ids, q, qs, self.counts, self.offsets, perm, pos, xs, xss, self.dispatch_ws)
        qm.qs_fp8_matmul(xs, xss, *self.gate_up, h, self.matmul_ws, self.offsets)
        qm.qs_silu_mul_quant(h, hq, hs, self.offsets[self.experts:])
        qm.qs_fp8_matmul(hq, hs, *self.down, ye, self.matmul_ws, self.offsets)
        qm.qs_combine_tokens(ye, pos, weights, out)

    def plain(self, x, residual, ids, weights):
        """The same without the 8-bit activations, in fp32, for given routing."""
        s = x.float() + residual.float()
        y = s * torch.rsqrt((s * s).mean(1, keepdim=True) + EPS) * self.norm
        wide = lambda c, s: c.float() * s.repeat_interleave(128, -2)[..., : c.shape[-2], :].repeat_interleave(128, -1)[..., : c.shape[-1]]  # noqa: E731
        out = torch.zeros_like(y)
        for e in ids.unique().tolist():
            token, slot = (ids == e).nonzero(as_tuple=True)
            gate, up = (y[token] @ wide(self.gate_up[0][e], self.gate_up[1][e]).T).chunk(2, 1)
            out.index_add_(0, token, weights[token, slot, None] * ((torch.nn.functional.silu(gate) * up) @ wide(self.down[0][e], self.down[1][e]).T))
        return out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--ffn", type=int, default=512)
    ap.add_argument("--experts", type=int, default=256)
    ap.add_argument("--top-k", type=int, default=8)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    block = Fp8MoeBlock(a.hidden, a.ffn, a.experts, a.top_k, a.tokens)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, residual = (torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16() for _ in range(2))
    total, out = torch.empty_like(x), torch.empty(a.tokens, a.hidden, device="cuda")
    block.step(x, residual, total, out)
    status = qm.qs_read_device_status(block.matmul_ws)
    if status != qm.QS_OK:
        raise qm.QsError(status, "qs_fp8_matmul")
    ref = block.plain(x, residual, block.ids[: a.tokens], block.weights[: a.tokens])
    rel = float((out - ref).norm() / ref.norm())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.step(x, residual, total, out)
    for _ in range(3):
        graph.replay()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"{a.tokens} tokens: {begin.elapsed_time(end) / a.steps * 1e3:.1f} us a step (graph), "
          f"rel-L2 against fp32 activations {rel:.2e}")
    return rel


if __name__ == "__main__":
    main()
