"""One mixture-of-experts layer through the library: serving with 4-bit expert
weights, and a training step with plain weights.

    python examples/moe_layer.py

Serving: router (mm_topk), then for one token the experts' products by id
(mm_q4_id_direct), for several the rows in expert order (mm_id_sort,
mm_q4_id_sorted), and back to the tokens with weights onto the residual stream
(mm_id_combine). Training: the same around one mm_gemm for each expert, with
the gradients of all of it. Every buffer is allocated once, so a serving loop
can call `ServingLayer.run` again, or capture it into a graph.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemv_expert_id_amd as mm  # noqa: E402

CODE = {torch.float32: mm.MM_F32, torch.float16: mm.MM_F16, torch.bfloat16: mm.MM_BF16}


def quantise(w: torch.Tensor, group: int, scale_dtype=torch.bfloat16):
    """Codes, scales and biases of [.., N, k] weights in the layout of mm_q4_*."""
    g = w.float().reshape(*w.shape[:-1], -1, group)
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    scale = ((hi - lo) / 15).clamp_min(torch.finfo(scale_dtype).tiny).to(scale_dtype)
    bias = lo.to(scale_dtype)
    q = ((g - bias.float()) / scale.float()).round().clamp(0, 15).to(torch.uint8).reshape(*w.shape[:-1], -1, 2)
    return (q[..., 0] | q[..., 1] << 4).contiguous(), scale[..., 0].contiguous(), bias[..., 0].contiguous()


class ServingLayer:
    """x + sum over the chosen experts of weight * down(silu(gate x) * up x), for `m` tokens a call."""

    def __init__(self, gate_up, down, m: int, top_k: int, dtype=torch.bfloat16, group: int = 32):
        self.experts, n2, width = gate_up.shape  # [E, 2n, width], down [E, width, n]
        n, dev, dt = n2 // 2, gate_up.device, CODE[dtype]
        self.m, self.top_k, rows = m, top_k, m * top_k
        self.gate_up, self.down = quantise(gate_up, group), quantise(down, group)
        empty = lambda *shape, d=dtype: torch.empty(*shape, dtype=d, device=dev)  # noqa: E731
        self.ids, self.weights = empty(m, top_k, d=torch.int32), empty(m, top_k, d=torch.float32)
        self.xs, self.mid, self.ys = empty(rows, width), empty(rows, n), empty(rows, width)
        self.offsets = empty(self.experts + 1, d=torch.int32)
        self.order, self.position = empty(rows, d=torch.int32), empty(rows, d=torch.int32)
        self.out = empty(m, width)
        sdt = CODE[self.gate_up[1].dtype]
        self.p_topk = mm.topk_params(dt, m, self.experts, top_k, renormalize=1)
        self.p_sort = mm.sort_params(dt, m, top_k, self.experts, width)
        shared = dict(n_experts=self.experts, top_k=top_k)
        self.p_up = mm.q4_params(dt, sdt, m, n, width, group, gated=1, **shared)
        # By id, the second product's rows are one for each slot.
        self.p_down = mm.q4_params(dt, sdt, m, width, n, group, input_layout=int(m == 1), **shared)

    def run(self, x: torch.Tensor, logits: torch.Tensor, stream=None) -> torch.Tensor:
        """x [m, width], router logits [m, experts]; returns the layer's buffer [m, width]."""
        stream = stream or torch.cuda.current_stream()
        b = mm.buf
        up, down = [b(t) for t in self.gate_up], [b(t) for t in self.down]
        mm.mm_topk(self.p_topk, b(logits), b(self.ids), b(self.weights), stream=stream)
        if self.m == 1:  # by id: a row in routed order, no sort
            mm.mm_q4_id_direct(self.p_up, *up, b(x), b(self.ids), b(self.mid), stream=stream)
            mm.mm_q4_id_direct(self.p_down, *down, b(self.mid), b(self.ids), b(self.ys), stream=stream)
            offsets = position = None
        else:
            mm.mm_id_sort(self.p_sort, b(x), b(self.ids), b(self.xs), b(self.offsets), b(self.order),
                          b(self.position), stream=stream)
            mm.mm_q4_id_sorted(self.p_up, *up, b(self.xs), b(self.offsets), b(self.mid), stream=stream)
            mm.mm_q4_id_sorted(self.p_down, *down, b(self.mid), b(self.offsets), b(self.ys), stream=stream)
            offsets, position = b(self.offsets), b(self.position)
        mm.mm_id_combine(self.p_sort, b(self.ys), offsets, position, b(self.weights), b(x), b(self.out), stream=stream)
        return self.out


def train_step(x, logits, w, dout, top_k: int):
    """out = x + sum over the chosen of weight * W_e x for w [E, width, width], and the gradients of
    sum(out * dout): returns out, dx, dlogits, dw. One mm_gemm for each expert that has rows."""
    m, width = x.shape
    experts, dt, dev, rows = w.shape[0], CODE[x.dtype], x.device, x.shape[0] * top_k
    s, b = torch.cuda.current_stream(), mm.buf
    ids, weights = torch.empty(m, top_k, dtype=torch.int32, device=dev), torch.empty(m, top_k, device=dev)
    xs, ys, dys, dxs = (torch.empty(rows, width, dtype=x.dtype, device=dev) for _ in range(4))
    offsets = torch.empty(experts + 1, dtype=torch.int32, device=dev)
    order, position = (torch.empty(rows, dtype=torch.int32, device=dev) for _ in range(2))
    out, dx, dlogits = torch.empty_like(x), torch.empty_like(x), torch.empty_like(logits)
    dweights, dw = torch.empty_like(weights), torch.zeros_like(w)
    p_topk = mm.topk_params(dt, m, experts, top_k, renormalize=1)
    p_sort = mm.sort_params(dt, m, top_k, experts, width)

    mm.mm_topk(p_topk, b(logits), b(ids), b(weights), stream=s)
    mm.mm_id_sort(p_sort, b(x), b(ids), b(xs), b(offsets), b(order), b(position), stream=s)
    at = offsets.tolist()  # the products' sizes are host arguments
    for e in range(experts):
        lo, n = at[e], at[e + 1] - at[e]
        if n:
            d = mm.gemm_desc(dt, n, width, width, trans_b=True)
            mm.mm_gemm(d, b(xs[lo:lo + n]), b(w[e]), b(ys[lo:lo + n]), stream=s)
    mm.mm_id_combine(p_sort, b(ys), b(offsets), b(position), b(weights), b(x), b(out), stream=s)

    mm.mm_id_combine_grad(p_sort, b(dout), b(ys), b(offsets), b(position), b(weights), b(dys), b(dweights), stream=s)
    for e in range(experts):
        lo, n = at[e], at[e + 1] - at[e]
        if n:
            g = dys[lo:lo + n]
            mm.mm_gemm(mm.gemm_desc(dt, n, width, width), b(g), b(w[e]), b(dxs[lo:lo + n]), stream=s)
            mm.mm_gemm(mm.gemm_desc(dt, width, width, n, trans_a=True), b(g), b(xs[lo:lo + n]), b(dw[e]), stream=s)
    mm.mm_topk_grad(p_topk, b(logits), b(ids), b(dweights), b(dlogits), stream=s)
    mm.mm_id_sort_grad(p_sort, b(dxs), b(offsets), b(position), b(dx), stream=s)
    return out, dx + dout, dlogits, dw


def main():
    g = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *shape, scale=1.0: torch.randn(*shape, generator=g, device="cuda") * scale  # noqa: E731
    experts, top_k, width, n = 64, 8, 2048, 1408
    gate_up, down = randn(experts, 2 * n, width, scale=0.02), randn(experts, width, n, scale=0.02)
    for m in (1, 16, 64):
        layer = ServingLayer(gate_up, down, m, top_k)
        x, logits = randn(m, width).to(torch.bfloat16), randn(m, experts).to(torch.bfloat16)
        for _ in range(3):
            layer.run(x, logits)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer.run(x, logits)
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        graph.replay()
        start.record()
        for _ in range(100):
            graph.replay()
        end.record()
        torch.cuda.synchronize()
        print(f"serving, {m} tokens: {start.elapsed_time(end) * 10:.1f} us a layer "
              f"({experts} experts of {width} x {n}, top {top_k}, 4-bit)", flush=True)
    w = randn(8, 512, 512, scale=0.05)
    out, dx, dlogits, dw = train_step(randn(256, 512), randn(256, 8), w, randn(256, 512), 2)
    torch.cuda.synchronize()
    print("training step: gradient norms", [round(float(t.norm()), 3) for t in (dx, dlogits, dw)], flush=True)


if __name__ == "__main__":
    main()
