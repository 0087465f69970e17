"""A dense transformer layer's feed-forward block through the library: a training
step, and serving with 8-bit weights and activations.

    python examples/feed_forward.py

y = down(act(gate x) * up x). Training: mm_gated keeps the pre-activations, mm_gemm
does the down projection, and mm_gated_grad gives the gradients of the block's input
and of both projections in one call. Serving: every weight row is turned into 8-bit
codes with a scale once (mm_i8_quant); a call turns the tokens into codes, multiplies
and gates (mm_i8_gemm), and does the same for the down projection. Every buffer is
allocated once, so a loop can call `run` again, or capture it into a graph.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemv_expert_id_amd as mm  # noqa: E402

CODE = {torch.float32: mm.MM_F32, torch.float16: mm.MM_F16, torch.bfloat16: mm.MM_BF16}


def codes(rows: torch.Tensor):
    """8-bit codes of each row and their scales."""
    q = torch.empty(rows.shape, dtype=torch.int8, device=rows.device)
    scales = torch.empty(rows.shape[0], device=rows.device)
    p = mm.quant_params(CODE[rows.dtype], *rows.shape)
    mm.mm_i8_quant(p, mm.buf(rows), mm.buf(q), mm.buf(scales), stream=torch.cuda.current_stream())
    return q, scales


class ServingBlock:
    """gate_up [2n, width] and down [width, n] in 8-bit codes, for `m` tokens a call; width and n multiples of 16."""

    def __init__(self, gate_up, down, m: int, dtype=torch.bfloat16, gate: int = mm.MM_GATE_SILU):
        n2, width = gate_up.shape
        n, dev, dt = n2 // 2, gate_up.device, CODE[dtype]
        self.gate_up, self.down = codes(gate_up), codes(down)
        empty = lambda *shape, d=dtype: torch.empty(*shape, dtype=d, device=dev)  # noqa: E731
        self.qx, self.sx = empty(m, width, d=torch.int8), empty(m, d=torch.float32)
        self.h, self.qh, self.sh = empty(m, n), empty(m, n, d=torch.int8), empty(m, d=torch.float32)
        self.y = empty(m, width)
        self.p_x, self.p_h = mm.quant_params(dt, m, width), mm.quant_params(dt, m, n)
        self.p_up = mm.i8_params(dt, m, n, width, gate=gate)
        self.p_down = mm.i8_params(dt, m, width, n)

    def run(self, x: torch.Tensor, stream=None) -> torch.Tensor:
        """x [m, width]; returns the block's buffer [m, width]."""
        s, b = stream or torch.cuda.current_stream(), mm.buf
        mm.mm_i8_quant(self.p_x, b(x), b(self.qx), b(self.sx), stream=s)
        mm.mm_i8_gemm(self.p_up, b(self.qx), b(self.sx), *[b(t) for t in self.gate_up], b(self.h), stream=s)
        mm.mm_i8_quant(self.p_h, b(self.h), b(self.qh), b(self.sh), stream=s)
        mm.mm_i8_gemm(self.p_down, b(self.qh), b(self.sh), *[b(t) for t in self.down], b(self.y), stream=s)
        return self.y


def train_step(x, gate_up, down, dy, gate: int = mm.MM_GATE_SILU, keep: bool = True):
    """y = down . (act(gate x) * up x) and the gradients of sum(y * dy): returns y, dx, dgate_up, ddown. Without
    `keep` the pre-activations are computed again in the backward pass instead of being kept."""
    (m, width), n, dt, dev = x.shape, gate_up.shape[0] // 2, CODE[x.dtype], x.device
    s, b = torch.cuda.current_stream(), mm.buf
    empty = lambda *shape: torch.empty(*shape, dtype=x.dtype, device=dev)  # noqa: E731
    h, y, dh, dx, pre = empty(m, n), empty(m, width), empty(m, n), empty(m, width), empty(m, 2 * n)
    dgate_up, ddown = torch.empty_like(gate_up), torch.empty_like(down)
    p = mm.gated_params(dt, m, n, width, gate=gate)
    kept = b(pre) if keep else None

    mm.mm_gated(p, b(x), b(gate_up), b(h), kept, stream=s)
    mm.mm_gemm(mm.gemm_desc(dt, m, width, n, trans_b=True), b(h), b(down), b(y), stream=s)

    mm.mm_gemm(mm.gemm_desc(dt, m, n, width), b(dy), b(down), b(dh), stream=s)
    mm.mm_gemm(mm.gemm_desc(dt, width, n, m, trans_a=True), b(dy), b(h), b(ddown), stream=s)
    # The pre-activations' gradients take their place.
    mm.mm_gated_grad(p, b(x), b(gate_up), kept, b(dh), b(pre), b(dx), b(dgate_up), stream=s)
    return y, dx, dgate_up, ddown


def main():
    g = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *shape, scale=1.0: torch.randn(*shape, generator=g, device="cuda") * scale  # noqa: E731
    width, n = 4096, 11008
    gate_up, down = randn(2 * n, width, scale=0.02), randn(width, n, scale=0.01)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for m in (1, 16, 512):
        block = ServingBlock(gate_up, down, m)
        x = randn(m, width).to(torch.bfloat16)
        for _ in range(3):
            block.run(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            block.run(x)
        graph.replay()
        start.record()
        for _ in range(50):
            graph.replay()
        end.record()
        torch.cuda.synchronize()
        print(f"serving, {m} tokens: {start.elapsed_time(end) * 20:.1f} us a block ({width} x {n}, 8-bit)", flush=True)
    w, d = gate_up.to(torch.bfloat16), down.to(torch.bfloat16)
    x, dy = randn(2048, width).to(torch.bfloat16), randn(2048, width).to(torch.bfloat16)
    for keep in (True, False):
        train_step(x, w, d, dy, keep=keep)
        start.record()
        y, dx, dw, dd = train_step(x, w, d, dy, keep=keep)
        end.record()
        torch.cuda.synchronize()
        how = "pre-activations kept" if keep else "computed again"
        print(f"training step, 2048 tokens, {how}: {start.elapsed_time(end):.2f} ms; gradient norms "
              f"{[round(float(t.float().norm()), 1) for t in (dx, dw, dd)]}", flush=True)


if __name__ == "__main__":
    main()
