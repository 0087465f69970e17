"""The feed-forward block as a program uses it: the example's serving block and
training step against the 64-bit definitions, and the calls' behaviour on streams
and in graphs."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

import ffn_ref as ref
import gemv_expert_id_amd as mm
from ffn_ref import TORCH, U, rounding

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("feed_forward", os.path.join(ROOT, "examples", "feed_forward.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def randn(seed, *shape, scale=1.0, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def near(got, want, bound, what):
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), f"{what}: {float((err / bound).max()):.3g} of its bound"


@pytest.mark.parametrize("dt", [0, 1, 2])
@pytest.mark.parametrize("m", [1, 5, 130])
@pytest.mark.parametrize("gate", [ref.SILU, ref.GELU])
def test_serving(ex, dt, m, gate):
    t, width, n = TORCH[dt], 208, 144
    gate_up, down = randn(1, 2 * n, width, scale=0.1), randn(2, width, n, scale=0.1)
    block, x = ex.ServingBlock(gate_up, down, m, t, gate), randn(3, m, width, dtype=t)
    y = block.run(x)
    torch.cuda.synchronize()
    for rows, (q, s) in ((gate_up, block.gate_up), (down, block.down), (x, (block.qx, block.sx)), (block.h, (block.qh, block.sh))):
        wq, ws = ref.quantise(rows)
        assert torch.equal(q, wq) and torch.equal(s, ws)
    h, e = ref.i8(block.qx, block.sx, *block.gate_up, gate)
    near(block.h, h, e + rounding(dt, h.abs() + e), "h")
    want, e = ref.i8(block.qh, block.sh, *block.down, ref.NONE)
    near(y, want, e + rounding(dt, want.abs() + e), "y")
    # against the block in 64 bits: a code is off by at most half a scale, on both sides of each product
    full = ref.act(x.double() @ gate_up[:n].double().t(), gate) * (x.double() @ gate_up[n:].double().t())
    full = full @ down.double().t()
    assert float((y.double() - full).norm() / full.norm()) < 0.05


@pytest.mark.parametrize("dt", [0, 1, 2])
@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("m,width,n", [(7, 40, 24), (130, 136, 72), (300, 264, 520)])
def test_training_step(ex, dt, keep, m, width, n):
    t = TORCH[dt]
    x, dy = randn(1, m, width, dtype=t), randn(2, m, width, dtype=t)
    w, d = randn(3, 2 * n, width, scale=width ** -0.5, dtype=t), randn(4, width, n, scale=n ** -0.5, dtype=t)
    y, dx, dw, dd = ex.train_step(x, w, d, dy, keep=keep)
    xs = [v.double().requires_grad_() for v in (x, w, d)]
    pre = xs[0] @ xs[1].t()
    h = pre[:, :n] * torch.sigmoid(pre[:, :n]) * pre[:, n:]
    want = h @ xs[2].t()
    grads = torch.autograd.grad((want * dy.double()).sum(), xs)
    # in norm: each of at most six tensors on the way is rounded by half a step at most, f32 sums by 2^-24 a term
    tol = 6 * torch.finfo(t).eps / 2 + 2 * U * max(m, width, 2 * n)
    for got, v, what in ((y, want, "y"), (dx, grads[0], "dx"), (dw, grads[1], "dw"), (dd, grads[2], "ddown")):
        v = v.detach()
        assert float((got.double() - v).norm() / v.norm()) < tol, what


def calls(dt, m, n, k, seed):
    """Every entry point with buffers of its own; each returns its outputs."""
    t, s = TORCH[dt], seed * 10
    x, w, dh = randn(s, m, k, dtype=t), randn(s + 1, 2 * n, k, scale=0.1, dtype=t), randn(s + 2, m, n, dtype=t)
    e = lambda *shape, d=t: torch.zeros(*shape, dtype=d, device=DEV)  # noqa: E731
    h, pre, dpre, dx, dw, y = e(m, n), e(m, 2 * n), e(m, 2 * n), e(m, k), e(2 * n, k), e(m, n)
    q, qs, wq, ws = e(m, k, d=torch.int8), e(m, d=torch.float32), e(2 * n, k, d=torch.int8), e(2 * n, d=torch.float32)
    p, b = mm.gated_params(dt, m, n, k), mm.buf

    def run(stream):
        mm.mm_gated(p, b(x), b(w), b(h), b(pre), stream=stream)
        mm.mm_gated_grad(p, b(x), b(w), b(pre), b(dh), b(dpre), b(dx), b(dw), stream=stream)
        mm.mm_gated_grad(p, b(x), b(w), None, b(dh), b(pre), None, None, stream=stream)
        mm.mm_i8_quant(mm.quant_params(dt, m, k), b(x), b(q), b(qs), stream=stream)
        mm.mm_i8_quant(mm.quant_params(dt, 2 * n, k), b(w), b(wq), b(ws), stream=stream)
        mm.mm_i8_gemm(mm.i8_params(dt, m, n, k, gate=2), b(q), b(qs), b(wq), b(ws), b(y), stream=stream)

    return run, [h, pre, dpre, dx, dw, q, qs, wq, ws, y]


@pytest.mark.parametrize("dt", [0, 1, 2])
@pytest.mark.parametrize("m,n,k", [(1, 48, 64), (33, 200, 144), (200, 264, 400), (20, 700, 144), (280, 3272, 208), (1500, 1100, 1024)])
def test_graph_replays_and_streams(dt, m, n, k):
    """Replays, with eager work between them, and runs on two other streams at once give the eager bits."""
    run, outs = calls(dt, m, n, k, 1)
    run(torch.cuda.current_stream())
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(torch.cuda.current_stream())
    for _ in range(4):
        for t in outs:
            t.zero_()
        other, _ = calls(dt, m, n, k, 2)
        other(torch.cuda.current_stream())
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    streams = [torch.cuda.Stream() for _ in range(2)]
    pairs = [calls(dt, m, n, k, 1) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, (go, _) in zip(streams, pairs):
            go(s)
    torch.cuda.synchronize()
    for _, got in pairs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_example_runs(ex, capsys):
    ex.main()
    assert "training step" in capsys.readouterr().out
