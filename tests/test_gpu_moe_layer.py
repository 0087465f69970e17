"""The example layer against a 64-bit computation of the same layer."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

import moe_ref as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rel(got, want):
    return float((got.double().cpu() - want).norm() / want.norm())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m", [1, 3, 40])
def test_serving_layer(ex, dtype, m):
    E, top_k, width, n, group = 8, 3, 256, 96, 32
    g = torch.Generator().manual_seed(m)
    gate_up, down = torch.randn(E, 2 * n, width, generator=g) * 0.05, torch.randn(E, width, n, generator=g) * 0.05
    x, logits = torch.randn(m, width, generator=g).to(dtype), torch.randn(m, E, generator=g).to(dtype)
    layer = ex.ServingLayer(gate_up.cuda(), down.cuda(), m, top_k, dtype=dtype, group=group)
    xd, ld = x.cuda(), logits.cuda()
    got = layer.run(xd, ld).clone()
    torch.cuda.synchronize()

    wu = ref.q4_weights(*layer.gate_up, group)
    wd = ref.q4_weights(*layer.down, group)
    ids, w = ref.topk(logits.double().numpy(), top_k, True)
    want = x.double().clone()
    for t in range(m):
        for s in range(top_k):
            h = wu[int(ids[t, s])] @ x[t].double()
            mid = h[:n] * torch.sigmoid(h[:n]) * h[n:]
            want[t] += w[t, s] * (wd[int(ids[t, s])] @ mid)
    # Three roundings to the type on the way (mid, ys, out), each at most half a
    # step of its value; the sums in 32 bits are far below that for 16 bits.
    u = torch.finfo(dtype).eps / 2
    assert rel(got, want) <= 3 * u + 1e-5


@pytest.mark.parametrize("m,E,top_k", [(1, 4, 2), (50, 6, 2), (33, 3, 3)])
def test_training_step(ex, m, E, top_k):
    width = 64
    g = torch.Generator().manual_seed(m)
    x, logits = torch.randn(m, width, generator=g), torch.randn(m, E, generator=g)
    w, dout = torch.randn(E, width, width, generator=g) * 0.1, torch.randn(m, width, generator=g)
    out, dx, dl, dw = ex.train_step(x.cuda(), logits.cuda(), w.cuda(), dout.cuda(), top_k)
    torch.cuda.synchronize()

    xd, ld, wd = (t.double().requires_grad_() for t in (x, logits, w))
    top = ld.topk(top_k, dim=1)
    weight = torch.softmax(top.values, 1)
    y = torch.stack([torch.stack([wd[int(e)] @ xd[t] for e in top.indices[t]]) for t in range(m)])
    full = xd + (weight[..., None] * y).sum(1)
    (full * dout.double()).sum().backward()
    # f32 throughout: products of 64 or m terms, 1e-6 sqrt(k) of the operands' range each
    for got, want in ((out, full.detach()), (dx, xd.grad), (dl, ld.grad), (dw, wd.grad)):
        assert rel(got, want) <= 2e-5
