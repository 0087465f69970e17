"""Expert rows of 128 MiB and more, which combine and the sort's gradient read
past the caches: whole 16-byte rows, and odd ones that are only element-aligned."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gemv_expert_id_amd as mm
from test_gpu_moe import DEV, Padded, TORCH, U, ids_buf, some_ids, stream

pytestmark = pytest.mark.gpu


# 4100 x 8 rows: above 128 MiB at each width
@pytest.mark.parametrize("dt,h,pad", [(0, 1024, 0), (0, 1027, 2), (1, 2048, 0), (1, 2051, 4), (2, 2048, 0), (2, 2049, 1)])
@pytest.mark.parametrize("what", ["combine", "combine in place", "sort_grad"])
def test_rows_read_past_the_caches(dt, h, pad, what):
    m, k, E = 4100, 8, 40
    t, z = TORCH[dt], torch.tensor([], dtype=TORCH[dt]).element_size()
    assert m * k * h * z >= 128 << 20
    ids = some_ids(m, k, E, h, repeat=True)
    ids[1] = 0xFFFFFFFF
    key = np.minimum(ids.reshape(-1).astype(np.int64), E)
    order = np.argsort(key, kind="stable")
    pos = np.empty(m * k, dtype=np.uint32)
    pos[order] = np.arange(m * k)
    off = np.searchsorted(key[order], np.arange(E + 1)).astype(np.uint32)
    live = int(off[E])
    shift = pad % 2
    g = torch.Generator(device=DEV).manual_seed(h)
    y = torch.randn(m * k, h, generator=g, device=DEV).to(t)
    y[live:] = float("nan")
    rows = Padded(m * k, h, t, h + pad, shift, y)
    out = Padded(m, h, t, h + pad, shift)
    w = torch.rand(m, k, generator=g, device=DEV)
    res = torch.randn(m, h, generator=g, device=DEV).to(t)
    doff, dpos = ids_buf(off), ids_buf(pos)
    p = mm.sort_params(dt, m, k, E, h, ld_tokens=h + pad, ld_rows=h + pad)
    if what == "sort_grad":
        w.fill_(1.0)
        res.zero_()
        mm.mm_id_sort_grad(p, rows.buf, mm.buf(doff), mm.buf(dpos), out.buf, stream=stream())
    else:
        if what == "combine":
            apart = Padded(m, h, t, h + pad, shift, res)
            rb = apart.buf
        else:
            out.t.copy_(res)
            rb = out.buf
        mm.mm_id_combine(p, rows.buf, mm.buf(doff), mm.buf(dpos), mm.buf(w), rb, out.buf, stream=stream())
    torch.cuda.synchronize()
    y[live:] = 0
    at = torch.from_numpy(pos.astype(np.int64)).to(DEV).reshape(m, k)
    wl = torch.where(at < live, w, torch.zeros_like(w)).double()
    for t0 in range(0, m, 256):
        s = slice(t0, t0 + 256)
        terms = wl[s, :, None] * y[at[s]].double()
        want = res[s].double() + terms.sum(1)
        mag = res[s].double().abs() + terms.abs().sum(1)
        # k + 1 additions in 32 bits, then half a step of the type
        half = torch.finfo(t).eps / 2 * want.abs().clamp_min(torch.finfo(t).tiny)
        assert bool(((out.t[s].double() - want).abs() <= half + (k + 1) * U * mag).all())
    out.untouched()
