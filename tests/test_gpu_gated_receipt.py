"""The receipt of mm_gated_grad describes the last of the call's launches alone."""
from __future__ import annotations

import pytest
import torch

import gemv_expert_id_amd as mm
from ffn_ref import TORCH

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
OWN, GEMM = mm.MM_KERNEL_GATED_GRAD, mm.MM_KERNEL_GEMM_LARGE
FORMS = {16 + 4096 * 16, 32 + 4096 * 16, 64 + 4096 * 64, 64 + 4096 * 128, 128 + 4096 * 128, 256 + 4096 * 128, 256 + 4096 * 256}


# dx and dw: the kernel that makes each; all four mixtures (a pitch of 3980 elements
# is no whole number of 16-byte pieces)
@pytest.mark.parametrize("dt,m,n,k,dx,dw", [
    (2, 770, 3520, 1472, GEMM, OWN), (2, 4001, 1024, 4096, GEMM, OWN), (1, 4001, 1024, 4096, GEMM, OWN),
    (2, 3329, 1990, 4096, OWN, OWN), (2, 3329, 1992, 4096, OWN, GEMM), (1, 2048, 1024, 2048, GEMM, GEMM), (1, 300, 257, 96, OWN, OWN),
    (0, 40, 600, 65, OWN, OWN), (0, 300, 1409, 72, OWN, OWN), (2, 9, 2048, 64, OWN, OWN)])
@pytest.mark.parametrize("saved", [True, False])
def test_last_launch(dt, m, n, k, dx, dw, saved):
    t, b = TORCH[dt], mm.buf
    e = lambda *shape: torch.zeros(*shape, dtype=t, device=DEV)  # noqa: E731
    x, w, pre, dh, dpre, gx, gw = e(m, k), e(2 * n, k), e(m, 2 * n), e(m, n), e(m, 2 * n), e(m, k), e(2 * n, k)
    for to_x, to_w in ((1, 1), (1, 0), (0, 1), (0, 0)):
        r = mm.mm_gated_grad(mm.gated_params(dt, m, n, k), b(x), b(w), b(pre) if saved else None, b(dh), b(dpre),
                             b(gx) if to_x else None, b(gw) if to_w else None, stream=torch.cuda.current_stream())
        assert r.route == mm.MM_ROUTE_GATED and r.dtype == dt and r.dispatch_count == 1 + to_x + to_w
        last = dw if to_w else dx if to_x else OWN
        assert r.kernel == last
        if last == GEMM:
            assert r.variant in (128, 129, 256, 257)
        elif to_x or to_w or saved:
            assert r.variant == 0
        else:
            assert r.variant in (FORMS if dt else FORMS | {0})
