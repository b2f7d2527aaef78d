"""MXFP4 operators where their precision, launch limits and stream order are at their edges, against
64 bits (tests/mx4_reference.py)."""
import numpy as np
import pytest

import mx4_reference as ref
from routed_expert_ffn_gemv_gb300 import _lib as L

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from test_gpu_mx4 import DT, XT, Layer, clean_status, dev  # noqa: E402,F401


# ------------------------------------------------------------------ stream order

@pytest.mark.parametrize("E", [256, 20])
def test_layer_router_weights_of_the_kernel_before(E):
    """The stream's previous kernel writes w_router."""
    l = Layer(8, 2048, 32, E, 4, seed=21, bias=False, extra=False)
    want, ids, w = l.run()
    wr = l.d_wr.float()
    l.d_wr = torch.zeros_like(l.d_wr)
    y, ids2, w2 = torch.zeros_like(want), torch.zeros_like(ids), torch.zeros_like(w)
    for i in range(20):
        l.d_wr.zero_()
        y.fill_(7.0)
        l.d_wr.copy_(wr)
        L.moe_mx4_layer(l.x, L.MOE_F32, l.T, l.H, l.F, E, l.k, l.d_wr, None, l.table, l.n_slots, l.pool, l.sb, None, y,
                        ids2, w2, l.ws, l.ws.numel())
        assert torch.equal(ids2, ids) and torch.equal(w2, w) and torch.equal(y, want), i
