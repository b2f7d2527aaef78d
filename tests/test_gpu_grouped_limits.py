"""The 16-bit products whose rows choose their matrix at their limits: offsets whose ranges overlap (GPU)."""
import pytest

torch = pytest.importorskip("torch")

import grouped_reference as ref
from routed_expert_ffn_gemv_gb300 import _lib as L
from test_gpu_grouped import gen, matmul, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def status():
    L.moe_device_status(clear=True)
    yield
    torch.cuda.synchronize()
    assert L.moe_device_status(clear=True) == 0


# ------------------------------------------------------------------------------ offsets that descend

def owned(o, R):
    """The rows of each group: those of its range, where it is one, that no earlier group has."""
    end, rows = 0, []
    for a, b in zip(o, o[1:]):
        ok = 0 <= a <= b <= R
        rows.append((max(a, end), b) if ok and max(a, end) < b else (0, 0))
        end = max(end, b) if ok else end
    return rows


# few rows, narrow tiles that share their reduction (nine items for clusters of seven), narrow tiles, pairs
@pytest.mark.parametrize("R,N,K", [(8, 64, 128), (80, 128, 512), (80, 128, 2048), (60, 4096, 64), (2000, 136, 72)])
@pytest.mark.parametrize("t,out", [("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("form", ["alternating", "overlapping", "many", "outside"])
def test_ranges_that_overlap_are_cut_and_recorded(R, N, K, t, out, form):
    o = {"alternating": [0, R, 0, R, 0, R],
         "overlapping": [0, R // 2, R // 4, R - 1, R // 3, R],
         "many": [R // 2, R] * 150 + [1, R // 2 + 1, R],
         "outside": [2, -3, 4, R + 1, 1, R // 2, R // 2, 0, R]}[form]
    g, G = gen(R + K), len(o) - 1
    x, w = rand(g, t, R, K), rand(g, t, G, N, K, scale=K ** -0.5)
    d_off = torch.tensor(o, dtype=torch.int32, device="cuda")
    for _ in range(3):
        y = matmul(x, t, d_off, w, L.MOE_ORDER_NK, N, K, G=G, R=R, out=out)
        assert L.moe_device_status(clear=True) == L.MOE_ERR_INVALID
        free = torch.ones(R, dtype=torch.bool, device="cuda")
        for i, (a, b) in enumerate(owned(o, R)):
            if b > a:
                free[a:b] = False
                v, e = ref.product(x[a:b], w[i])
                ref.check(y[a:b], v, ref.rounded(v, e, out), i)
        assert bool((y[free] == 7.0).all())


@pytest.mark.parametrize("out", ["f32", "f16"])
@pytest.mark.parametrize("form", ["alternating", "overlapping"])
def test_gradient_of_ranges_that_overlap(out, form):
    g, R, N, K = gen(2), 300, 72, 136
    o = {"alternating": [0, R, 0, R, 0, R], "overlapping": [0, R // 2, R // 4, R - 1, R // 3, R]}[form]
    G = len(o) - 1
    x, dy = rand(g, "f16", R, K), rand(g, "f16", R, N)
    dw = torch.full((G, N, K), float("nan"), dtype=ref.dtype(out), device="cuda")
    L.moe_grouped_weight_grad(x, L.MOE_F16, R, K, None, 1, dy, R, N, None, torch.tensor(o, dtype=torch.int32, device="cuda"), G, R,
                              N, K, 0, dw, ref.code(out))
    torch.cuda.synchronize()
    assert L.moe_device_status(clear=True) == L.MOE_ERR_INVALID
    for i, (a, b) in enumerate(owned(o, R)):
        if b > a:
            v, e = ref.product(dy[a:b].T, x[a:b].T)
            ref.check(dw[i], v, ref.rounded(v, e, out), i)
        else:
            assert bool((dw[i] == 0).all())
