"""The 16-bit products whose rows choose their matrix at their limits: offsets whose ranges overlap, infinite weights of
adapters, empty groups (GPU)."""
import pytest

torch = pytest.importorskip("torch")

import grouped_reference as ref
from routed_expert_ffn_gemv_gb300 import _lib as L
from test_gpu_grouped import gen, lora, matmul, rand
from test_gpu_grouped_edges import LORA_PATHS

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


# ------------------------------------------------------------------------------ infinite weights

@pytest.mark.parametrize("T,N,K", LORA_PATHS)
@pytest.mark.parametrize("t,out", [("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("whole", [True, False])
def test_an_infinite_weight_gives_what_the_formula_gives(T, N, K, t, out, whole):
    """inf * u is an infinity of u's sign, however u is held (whole: u has the bits of one part, its others are 0); infinities of both
    signs, and a NaN, give NaN."""
    g, n, rank, inf = gen(T + N + whole), 3, 40, float("inf")
    x, w = rand(g, t, T, K), rand(g, t, N, K, scale=K ** -0.5)
    a, b = rand(g, t, n, rank, K, scale=K ** -0.5), rand(g, t, n, N, rank, scale=rank ** -0.5)
    if whole:
        a.zero_()
        a[:, torch.arange(rank), torch.arange(rank)] = 1.0
    adapter = torch.arange(T, device="cuda").int() % n
    put = [(0, 5, inf), (3, 39, -inf), (N - 1, 32, inf)]                      # one
    put += [(9, 3, inf), (9, 7, inf), (17, 2, inf), (17, 35, -inf), (33, 38, -inf), (33, 39, float("nan"))]  # two
    for m, r, v in put:
        b[1, m, r] = v
    y = lora(x, t, w, adapter, a, b, None, out)
    mine = adapter == 1
    u = x[mine].double() @ a[1].double().T
    for m in {p[0] for p in put}:
        want = sum(u[:, r] * v for k, r, v in put if k == m)
        got = y[mine, m].double()
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got[~got.isnan()], want[~want.isnan()]), m
    assert int((~y.isfinite()).sum()) == int(mine.sum()) * len({p[0] for p in put})


# ------------------------------------------------------------------------------ empty groups

@pytest.mark.parametrize("G,R,N,K", [(5, 300, 72, 136), (3, 4000, 520, 64)])
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
def test_accumulation_leaves_empty_groups_bit_for_bit(G, R, N, K, out):
    g, bits = gen(R), torch.int32 if out == "f32" else torch.int16
    x, dy = rand(g, "bf16", R, K), rand(g, "bf16", R, N)
    dw = torch.randint(-2 ** (31 if out == "f32" else 15), 2 ** (31 if out == "f32" else 15), (G, N, K), generator=g, device="cuda",
                       dtype=torch.int64).to(bits).view(ref.dtype(out))  # any bits: NaN, subnormal values and both zeros among them
    dw[:, 0] = -0.0
    o = [0, 0] + [R // 2] * (G - 2) + [R]
    dw[1] = dw[G - 1] = 0.25
    was = dw.clone()
    L.moe_grouped_weight_grad(x, L.MOE_BF16, R, K, None, 1, dy, R, N, None, torch.tensor(o, dtype=torch.int32, device="cuda"), G, R, N,
                              K, 1, dw, ref.code(out))
    torch.cuda.synchronize()
    for i in range(G):
        a, b = o[i], o[i + 1]
        if a == b:
            assert torch.equal(dw[i].view(bits), was[i].view(bits)), i
        else:
            v, e = ref.product(dy[a:b].T, x[a:b].T)
            ref.check(dw[i], v + 0.25, ref.rounded(v + 0.25, e + 2.0 ** -24 * ((v + 0.25).abs() + e), out), i)
