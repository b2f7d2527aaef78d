"""The 16-bit products whose rows choose their matrix at their limits: offsets whose ranges overlap, infinite weights of
adapters, empty groups, long reductions, small values of fp16 (GPU)."""
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


# ------------------------------------------------------------------------------ long reductions

# Relative to the results' norm.  A step of 16 in an MMA drops less than a unit of the sum so far, half of one on average: between
# 2^-25 and 2^-24 of the sum, 0.72 2^-24 on average, and a sum of independent terms is on its way two thirds of what it ends
# at.  32 steps: 32 * 0.72 * 2^-24 * 2 / 3 = 0.92e-6, if every loss pointed the same way.  Sums of accumulators, rounded to nearest,
# add 1.4e-8 sqrt(their number): 0.2e-6 for 256 of them, in quadrature.
FP32_SUMS = 1e-6


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def product_off(g, G, R, N, K, t="bf16", out="f32", order=L.MOE_ORDER_NK, act=L.MOE_ACT_NONE):
    """How far a product of equal groups is off, and how far the exact one would be once rounded."""
    x, w = rand(g, t, R, K), rand(g, t, G, 2 * N if act else N, K, scale=K ** -0.5)
    o = [i * R // G for i in range(G + 1)]
    y = matmul(x, t, torch.tensor(o, dtype=torch.int32, device="cuda"), w if order == L.MOE_ORDER_NK else w.transpose(1, 2).contiguous(),
               order, N, K, G=G, R=R, act=act, out=out)
    want = torch.cat([x[a:b].double() @ w[i].double().T for i, (a, b) in enumerate(zip(o, o[1:]))])
    if act:
        want = want[:, :N] * torch.sigmoid(want[:, :N]) * want[:, N:]
    return off(y, want), off(want.to(y.dtype), want)


# few rows, a matrix too large for that, narrow tiles that share their reduction, narrow tiles, pairs
@pytest.mark.parametrize("G,R,N", [(1, 4, 64), (1, 8, 6400), (4, 40, 256), (16, 200, 1280), (2, 512, 256)])
@pytest.mark.parametrize("K", [1024, 1032, 2048, 8192, 65536])
@pytest.mark.parametrize("form", ["nk", "kn", "swiglu"])
def test_fp32_sums_do_not_lose_with_the_reduction(G, R, N, K, form):
    if N * K * G > 2 ** 29:
        N = 2 ** 26 // K
    e, _ = product_off(gen(K), G, R, N, K, order=L.MOE_ORDER_KN if form == "kn" else L.MOE_ORDER_NK,
                       act=L.MOE_ACT_SWIGLU if form == "swiglu" else L.MOE_ACT_NONE)
    assert e <= FP32_SUMS


@pytest.mark.parametrize("G,R,N", [(1, 4, 64), (4, 40, 256), (2, 512, 256)])
@pytest.mark.parametrize("K", [2048, 65536])
@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("act", [L.MOE_ACT_NONE, L.MOE_ACT_SWIGLU])
def test_16_bit_results_of_long_reductions(G, R, N, K, t, act):
    """What the sums lose (at most 2e-5) is not seen beside the rounding (fp16: 2e-4), in quadrature one percent of it."""
    e, least = product_off(gen(K), G, R, N, K, t=t, out=t, act=act)
    assert e <= 1.01 * least


def gradient_off(g, o, N, K, out, accumulate=False):
    G, R = len(o) - 1, o[-1]
    x, dy = rand(g, "f16", R, K), rand(g, "f16", R, N, scale=max(b - a for a, b in zip(o, o[1:])) ** -0.5)
    dw = torch.zeros(G, N, K, dtype=ref.dtype(out), device="cuda")
    L.moe_grouped_weight_grad(x, L.MOE_F16, R, K, None, 1, dy, R, N, None, torch.tensor(o, dtype=torch.int32, device="cuda"), G, R, N, K,
                              accumulate, dw, ref.code(out))
    torch.cuda.synchronize()
    want = torch.stack([dy[a:b].double().T @ x[a:b].double() for a, b in zip(o, o[1:])])
    return off(dw, want), off(want.to(dw.dtype), want)


@pytest.mark.parametrize("accumulate", [0, 1])
@pytest.mark.parametrize("o", [[0, 300, 700], [0, 65536], [0] + [32768 + i for i in range(128)], [0, 100, 4000, 4100] + [4100] * 30])
def test_gradients_of_long_groups(o, accumulate):
    """One group, and one of many rows among others that have few."""
    assert gradient_off(gen(len(o)), o, 200, 264, "f32", accumulate)[0] <= FP32_SUMS


@pytest.mark.parametrize("out", ["bf16", "f16"])
def test_16_bit_gradient_of_a_long_group(out):
    e, least = gradient_off(gen(1), [0, 1 << 20], 64, 64, out)
    assert e <= 1.01 * least


# few rows, narrow tiles, pairs; more tokens than the kernel of u shares K for
@pytest.mark.parametrize("T,N,K", [(5, 64, 2048), (30, 264, 65536), (7, 6400, 8192), (50, 264, 2048), (300, 264, 65536), (600, 1032, 2048),
                                   (600, 1032, 65536), (20000, 128, 2048), (20000, 128, 8192)])
@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("rank", [64, 256])
@pytest.mark.parametrize("alone", [True, False])
def test_fp32_sums_of_adapters(T, N, K, t, rank, alone):
    """alone: the shared projection is zero, so that u's own sums show."""
    g, n = gen(T + K), 3
    x, w = rand(g, t, T, K), rand(g, t, N, K, scale=0.0 if alone else K ** -0.5)
    a, b = rand(g, t, n, rank, K, scale=K ** -0.5), rand(g, t, n, N, rank, scale=rank ** -0.5)
    adapter = torch.randint(0, n, (T,), generator=g, device="cuda").int()
    y = lora(x, t, w, adapter, a, b, None, "f32")
    want = x.double() @ w.double().T
    for i in range(n):
        m = adapter == i
        want[m] += x[m].double() @ a[i].double().T @ b[i].double().T
    assert off(y, want) <= FP32_SUMS


# ------------------------------------------------------------------------------ fp16's range between the adapter's two matrices

def adapters_off(g, T, N, K, rank, out, xs=1.0, scale=None, bs=1.0, spread=0):
    """fp16 adapters alone (the shared projection is zero).  spread: a's ranks and the tokens differ in size by powers of two."""
    n = 3
    x, w = rand(g, "f16", T, K, scale=xs), torch.zeros(N, K, dtype=torch.float16, device="cuda")
    a, b = rand(g, "f16", n, rank, K, scale=K ** -0.5), rand(g, "f16", n, N, rank, scale=bs * rank ** -0.5)
    if spread:
        x *= 2.0 ** -(torch.arange(T, device="cuda") % 5)[:, None].half()
        p = 2.0 ** -(torch.arange(rank, device="cuda") * spread // rank).half()  # ranks from 1 to 2^-spread, weighed back by b
        a, b = a * p[:, None], b / p
        assert bool(b.isfinite().all())
    adapter = torch.arange(T, device="cuda").int() % (n + 1) - 1
    d_scale = None if scale is None else torch.full((n,), scale, device="cuda")
    y = lora(x, "f16", w, adapter, a.contiguous(), b.contiguous(), d_scale, out)
    want = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    for i in range(n):
        m = adapter == i
        want[m] = (scale or 1.0) * (x[m].double() @ a[i].double().T) @ b[i].double().T
    assert bool((y[adapter < 0] == 0).all())
    rows = want.norm(dim=1).clamp_min(1e-300)  # every token by its own size
    return off(y / rows[:, None], want / rows[:, None]), off(want.to(y.dtype) / rows[:, None], want / rows[:, None])


FP16_PATHS = [(5, 64, 200), (30, 264, 2048), (7, 6400, 128), (31, 5128, 72), (50, 264, 2048), (300, 264, 520), (600, 1032, 2048),
              (20000, 128, 2048)]


@pytest.mark.parametrize("T,N,K", FP16_PATHS)
@pytest.mark.parametrize("rank", [24, 64, 256])
@pytest.mark.parametrize("xs,scale,bs", [(1.0, None, 1.0), (2.0 ** -7, None, 1.0), (2.0 ** -12, 8.0, 64.0), (1.0, 2.0 ** -12, 2.0 ** 10),
                                         (1.0, 1e-20, 1.0), (8.0, 2.0 ** 9, 2.0 ** -4)])
def test_fp16_adapters_keep_their_bits_at_every_size(T, N, K, rank, xs, scale, bs):
    """u from 1e-20 to thousands: 22 bits (2^-23 of a value at most, a fifth of the sums' allowance) and the sums."""
    assert adapters_off(gen(T + rank), T, N, K, rank, "f32", xs, scale, bs)[0] <= FP32_SUMS


@pytest.mark.parametrize("T,N,K", FP16_PATHS)
@pytest.mark.parametrize("rank", [24, 64, 256])
@pytest.mark.parametrize("spread", [6, 10])
def test_fp16_adapters_of_ranks_of_many_sizes(T, N, K, rank, spread):
    """Ranks whose u differs by 2^10 and counts alike, tokens that differ by 2^4."""
    assert adapters_off(gen(T + rank), T, N, K, rank, "f32", spread=spread)[0] <= FP32_SUMS


@pytest.mark.parametrize("T,N,K", FP16_PATHS)
@pytest.mark.parametrize("empty", [[0], [1], [0, 2]])
@pytest.mark.parametrize("out", ["f32", "f16"])
def test_fp16_adapters_with_ranks_of_zeros(T, N, K, empty, out):
    """Adapters of a smaller rank than the table's: 32 ranks of zeros say nothing about the size of the others."""
    g, n, rank = gen(T), 3, 96
    x, w = rand(g, "f16", T, K, scale=2.0 ** -9), torch.zeros(N, K, dtype=torch.float16, device="cuda")
    a, b = rand(g, "f16", n, rank, K, scale=K ** -0.5), rand(g, "f16", n, N, rank, scale=2.0 ** 9 * rank ** -0.5)
    for c in empty:
        a[1:, 32 * c:32 * c + 32] = 0.0
    adapter = torch.arange(T, device="cuda").int() % n
    d_scale = torch.tensor([1.0, 2.0 ** -8, 1.0], device="cuda")
    y = lora(x, "f16", w, adapter, a, b, d_scale, out)
    want = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    for i in range(n):
        m = adapter == i
        want[m] = float(d_scale[i]) * (x[m].double() @ a[i].double().T) @ b[i].double().T
    rows = want.norm(dim=1, keepdim=True)
    e, least = off(y / rows, want / rows), off(want.to(y.dtype) / rows, want / rows)
    assert e <= (FP32_SUMS if out == "f32" else 1.01 * least)


@pytest.mark.parametrize("T,N,K", FP16_PATHS)
@pytest.mark.parametrize("rank", [24, 256])
@pytest.mark.parametrize("out", ["f16", "bf16"])
@pytest.mark.parametrize("scale,bs,spread", [(2.0 ** -12, 2.0 ** 10, 0), (None, 1.0, 0), (0.25, 1.0, 10), (2.0 ** -9, 1.0, 10)])
def test_fp16_adapters_small_between_the_matrices_of_16_bit_results(T, N, K, rank, out, scale, bs, spread):
    """The sums' 6e-6 (u of long reductions: as much) are not seen beside the rounding (2e-4), nor is what u's smaller ranks lose beside
    a largest one of 1/8 or more: 2^-25 each at most, 1.7e-8 on average, weighed back by 1 to 2^9, 187 on average: 3.2e-6 over the
    size of u's first ranks, which is 1/4, 1/8 or 1/16 for three tokens in five (the others come by a power of two): 2.7e-5 on
    average over the tokens, in quadrature 0.9 percent of the rounding."""
    e, least = adapters_off(gen(T + rank), T, N, K, rank, out, 1.0, scale, bs, spread)
    assert e <= 1.01 * least


# ------------------------------------------------------------------------------ together

@pytest.mark.parametrize("T,N,K", [(20, 64, 16384), (40, 136, 16384), (600, 1032, 16392), (600, 520, 40000)])
@pytest.mark.parametrize("t,out", [("f16", "f16"), ("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("scale", [None, 2.0 ** -12])
def test_adapters_of_long_reductions_beside_their_projection(T, N, K, t, out, scale):
    """More than one accumulator for the projection, with and without the adapters' own, and tokens of zeros."""
    g, n, rank = gen(T), 3, 72
    x, w = rand(g, t, T, K), rand(g, t, N, K, scale=K ** -0.5)
    x[::7] = 0.0
    a, b = rand(g, t, n, rank, K, scale=K ** -0.5), rand(g, t, n, N, rank, scale=rank ** -0.5 / (scale or 1.0) / 8)
    adapter = torch.arange(T, device="cuda").int() % (n + 1) - 1
    y = lora(x, t, w, adapter, a, b, None if scale is None else torch.full((n,), scale, device="cuda"), out)
    want = x.double() @ w.double().T
    for i in range(n):
        m = adapter == i
        want[m] += (scale or 1.0) * (x[m].double() @ a[i].double().T) @ b[i].double().T
    assert bool((y[::7] == 0).all())
    e, least = off(y, want), off(want.to(y.dtype), want)
    assert e <= (FP32_SUMS if out == "f32" else 1.01 * least)


@pytest.mark.parametrize("T,N,K,rank", [(1, 64, 128, 16), (30, 264, 256, 64), (50, 264, 128, 64), (700, 520, 256, 48)])
@pytest.mark.parametrize("out", ["f16", "f32"])
def test_fp16_adapters_captured_and_on_two_streams(T, N, K, rank, out):
    """The same bits again, replayed, and beside another call on another stream, of large and of small u."""
    calls = []
    for seed, xs in ((1, 1.0), (2, 2.0 ** -9)):
        g, n = gen(seed), 3
        x, w = rand(g, "f16", T, K, scale=xs), rand(g, "f16", N, K, scale=K ** -0.5)
        a, b = rand(g, "f16", n, rank, K, scale=K ** -0.5), rand(g, "f16", n, N, rank, scale=rank ** -0.5)
        adapter = torch.randint(-1, n, (T,), generator=g, device="cuda").int()
        y, ws = torch.zeros(T, N, dtype=ref.dtype(out), device="cuda"), torch.empty(L.moe_lora_workspace(T, rank), dtype=torch.uint8,
                                                                                 device="cuda")

        def call(stream=None, v=(x, w, adapter, a, b, y, ws)):
            x, w, adapter, a, b, y, ws = v
            L.moe_lora_matmul(x, L.MOE_F16, T, K, w, N, K, adapter, 3, a, b, rank, None, y, ref.code(out), N, ws, ws.numel(), stream)

        call()
        torch.cuda.synchronize()
        want = y.clone()
        gr, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(gr, stream=side):
            call()
        for _ in range(3):
            y.zero_()
            ws.fill_(0xFF)
            gr.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want)
        calls.append((call, gr, y, want, torch.cuda.Stream()))
    for _, _, y, _, _ in calls:
        y.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for call, gr, _, _, st in calls:
            call(st)
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for _, _, y, want, _ in calls)


def test_long_groups_captured_and_on_two_streams():
    """Accumulators that are folded on the way: the same bits again, replayed and beside another call."""
    g, o = gen(4), [0, 20000, 20010, 20010, 41000]
    G, R, N, K = 4, 41000, 264, 136
    x, dy, w = rand(g, "bf16", R, K), rand(g, "bf16", R, N), rand(g, "bf16", G, K, N, scale=N ** -0.5)
    xl, wl = rand(g, "bf16", 300, 8200), rand(g, "bf16", G, N, 8200, scale=8200 ** -0.5)
    d_off, l_off = torch.tensor(o, dtype=torch.int32, device="cuda"), torch.tensor([0, 100, 101, 101, 300], dtype=torch.int32, device="cuda")
    outs = [torch.zeros(G, N, K, device="cuda"), torch.zeros(G, N, K, dtype=torch.bfloat16, device="cuda"), torch.zeros(300, N, device="cuda"),
            torch.zeros(300, N // 2 // 8 * 8, device="cuda")]
    grads = [lambda s=None: L.moe_grouped_weight_grad(x, 1, R, K, None, 1, dy, R, N, None, d_off, G, R, N, K, 0, outs[0], 0, s),
             lambda s=None: L.moe_grouped_weight_grad(x, 1, R, K, None, 1, dy, R, N, None, d_off, G, R, N, K, 0, outs[1], 1, s)]
    products = [lambda s=None: L.moe_grouped_matmul(xl, 1, 300, 8200, None, 1, l_off, G, 300, wl, 0, N, 8200, 0, None, None, outs[2], 0, 300, N, s),
                lambda s=None: L.moe_grouped_matmul(xl, 1, 300, 8200, None, 1, l_off, G, 300, wl, 0, N // 2 // 8 * 8, 8200, 1, None, None, outs[3],
                                                    0, 300, N // 2 // 8 * 8, s)]
    for f in grads + products:
        f()
    torch.cuda.synchronize()
    want = [v.clone() for v in outs]
    gr, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(gr, stream=side):
        for f in products:
            f()
    for v in outs:
        v.zero_()
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        for f in grads:
            f(one)
        with torch.cuda.stream(two):
            gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
