"""The 16-bit products whose rows choose their matrix where they could go wrong: values that are not finite beside other
requests' rows, indexes outside, more items than a table holds, captured and concurrent calls (GPU)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import grouped_reference as ref
from routed_expert_ffn_gemv_gb300 import _lib as L
from test_gpu_grouped import gen, lora, lora_bound, matmul, rand, uneven

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def status():
    L.moe_device_status(clear=True)
    yield
    torch.cuda.synchronize()
    assert L.moe_device_status(clear=True) == 0


# ------------------------------------------------------------------------------ values that are not finite

# few rows (8, 32), a matrix too large for that (split over a cluster), several narrow tiles, wide ones
LORA_PATHS = [(5, 64, 200), (30, 264, 128), (7, 5128, 72), (31, 6400, 64), (40, 136, 72), (300, 520, 64), (600, 128, 520),
              (600, 1032, 520), (40, 9736, 64)]


@pytest.mark.parametrize("T,N,K", LORA_PATHS)
@pytest.mark.parametrize("t,out", [("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_an_adapters_broken_weights_stay_with_its_tokens(T, N, K, t, out, value):
    """b, a or x with an infinity or a NaN: the outputs of no other token change, and of its own only those it reaches."""
    rng, g = np.random.default_rng(T), gen(T + N)
    n, rank = 5, 40
    adapter = rng.integers(-1, n, size=T).astype(np.int32)
    adapter[:5] = [0, 1, 2, 3, 4]
    x, w = rand(g, t, T, K), rand(g, t, N, K, scale=K ** -0.5)
    a, b = rand(g, t, n, rank, K, scale=K ** -0.5), rand(g, t, n, N, rank, scale=rank ** -0.5)
    rows = {1: sorted({0, 33, N - 1}), 3: [5]}  # broken outputs of two adapters
    for m in rows[1]:
        b[1, m, (7 * m) % rank] = value
    b[3, 5, 39] = value
    a[2, 3, K - 1] = value
    last = int((adapter == 0).nonzero()[0][-1])
    x[last, 1] = value
    y = lora(x, t, w, torch.from_numpy(adapter).cuda(), a, b, None, out)
    for i in range(-1, n):
        mine = [k for k in (adapter == i).nonzero()[0].tolist() if k != last]
        if not mine:
            continue
        idx = torch.tensor(mine, device="cuda")
        if i < 0:
            v, e = ref.product(x[idx], w)
            ref.check(y[idx], v, ref.rounded(v, e, out), i)
        elif i == 2:
            assert not bool(y[idx].isfinite().any())
        else:
            keep = torch.tensor([m for m in range(N) if m not in rows.get(i, [])], device="cuda")
            v, e = lora_bound(x[idx], t, w[keep], a[i], b[i][keep], 1.0, out)
            ref.check(y[idx][:, keep], v, e, i)
            if i in rows:
                assert not bool(y[idx][:, torch.tensor(rows[i], device="cuda")].isfinite().any())
    assert not bool(y[last].isfinite().any())


@pytest.mark.parametrize("T,N,K", LORA_PATHS)
def test_an_overflowing_inner_product_stays_with_its_token(T, N, K):
    g = gen(T)
    x, w = rand(g, "f16", T, K), rand(g, "f16", N, K)
    a, b = rand(g, "f16", 1, 8, K), rand(g, "f16", 1, N, 8)
    a[0, 2] = 60000.0 / K
    x[1] = 60.0  # u[2] = 3.6e6: past fp16
    x[torch.arange(T) != 1] *= 0.01
    y = lora(x, "f16", w, torch.zeros(T, dtype=torch.int32, device="cuda"), a, b, None, "f32")
    assert not bool(y[1].isfinite().any())
    rest = torch.arange(T, device="cuda") != 1
    v, e = lora_bound(x[rest], "f16", w, a[0], b[0], 1.0, "f32")
    ref.check(y[rest], v, e)


@pytest.mark.parametrize("order", [L.MOE_ORDER_NK, L.MOE_ORDER_KN])
@pytest.mark.parametrize("G,R", [(4, 6), (4, 40), (4, 300)])
def test_broken_rows_and_matrices_stay_in_their_group(order, G, R):
    g = gen(R)
    N, K = 72, 200
    x, w = rand(g, "bf16", R, K), rand(g, "bf16", G, N, K)
    o = [0, R // 3, R // 3 + 1, R - 2, R]
    x[o[1]] = float("nan")  # the one row of group 1
    w[3] = float("inf")
    stored = w if order == L.MOE_ORDER_NK else w.transpose(1, 2).contiguous()
    y = matmul(x, "bf16", torch.tensor(o, dtype=torch.int32, device="cuda"), stored, order, N, K, G=G, R=R)
    for i in (0, 2):
        v, e = ref.product(x[o[i]:o[i + 1]], w[i])
        ref.check(y[o[i]:o[i + 1]], v, ref.rounded(v, e, "f32"), i)
    assert bool(y[o[1]:o[2]].isnan().all()) and not bool(y[o[3]:].isfinite().any())


@pytest.mark.parametrize("T,n,rank,N,K", [(300, 5, 128, 2056, 64), (1030, 7, 32, 1160, 2048), (513, 200, 16, 2048, 200),
                                          (2000, 1, 256, 512, 64), (40, 3, 24, 12000, 72)])
@pytest.mark.parametrize("t,out", [("bf16", "f32"), ("f16", "f16"), ("bf16", "bf16")])
def test_lora_in_wide_tiles(T, n, rank, N, K, t, out):
    rng, g = np.random.default_rng(T + n), gen(T + rank)
    adapter = rng.integers(-1, n, size=T).astype(np.int32)
    x, w = rand(g, t, T, K), rand(g, t, N, K, scale=K ** -0.5)
    a, b = rand(g, t, n, rank, K, scale=K ** -0.5), rand(g, t, n, N, rank, scale=rank ** -0.5)
    scale = torch.randn(n, generator=g, device="cuda")
    y = lora(x, t, w, torch.from_numpy(adapter).cuda(), a, b, scale, out)
    for i in range(-1, n):
        mine = torch.from_numpy((adapter == i).nonzero()[0]).cuda()
        if mine.numel():
            if i < 0:
                v, e = ref.product(x[mine], w)
                e = ref.rounded(v, e, out)
            else:
                v, e = lora_bound(x[mine], t, w, a[i], b[i], float(scale[i]), out)
            ref.check(y[mine], v, e, i)


@pytest.mark.parametrize("T,N", [(6, 64), (30, 200), (40, 136), (31, 5128), (700, 1032)])
def test_lora_of_bf16_keeps_24_bits_for_fp32_results(T, N):
    """u's split adds no more than half a step of bf16 three times over."""
    rng, g = np.random.default_rng(T), gen(N)
    K, n, rank = 136, 3, 48
    adapter = rng.integers(0, n, size=T).astype(np.int32)
    x, w = rand(g, "bf16", T, K), rand(g, "bf16", N, K, scale=1e-3)
    a, b = rand(g, "bf16", n, rank, K), rand(g, "bf16", n, N, rank)
    y = lora(x, "bf16", w, torch.from_numpy(adapter).cuda(), a, b, None, "f32")
    for i in range(n):
        mine = torch.from_numpy((adapter == i).nonzero()[0]).cuda()
        v, _ = ref.product(x[mine], w)
        u, eu = ref.product(x[mine], a[i])
        eu = eu + ref.HALF["bf16"] ** 3 * (u.abs() + eu) + ref.TINY["bf16"]
        m = b[i].double()
        total = x[mine].double().abs() @ w.double().abs().T + (u.abs() + eu) @ m.abs().T
        e = ref.rounded(v + u @ m.T, eu @ m.abs().T + (K + 3 * rank + 16) * 2.0 ** -23 * total, "f32")
        ref.check(y[mine], v + u @ m.T, e, i)


# ------------------------------------------------------------------------------ indexes and offsets outside

@pytest.mark.parametrize("R,G", [(6, 3), (60, 4), (900, 4)])
def test_rows_outside_are_recorded_and_skipped(R, G):
    g = gen(R)
    N, K, share = 64, 72, 2
    x, w = rand(g, "f16", (R + 1) // 2, K), rand(g, "f16", G, N, K)
    offsets = torch.from_numpy(uneven(np.random.default_rng(R), G, R)).cuda()
    xi = torch.randperm(R, generator=g, device="cuda").int()
    yi = torch.randperm(R, generator=g, device="cuda").int()
    bad_x, bad_y = [0, R - 1], [2, R - 2]
    was = [int(yi[i]) for i in bad_x + bad_y]
    xi[bad_x[0]], xi[bad_x[1]] = -3, 2 * ((R + 1) // 2)
    yi[bad_y[0]], yi[bad_y[1]] = -1, R
    y = matmul(x, "f16", offsets, w, L.MOE_ORDER_NK, N, K, G=G, R=R, x_index=xi, share=share, y_index=yi)
    assert L.moe_device_status(clear=True) == L.MOE_ERR_INVALID
    assert bool((y[was] == 7.0).all())
    o = offsets.tolist()
    for i in range(G):
        p = [k for k in range(o[i], o[i + 1]) if k not in bad_x + bad_y]
        if p:
            v, e = ref.product(x[xi[p].long() // share], w[i])
            ref.check(y[yi[p].long()], v, ref.rounded(v, e, "f32"), i)


@pytest.mark.parametrize("R", [8, 64, 2000])
def test_offsets_that_are_no_range_are_recorded_and_skipped(R):
    g = gen(R)
    N, K = 64, 64
    x, w = rand(g, "bf16", R, K), rand(g, "bf16", 4, N, K)
    # group 1 descends, group 3 ends past R
    offsets = torch.tensor([0, 5, 3, R - 1, R + 5], dtype=torch.int32, device="cuda")
    y = matmul(x, "bf16", offsets, w, L.MOE_ORDER_NK, N, K, G=4, R=R)
    assert L.moe_device_status(clear=True) == L.MOE_ERR_INVALID
    v0, e0 = ref.product(x[:5], w[0])
    v2, e2 = ref.product(x[3:R - 1], w[2])
    ref.check(y[:3], v0[:3], ref.rounded(v0, e0, "f32")[:3])
    ref.check(y[5:R - 1], v2[2:], ref.rounded(v2, e2, "f32")[2:])
    assert bool((y[R - 1] == 7.0).all())


@pytest.mark.parametrize("T,N", [(3, 32), (30, 64), (30, 5128), (900, 1032)])
def test_adapters_outside_are_recorded_and_left_out(T, N):
    g = gen(T)
    K = 72
    x, w = rand(g, "f16", T, K), rand(g, "f16", N, K)
    a, b = rand(g, "f16", 2, 16, K), rand(g, "f16", 2, N, 16)
    adapter = torch.full((T,), 1, dtype=torch.int32, device="cuda")
    adapter[0], adapter[T - 1] = 2, -2
    y = lora(x, "f16", w, adapter, a, b, None, "f32")
    assert L.moe_device_status(clear=True) == L.MOE_ERR_INVALID
    v, e = ref.product(x, w)
    ref.check(y[[0, T - 1]], v[[0, T - 1]], ref.rounded(v, e, "f32")[[0, T - 1]])
    v, e = lora_bound(x[1:T - 1], "f16", w, a[1], b[1], 1.0, "f32")
    ref.check(y[1:T - 1], v, e)


def test_gradient_of_rows_outside():
    g = gen(4)
    R, N, K = 150, 128, 64
    x, dy = rand(g, "bf16", R, K), rand(g, "bf16", R, N)
    perm = torch.randperm(R, generator=g, device="cuda").int()
    xi, yi = perm.clone(), perm.clone()
    xi[3], xi[90], yi[70], yi[149] = R, -1, -9, R + 7
    offsets = torch.tensor([0, 64, 64, R], dtype=torch.int32, device="cuda")
    dw = torch.empty(3, N, K, device="cuda")
    L.moe_grouped_weight_grad(x, L.MOE_BF16, R, K, xi, 1, dy, R, N, yi, offsets, 3, R, N, K, 0, dw, L.MOE_F32)
    torch.cuda.synchronize()
    assert L.moe_device_status(clear=True) == L.MOE_ERR_INVALID
    for i, (a, b) in ((0, (0, 64)), (2, (64, R))):
        p = [k for k in range(a, b) if k not in (3, 90, 70, 149)]
        v, e = ref.product(dy[perm[p].long()].T, x[perm[p].long()].T)
        ref.check(dw[i], v, ref.rounded(v, e, "f32"), i)
    assert bool((dw[1] == 0).all())


# ------------------------------------------------------------------------------ sizes

# few rows, narrow tiles, pairs; reductions of one accumulator and of several
@pytest.mark.parametrize("G,R,N,K", [(2, 3, 72, 136), (1, 8, 4096, 2048), (8, 60, 264, 2040), (4, 300, 136, 72), (3, 700, 200, 1024),
                                     (2, 900, 72, 2048), (2, 500, 8, 4104)])
@pytest.mark.parametrize("t,out", [("bf16", "f32"), ("f16", "f32"), ("f16", "bf16")])
def test_swiglu_with_results_of_another_type(G, R, N, K, t, out):
    rng, g = np.random.default_rng(R), gen(K)
    offsets = uneven(rng, G, R)
    x, w = rand(g, t, R, K), rand(g, t, G, 2 * N, K, scale=K ** -0.5)
    scale = torch.randn(R, generator=g, device="cuda")
    y = matmul(x, t, torch.from_numpy(offsets).cuda(), w, L.MOE_ORDER_NK, N, K, G=G, R=R, act=L.MOE_ACT_SWIGLU, scale=scale,
               out=out)
    for i in range(G):
        a, b = offsets[i], offsets[i + 1]
        if b > a:
            p, e = ref.product(x[a:b], w[i])
            h, eh = ref.swiglu(p[:, :N], e[:, :N], p[:, N:], e[:, N:])
            s = scale[a:b, None].double()
            ref.check(y[a:b], h * s, ref.rounded(h * s, eh * s.abs() + 2.0 ** -24 * (h * s).abs(), out), i)


@pytest.mark.parametrize("G,R,N,K", [(64, 1100, 32768, 16), (512, 512, 4096, 8)])
def test_more_items_than_a_ctas_table(G, R, N, K):
    rng, g = np.random.default_rng(G), gen(G)
    offsets = uneven(rng, G, R)
    x, w = rand(g, "f16", R, K), rand(g, "f16", G, N, K)
    y = matmul(x, "f16", torch.from_numpy(offsets).cuda(), w, L.MOE_ORDER_NK, N, K, G=G, R=R, out="f16")
    for i in range(G):
        a, b = offsets[i], offsets[i + 1]
        if b > a:
            v, e = ref.product(x[a:b], w[i])
            ref.check(y[a:b], v, ref.rounded(v, e, "f16"), i)


def test_gradient_with_more_items_than_a_ctas_table():
    g = gen(9)
    G, R, N, K = 512, 700, 1024, 1024
    offsets = uneven(np.random.default_rng(9), G, R)
    x, dy = rand(g, "f16", R, K), rand(g, "f16", R, N)
    dw = torch.full((G, N, K), float("nan"), dtype=torch.float16, device="cuda")
    L.moe_grouped_weight_grad(x, L.MOE_F16, R, K, None, 1, dy, R, N, None, torch.from_numpy(offsets).cuda(), G, R, N, K, 0, dw,
                              L.MOE_F16)
    torch.cuda.synchronize()
    for i in range(G):
        a, b = offsets[i], offsets[i + 1]
        if a == b:
            assert bool((dw[i] == 0).all())
        else:
            v, e = ref.product(dy[a:b].T, x[a:b].T)
            ref.check(dw[i], v, ref.rounded(v, e, "f16"), i)


def test_rows_past_2_31_elements():
    """A row's offset in a buffer of more than 2^31 elements, in x and in y."""
    g = gen(11)
    rows, ld, N, K = 33000, 65536, 64, 64
    x = torch.zeros(rows, ld, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(rows, ld, dtype=torch.bfloat16, device="cuda")
    pick = torch.tensor([0, 7, rows - 1, rows - 2] + list(range(100, 400)), dtype=torch.int32, device="cuda")
    R = pick.numel()
    x[pick.long(), :K] = rand(g, "bf16", R, K)
    w = rand(g, "bf16", 1, N, K)
    for n in (4, R):
        offsets = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        L.moe_grouped_matmul(x, L.MOE_BF16, rows, ld, pick, 1, offsets, 1, n, w, L.MOE_ORDER_NK, N, K, L.MOE_ACT_NONE, None,
                             pick, y, L.MOE_BF16, rows, ld)
        torch.cuda.synchronize()
        v, e = ref.product(x[pick[:n].long(), :K], w[0])
        ref.check(y[pick[:n].long(), :N], v, ref.rounded(v, e, "bf16"))
        y.zero_()


# ------------------------------------------------------------------------------ order, streams, graphs

def layer_calls(T, k, E, H, F, seed):
    """A routed layer's calls on its own buffers, and what they have to leave."""
    rng, g = np.random.default_rng(seed), gen(seed)
    R = T * k
    s = {"x": rand(g, "bf16", T, H), "w1": rand(g, "bf16", E, 2 * F, H, scale=H ** -0.5),
         "w2": rand(g, "bf16", E, H, F, scale=F ** -0.5),
         "ids": torch.from_numpy(rng.integers(0, E, size=(T, k)).astype(np.int32)).cuda(),
         "weights": torch.rand(T, k, generator=g, device="cuda"),
         "offsets": torch.zeros(E + 1, dtype=torch.int32, device="cuda"), "rows": torch.zeros(R, dtype=torch.int32, device="cuda"),
         "h": torch.zeros(R, F, dtype=torch.bfloat16, device="cuda"), "partial": torch.zeros(T, k, H, device="cuda"),
         "y": torch.zeros(T, H, device="cuda"), "dw": torch.zeros(E, H, F, device="cuda"),
         "a": rand(g, "bf16", 3, 16, H, scale=H ** -0.5), "b": rand(g, "bf16", 3, H, 16, scale=0.25),
         "adapter": torch.from_numpy(rng.integers(-1, 3, size=T).astype(np.int32)).cuda(), "ws0": rand(g, "bf16", H, H, scale=H ** -0.5),
         "z": torch.zeros(T, H, device="cuda")}
    s["ws"] = torch.empty(max(1, L.moe_lora_workspace(T, 16)), dtype=torch.uint8, device="cuda")
    s["gw"] = torch.empty(max(1, L.moe_group_rows_workspace(R, E)), dtype=torch.uint8, device="cuda")

    def call(stream=None):
        L.moe_group_rows(s["ids"], R, E, s["offsets"], s["rows"], s["gw"], s["gw"].numel(), stream)
        L.moe_grouped_matmul(s["x"], 1, T, H, s["rows"], k, s["offsets"], E, R, s["w1"], 0, F, H, 1, None, None, s["h"], 1, R, F,
                             stream)
        L.moe_grouped_matmul(s["h"], 1, R, F, None, 1, s["offsets"], E, R, s["w2"], 0, H, F, 0, s["weights"], s["rows"],
                             s["partial"], 0, R, H, stream)
        L.moe_combine(s["partial"], T, k, H, None, s["y"], stream)
        L.moe_grouped_weight_grad(s["h"], 1, R, F, None, 1, s["ws0"][:1].expand(1, H), 1, H, s["zero"], s["offsets"], E, R, H, F, 0,
                                  s["dw"], 0, stream)
        L.moe_lora_matmul(s["x"], 1, T, H, s["ws0"], H, H, s["adapter"], 3, s["a"], s["b"], 16, None, s["z"], 0, H, s["ws"],
                          s["ws"].numel(), stream)

    s["zero"] = torch.zeros(R, dtype=torch.int32, device="cuda")
    outs = ("offsets", "rows", "h", "partial", "y", "dw", "z")

    def wipe():
        for n in outs:
            s[n].zero_()

    call()
    torch.cuda.synchronize()
    want = {n: s[n].clone() for n in outs}
    return call, wipe, lambda: all(torch.equal(s[n], want[n]) for n in outs), s


@pytest.mark.parametrize("T,k,E,H,F", [(1, 4, 8, 256, 64), (20, 2, 8, 128, 72), (700, 4, 8, 256, 128)])
def test_the_same_bits_again_captured_and_on_two_streams(T, k, E, H, F):
    """Calls on the same inputs leave the same bits: again, replayed from a graph, and beside another set of calls on another
    stream (each with workspaces of its own)."""
    one, two = layer_calls(T, k, E, H, F, 1), layer_calls(T + 3, k, E, H, F, 2)
    for call, wipe, same, _ in (one, two):
        for _ in range(3):
            wipe()
            call()
            torch.cuda.synchronize()
            assert same()
    graphs = []
    for call, wipe, same, _ in (one, two):
        gr, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(gr, stream=side):
            call()
        graphs.append(gr)
        for _ in range(3):
            wipe()
            gr.replay()
            torch.cuda.synchronize()
            assert same()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _, wipe, _, _ in (one, two):
        wipe()
    torch.cuda.synchronize()
    for _ in range(5):
        for (call, _, _, _), st in zip((one, two), streams):
            call(st)
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    assert one[2]() and two[2]()


def test_inputs_of_the_kernel_before():
    """The calls read what the stream's previous kernel wrote: indexes, offsets, adapters, matrices, rows."""
    call, wipe, same, s = layer_calls(24, 2, 8, 128, 64, 5)
    inputs = ("x", "w1", "w2", "ids", "weights", "a", "b", "adapter", "ws0")
    kept = {n: s[n].clone() for n in inputs}
    for _ in range(10):
        for n in inputs:  # (other values first, which an early read would find)
            s[n].fill_(-1 if s[n].dtype == torch.int32 else 3.0)
        wipe()
        torch.cuda.synchronize()
        for n in inputs:
            s[n].copy_(kept[n])
        call()
        torch.cuda.synchronize()
        assert same()


# ------------------------------------------------------------------------------ gradients against differences

def test_input_and_weight_gradients_against_differences():
    """The loss sum(y * c) of a product y = x W^T by groups: its two gradients against differences of the plain 64-bit loss.
    It is linear in each input: a central difference in 64 bits is exact to rounding."""
    g = gen(21)
    G, R, N, K = 3, 40, 48, 56
    o = [0, 11, 11, 40]
    offsets = torch.tensor(o, dtype=torch.int32, device="cuda")
    x, w, c = rand(g, "bf16", R, K), rand(g, "bf16", G, N, K), rand(g, "bf16", R, N)
    dx, dw = torch.empty(R, K, device="cuda"), torch.empty(G, N, K, device="cuda")
    L.moe_grouped_matmul(c, 1, R, N, None, 1, offsets, G, R, w, L.MOE_ORDER_KN, K, N, 0, None, None, dx, 0, R, K)
    L.moe_grouped_weight_grad(x, 1, R, K, None, 1, c, R, N, None, offsets, G, R, N, K, 0, dw, 0)
    torch.cuda.synchronize()

    def loss(x, w):
        return sum(float((x[o[i]:o[i + 1]] @ w[i].T * c[o[i]:o[i + 1]].double()).sum()) for i in range(G))

    rng = np.random.default_rng(3)
    for _ in range(20):
        r, k, n, i = rng.integers(R), rng.integers(K), rng.integers(N), rng.integers(G)
        lx, hx, lw, hw = x.double(), x.double(), w.double(), w.double()
        lx[r, k] -= 1
        hx[r, k] += 1
        lw[i, n, k] -= 1
        hw[i, n, k] += 1
        wd, xd = w.double(), x.double()
        # bounds: 64-bit rounding of a loss of about 1e3, and the fp32 sums of at most 48 products of size under 25
        assert abs((loss(hx, wd) - loss(lx, wd)) / 2 - float(dx[r, k])) <= 1e-9 + (N + 16) * 2.0 ** -23 * 25 * N
        assert abs((loss(xd, hw) - loss(xd, lw)) / 2 - float(dw[i, n, k])) <= 1e-9 + (R + 16) * 2.0 ** -23 * 25 * R
