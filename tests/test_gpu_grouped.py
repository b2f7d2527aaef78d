"""The 16-bit products whose rows choose their matrix, against plain 64-bit forms (GPU)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import grouped_reference as ref
from routed_expert_ffn_gemv_gb300 import _lib as L

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def status():
    L.moe_device_status(clear=True)
    yield
    torch.cuda.synchronize()
    assert L.moe_device_status(clear=True) == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rand(g, t, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(ref.dtype(t))


# ------------------------------------------------------------------------------ groups

def group_rows(ids, G):
    n = ids.numel()
    offsets = torch.full((G + 1,), -7, dtype=torch.int32, device="cuda")
    rows = torch.full((n + 3,), -7, dtype=torch.int32, device="cuda")
    size = L.moe_group_rows_workspace(n, G)
    ws = torch.full((size + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    L.moe_group_rows(ids, n, G, offsets, rows, ws, size)
    torch.cuda.synchronize()
    assert rows[n:].tolist() == [-7] * 3 and bool((ws[size:] == 0x5A).all())
    return offsets.cpu().numpy(), rows[:n].cpu().numpy()


@pytest.mark.parametrize("n,G", [(0, 5), (1, 1), (8, 128), (31, 3), (33, 512), (1000, 7), (4096, 128), (4097, 32),
                                 (8193, 500), (32768, 128), (100001, 64), (131072, 1), (131073, 128), (300000, 511)])
def test_group_rows(n, G):
    rng = np.random.default_rng(n + G)
    # uneven groups, some empty, one id in ten without a group
    ids = np.minimum(rng.exponential(G / 6, size=n).astype(np.int32), G - 1)
    ids[rng.random(n) < 0.1] = -1
    offsets, rows = group_rows(torch.from_numpy(ids).cuda(), G)
    key = np.where(ids < 0, G, ids)
    order = np.argsort(key, kind="stable")
    count = np.bincount(key, minlength=G + 1)
    assert np.array_equal(offsets, np.concatenate(([0], np.cumsum(count[:G]))))
    total = offsets[-1]
    assert np.array_equal(rows[:total], order[:total]) and (rows[total:] == -1).all()
    if n <= 4097:
        o, r = ref.group(ids, G)
        assert np.array_equal(offsets, o) and np.array_equal(rows, r)


@pytest.mark.parametrize("n", [40, 9000, 140000])
@pytest.mark.parametrize("one", [True, False])
def test_group_rows_of_one_group_or_none(n, one):
    offsets, rows = group_rows(torch.full((n,), 3 if one else -1, dtype=torch.int32, device="cuda"), 6)
    assert offsets.tolist() == ([0] * 4 + [n] * 3 if one else [0] * 7)
    assert np.array_equal(rows, np.arange(n) if one else np.full(n, -1))


@pytest.mark.parametrize("n", [40, 140000])
def test_group_rows_reports_ids_outside(n):
    ids = torch.full((n,), 1, dtype=torch.int32, device="cuda")
    ids[5], ids[17] = 2, -2
    offsets, rows = group_rows(ids, 2)
    assert L.moe_device_status(clear=True) == L.MOE_ERR_INVALID
    assert offsets.tolist() == [0, 0, n - 2]
    assert np.array_equal(rows[:n - 2], [i for i in range(n) if i not in (5, 17)]) and (rows[n - 2:] == -1).all()


# ------------------------------------------------------------------------------ products

def matmul(x, t, offsets, w, order, N, K, *, G, R, act=L.MOE_ACT_NONE, x_index=None, share=1, scale=None, y_index=None,
           out="f32", y_rows=None, pad=8):
    """The call on rows of a wider y, whose other rows and columns have to stay."""
    y_rows = R if y_rows is None else y_rows
    y = torch.full((y_rows + 2, N + pad), 7.0, dtype=ref.dtype(out), device="cuda")
    L.moe_grouped_matmul(x, ref.code(t), x.shape[0], x.stride(0), x_index, share, offsets, G, R, w, order, N, K, act, scale,
                         y_index, y, ref.code(out), y_rows, N + pad)
    torch.cuda.synchronize()
    assert bool((y[:, N:] == 7.0).all()) and bool((y[y_rows:] == 7.0).all())
    return y[:y_rows, :N]


def uneven(rng, G, R):
    """Group sizes that sum to R, some of them 0."""
    cuts = np.sort(rng.integers(0, R + 1, size=G - 1)) if G > 1 else np.array([], np.int64)
    return np.concatenate(([0], cuts, [R])).astype(np.int32)


SHAPES = [  # G, R, N, K
    (1, 1, 8, 8), (1, 5, 136, 72), (4, 3, 256, 128), (8, 40, 64, 200), (3, 700, 264, 520), (128, 8, 512, 2048),
    (32, 152, 1024, 512), (5, 1024, 128, 64), (2, 1500, 2048, 1000), (64, 2048, 1408, 256), (7, 513, 24, 2040),
    (500, 499, 40, 48), (512, 17000, 16, 16),
]


@pytest.mark.parametrize("G,R,N,K", SHAPES)
@pytest.mark.parametrize("order", [L.MOE_ORDER_NK, L.MOE_ORDER_KN])
@pytest.mark.parametrize("t,out", [("bf16", "f32"), ("f16", "f16"), ("bf16", "bf16")])
def test_products_of_contiguous_groups(G, R, N, K, order, t, out):
    rng, g = np.random.default_rng(R + N), gen(G + K)
    offsets = uneven(rng, G, R)
    x, w = rand(g, t, R, K), rand(g, t, G, N, K, scale=K ** -0.5)
    stored = w if order == L.MOE_ORDER_NK else w.transpose(1, 2).contiguous()
    y = matmul(x, t, torch.from_numpy(offsets).cuda(), stored, order, N, K, G=G, R=R, out=out)
    for i in range(G):
        a, b = offsets[i], offsets[i + 1]
        if b > a:
            v, e = ref.product(x[a:b], w[i])
            ref.check(y[a:b], v, ref.rounded(v, e, out), i)


@pytest.mark.parametrize("T,k,E,H,F", [(1, 8, 128, 2048, 768), (3, 2, 5, 72, 40), (19, 8, 32, 1024, 512), (77, 2, 64, 512, 1408),
                                       (600, 4, 9, 136, 264), (700, 8, 128, 256, 96), (2500, 1, 3, 64, 8)])
@pytest.mark.parametrize("t,out", [("bf16", "bf16"), ("f16", "f32")])
def test_routed_layer_of_16_bit_experts(T, k, E, H, F, t, out):
    """group rows -> gate/up with SwiGLU of gathered tokens -> weighted down to the routes' rows -> combine."""
    rng, g = np.random.default_rng(T), gen(T + E)
    ids = np.stack([rng.choice(E, size=min(k, E), replace=False) for _ in range(T)]).astype(np.int32)
    ids[rng.random(ids.shape) < 0.1] = -1
    weights = rng.uniform(0.1, 1.0, size=ids.shape).astype(np.float32)
    R = T * k
    d_ids, d_weights = torch.from_numpy(ids).cuda(), torch.from_numpy(weights).cuda()
    offsets, rows = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(R, dtype=torch.int32, device="cuda")
    size = L.moe_group_rows_workspace(R, E)
    ws = torch.empty(size + 1, dtype=torch.uint8, device="cuda")
    L.moe_group_rows(d_ids, R, E, offsets, rows, ws, size)
    x = rand(g, t, T, H)
    w1, w2 = rand(g, t, E, 2 * F, H, scale=H ** -0.5), rand(g, t, E, H, F, scale=F ** -0.5)
    h = matmul(x, t, offsets, w1, L.MOE_ORDER_NK, F, H, G=E, R=R, act=L.MOE_ACT_SWIGLU, x_index=rows, share=k, out=t, pad=0)
    partial = torch.zeros(T, k, H, device="cuda")
    L.moe_grouped_matmul(h, ref.code(t), R, F, None, 1, offsets, E, R, w2, L.MOE_ORDER_NK, H, F, L.MOE_ACT_NONE, d_weights,
                         rows, partial, L.MOE_F32, R, H)
    y = torch.empty(T, H, device="cuda")
    L.moe_combine(partial, T, k, H, None, y)
    torch.cuda.synchronize()
    o, r = ref.group(ids.reshape(-1), E)
    assert np.array_equal(offsets.cpu().numpy(), o) and np.array_equal(rows.cpu().numpy(), r)
    want, off, total = (torch.zeros(T, H, dtype=torch.float64, device="cuda") for _ in range(3))
    flat = partial.reshape(R, H)
    for e in range(E):
        a, b = o[e], o[e + 1]
        if b == a:
            continue
        route = torch.from_numpy(r[a:b].astype(np.int64)).cuda()
        p, ep = ref.product(x[route // k], w1[e])
        hv, he = ref.swiglu(p[:, :F], ep[:, :F], p[:, F:], ep[:, F:])
        ref.check(h[a:b], hv, ref.rounded(hv, he, t), ("h", e))
        v, ev = ref.product(h[a:b], w2[e])  # of the h that the first product left
        s = d_weights.reshape(-1)[route, None].double()
        ref.check(flat[route], v * s, ref.rounded(v * s, ev * s, "f32"), ("partial", e))
        want.index_add_(0, route // k, v * s)
        off.index_add_(0, route // k, ref.rounded(v * s, ev * s, "f32"))
        total.index_add_(0, route // k, (v * s).abs() + ev * s)
    dropped = torch.from_numpy((ids.reshape(-1) < 0).nonzero()[0]).cuda()
    assert bool((flat[dropped] == 0).all())
    ref.check(y, want, off + k * 2.0 ** -24 * total, "y")  # k additions of the partial rows


@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_strided_rows_shared_rows_and_scale(t):
    g = gen(3)
    T, share, N, K, G = 50, 3, 72, 88, 4
    R = T * share
    wide = rand(g, t, T, K + 40)
    x = wide[:, 16:16 + K]
    w, scale = rand(g, t, G, N, K), torch.randn(R, generator=g, device="cuda")
    perm = torch.randperm(R, generator=g, device="cuda").int()
    offsets = torch.tensor([0, 20, 20, 149, R], dtype=torch.int32, device="cuda")
    y = matmul(x, t, offsets, w, L.MOE_ORDER_NK, N, K, G=G, R=R, x_index=perm, share=share, scale=scale, y_index=perm)
    o = offsets.tolist()
    for i in range(G):
        p = perm[o[i]:o[i + 1]].long()
        if p.numel():
            v, e = ref.product(x[p // share], w[i])
            s = scale[p, None].double()
            ref.check(y[p], v * s, ref.rounded(v * s, e * s.abs(), "f32"), i)


# ------------------------------------------------------------------------------ gradients

@pytest.mark.parametrize("G,R,N,K", [(1, 1, 8, 8), (3, 5, 136, 72), (4, 64, 64, 128), (8, 700, 264, 520), (5, 1000, 128, 2048),
                                     (33, 129, 512, 256), (200, 3000, 72, 40), (2, 4096, 768, 512)])
@pytest.mark.parametrize("t,out", [("bf16", "f32"), ("f16", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("indexed", [0, 1, 2])
def test_weight_gradient(G, R, N, K, t, out, indexed):
    rng, g = np.random.default_rng(R + N), gen(G + K + indexed)
    offsets = uneven(rng, G, R)
    share = 2 if indexed == 1 else 1
    x, dy = rand(g, t, (R + share - 1) // share, K), rand(g, t, R, N)
    perm = torch.randperm(R, generator=g, device="cuda").int()
    xi, yi = (perm if indexed == 1 else None), (perm if indexed == 2 else None)
    dw = torch.full((G, N, K), float("nan"), dtype=ref.dtype(out), device="cuda")
    d_off = torch.from_numpy(offsets).cuda()

    def call(accumulate):
        L.moe_grouped_weight_grad(x, ref.code(t), x.shape[0], K, xi, share, dy, R, N, yi, d_off, G, R, N, K, accumulate, dw,
                                  ref.code(out))
        torch.cuda.synchronize()

    call(0)
    once = dw.clone()
    dw[:, 0] = 0.5
    call(1)
    for i in range(G):
        a, b = offsets[i], offsets[i + 1]
        if a == b:
            assert bool((once[i] == 0).all())
            assert bool((dw[i, 1:] == 0).all()) and bool((dw[i, 0] == 0.5).all())
            continue
        xs = x[perm[a:b].long() // share] if xi is not None else x[a:b]
        ds = dy[perm[a:b].long()] if yi is not None else dy[a:b]
        v, e = ref.product(ds.T, xs.T)
        ref.check(once[i], v, ref.rounded(v, e, out), i)
        before = once[i].double()
        before[0] = 0.5
        e2 = e + 2.0 ** -24 * ((v + before).abs() + e)
        ref.check(dw[i], v + before, ref.rounded(v + before, e2, out), ("accumulated", i))


def test_weight_gradient_ignores_rows_of_other_groups():
    """NaN and infinite rows of the next group, and behind the last, reach no other group's gradient."""
    g = gen(1)
    x, dy = rand(g, "bf16", 200, 64), rand(g, "bf16", 200, 128)
    offsets = torch.tensor([0, 37, 101, 160], dtype=torch.int32, device="cuda")
    x[37:101], dy[37:101] = float("nan"), float("inf")
    x[160:], dy[160:] = float("inf"), float("nan")
    dw = torch.empty(3, 128, 64, device="cuda")
    L.moe_grouped_weight_grad(x, L.MOE_BF16, 200, 64, None, 1, dy, 200, 128, None, offsets, 3, 200, 128, 64, 0, dw, L.MOE_F32)
    torch.cuda.synchronize()
    for i, (a, b) in ((0, (0, 37)), (2, (101, 160))):
        v, e = ref.product(dy[a:b].T, x[a:b].T)
        ref.check(dw[i], v, ref.rounded(v, e, "f32"), i)
    assert bool(dw[1].isnan().all())


# ------------------------------------------------------------------------------ adapters

def lora(x, t, w, adapter, a, b, scale, out, pad=8):
    T, K = x.shape
    N, n, r = w.shape[0], a.shape[0], a.shape[1]
    y = torch.full((T + 1, N + pad), 7.0, dtype=ref.dtype(out), device="cuda")
    size = L.moe_lora_workspace(T, r)
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN wherever it is read unwritten
    L.moe_lora_matmul(x, ref.code(t), T, x.stride(0), w, N, K, adapter, n, a, b, r, scale, y, ref.code(out), N + pad, ws, size)
    torch.cuda.synchronize()
    assert bool((y[:, N:] == 7.0).all()) and bool((y[T] == 7.0).all()) and bool((ws[size:] == 0xFF).all())
    return y[:T, :N]


def lora_bound(x, t, w, a, b, s, out):
    """The product of one adapter's tokens and its bound: u's sum, its split (half a step twice) and the joint sum."""
    v, _ = ref.product(x, w)
    u, eu = ref.product(x, a)
    u, eu = u * s, eu * abs(s) + 2.0 ** -24 * (u * s).abs()
    eu = eu + ref.HALF[t] ** 2 * (u.abs() + eu) + ref.TINY[t]
    r = b.double()
    total = x.double().abs() @ w.double().abs().T + (u.abs() + eu) @ r.abs().T
    n = x.shape[1] + 2 * a.shape[0]
    y = v + u @ r.T
    return y, ref.rounded(y, eu @ r.abs().T + (n + 16) * 2.0 ** -23 * total, out)


@pytest.mark.parametrize("T,n,rank,N,K", [(1, 1, 8, 8, 8), (1, 4, 16, 2816, 2048), (5, 3, 24, 136, 72), (32, 48, 64, 512, 520),
                                          (33, 2, 40, 264, 128), (100, 64, 8, 256, 256), (300, 5, 128, 1000, 64),
                                          (257, 300, 16, 128, 200), (1030, 7, 32, 384, 2048), (64, 1, 256, 64, 64)])
@pytest.mark.parametrize("t,out", [("bf16", "f32"), ("f16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("runs", [True, False])
def test_lora(T, n, rank, N, K, t, out, runs):
    rng, g = np.random.default_rng(T + n), gen(T + rank)
    adapter = rng.integers(-1, n, size=T).astype(np.int32)
    if runs:
        adapter = np.sort(adapter)[::-1].copy()
    x, w = rand(g, t, T, K), rand(g, t, N, K, scale=K ** -0.5)
    a, b = rand(g, t, n, rank, K, scale=K ** -0.5), rand(g, t, n, N, rank, scale=rank ** -0.5)
    scale = torch.randn(n, generator=g, device="cuda") if runs else None
    y = lora(x, t, w, torch.from_numpy(adapter).cuda(), a, b, scale, out)
    for i in range(-1, n):
        mine = torch.from_numpy((adapter == i).nonzero()[0]).cuda()
        if not mine.numel():
            continue
        if i < 0:
            v, e = ref.product(x[mine], w)
            e = ref.rounded(v, e, out)
        else:
            v, e = lora_bound(x[mine], t, w, a[i], b[i], float(scale[i]) if scale is not None else 1.0, out)
        ref.check(y[mine], v, e, i)


def test_lora_reports_adapters_outside():
    g = gen(5)
    T, K, N = 40, 64, 32
    x, w = rand(g, "bf16", T, K), rand(g, "bf16", N, K)
    a, b = rand(g, "bf16", 2, 8, K), rand(g, "bf16", 2, N, 8)
    adapter = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    adapter[3], adapter[39] = 2, -5
    y = lora(x, "bf16", w, adapter, a, b, None, "f32")
    assert L.moe_device_status(clear=True) == L.MOE_ERR_INVALID
    v, e = ref.product(x, w)
    ref.check(y, v, ref.rounded(v, e, "f32"))
