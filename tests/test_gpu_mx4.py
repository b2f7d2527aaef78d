"""The MXFP4 operators on the GPU against plain 64-bit arithmetic (tests/mx4_reference.py)."""
import ctypes

import numpy as np
import pytest

import mx4_reference as ref
import oracle
from gpu_helpers import ids_match
from routed_expert_ffn_gemv_gb300 import _lib as L

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

XT = {"f32": L.MOE_F32, "bf16": L.MOE_BF16}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def clean_status():
    L.load()
    L.moe_device_status(clear=True)
    yield
    torch.cuda.synchronize()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def quantise_gpu(x, xtype="f32", ld=None):
    rows, cols = x.shape
    codes = torch.zeros(rows, cols // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(rows, cols // 32, dtype=torch.uint8, device="cuda")
    L.moe_mx4_quantize(x, XT[xtype], rows, cols, ld or cols, codes, scales)
    return codes, scales


def special_blocks():
    """Every border between codes at several scales, signed zeros, subnormals, the largest floats,
    infinities and NaN."""
    borders = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7.9], np.float32)
    near = np.concatenate([borders, np.nextafter(borders, np.float32(9)), -borders, -np.nextafter(borders, np.float32(-9))])
    rows = []
    for e in (0, -3, 60, -120, 124):
        rows.append(near[:32] * np.float32(2.0 ** e))
        rows.append(near[32:] * np.float32(2.0 ** e))
    zero = np.zeros(32, np.float32)
    rows += [zero, -zero]
    tiny = zero.copy(); tiny[3] = 1e-45; tiny[4] = -3e-45; tiny[5] = 1.1754944e-38
    rows.append(tiny)
    big = zero.copy(); big[0] = 3.4028235e38; big[1] = -1e38; big[2] = 1e30
    rows.append(big)
    for v in (np.inf, -np.inf, np.nan):
        bad = np.ones(32, np.float32); bad[31] = v
        rows.append(bad)
    return np.stack(rows)


@pytest.mark.parametrize("xtype", ["f32", "bf16"])
def test_quantise_borders_and_non_finite_blocks(xtype):
    x = dev(special_blocks()).to(DT[xtype])
    codes, scales = quantise_gpu(x, xtype)
    rc, rs = ref.quantise(x.float().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), ref.pack(rc))
    y = torch.zeros_like(x)
    L.moe_mx4_dequantize(codes, scales, *x.shape, y, XT[xtype], x.shape[1])
    np.testing.assert_array_equal(y.double().cpu().numpy(), ref.values(rc, rs))


@pytest.mark.parametrize("xtype", ["f32", "bf16"])
def test_dequantise_every_scale(xtype):
    """2^(s-127) * e2m1 exactly for every scale byte; an infinity of its sign past the type's range."""
    scales = np.arange(256, dtype=np.uint8)[:, None]
    codes = np.tile(np.arange(16, dtype=np.uint8), 2)[None, :].repeat(256, 0)
    y = torch.zeros(256, 32, dtype=DT[xtype], device="cuda")
    L.moe_mx4_dequantize(dev(ref.pack(codes)), dev(scales), 256, 32, y, XT[xtype], 32)
    want = ref.values(codes, scales)  # 64 bits: nothing overflows there
    want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)
    np.testing.assert_array_equal(y.double().cpu().numpy(), want)


@pytest.mark.parametrize("xtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,pad,off", [(1, 32, 0, 0), (3, 96, 8, 0), (17, 160, 5, 0), (5, 2048, 1, 1), (700, 64, 3, 1),
                                               (257, 224, 32, 8), (2440, 1056, 5, 1)])
def test_quantise_rows_strides_and_alignment(rows, cols, pad, off, xtype):
    rng = np.random.default_rng(rows + cols)
    ld = cols + pad
    flat = dev(rng.standard_normal(rows * ld + off) * np.exp(rng.uniform(-30, 30))).to(DT[xtype])
    x = flat[off:].reshape(rows, ld)
    codes, scales = quantise_gpu_view(x, cols, ld, xtype)
    rc, rs = ref.quantise(x[:, :cols].double().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), ref.pack(rc))
    back = torch.full((rows * ld + off,), 7.0, device="cuda", dtype=DT[xtype])
    L.moe_mx4_dequantize(codes, scales, rows, cols, back[off:], XT[xtype], ld)
    v = back[off:].reshape(rows, ld).double().cpu().numpy()
    np.testing.assert_array_equal(v[:, :cols], ref.values(rc, rs))
    assert (v[:, cols:] == 7.0).all()


@pytest.mark.slow
def test_quantise_past_32_bit_offsets():
    """2^31 groups of eight columns and some: the same codes as of its two halves."""
    rows, cols = (1 << 21) + 6, 8192
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_()
    codes, scales = quantise_gpu(x, "bf16")
    half = rows // 2
    for part in (slice(0, half), slice(half, rows)):
        c, s = quantise_gpu(x[part], "bf16")
        assert torch.equal(codes[part], c) and torch.equal(scales[part], s)
        del c, s
    tail = x[-2:].double().cpu().numpy()
    y = x  # the values take the tokens' place
    L.moe_mx4_dequantize(codes, scales, rows, cols, y, L.MOE_BF16, cols)
    np.testing.assert_array_equal(y[-2:].double().cpu().numpy(), ref.values(*ref.quantise(tail)))
    z = torch.empty(rows - half, cols, dtype=torch.bfloat16, device="cuda")
    L.moe_mx4_dequantize(codes[half:], scales[half:], rows - half, cols, z, L.MOE_BF16, cols)
    assert torch.equal(y[half:], z)


def quantise_gpu_view(x, cols, ld, xtype):
    rows = x.shape[0]
    codes = torch.zeros(rows, cols // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(rows, cols // 32, dtype=torch.uint8, device="cuda")
    L.moe_mx4_quantize(x, XT[xtype], rows, cols, ld, codes, scales)
    return codes, scales


@pytest.mark.parametrize("wtype", ["f32", "bf16"])
@pytest.mark.parametrize("H,F,shift", [(32, 32, 0), (128, 64, 0), (96, 160, 1), (288, 192, 0)])
def test_quantise_experts_writes_the_packed_image(H, F, shift, wtype):
    rng = np.random.default_rng(H + F)
    n, n_slots = 3, 5
    slots = dev(np.array([4, 0, 2], np.int32))
    raw = [dev(rng.standard_normal(n * R * K + shift)).to(DT[wtype]) for R, K in ((F, H), (F, H), (H, F))]
    mats = [r[shift:] for r in raw]  # shift 1: not 16-byte aligned
    sb = ref.slot_bytes(H, F)
    pool = torch.full((n_slots * sb,), 0x5A, dtype=torch.uint8, device="cuda")
    L.moe_mx4_quantize_experts(*mats, XT[wtype], n, H, F, pool, sb, slots, n_slots)
    got = pool.cpu().numpy().reshape(n_slots, sb)
    size = L.moe_slot_image_bytes(L.MOE_MXFP4, H, F)
    shapes = ((F, H), (F, H), (H, F))
    for i, s in enumerate((4, 0, 2)):
        parts = [ref.quantise(m.double().cpu().numpy().reshape(n, R, K)[i]) for m, (R, K) in zip(mats, shapes)]
        assert np.array_equal(got[s, :size], ref.image(*parts))
        assert (got[s, size:] == 0x5A).all()
    assert (got[[1, 3]] == 0x5A).all()
    out = [torch.zeros(n * R * K + shift, device="cuda", dtype=DT[wtype]) for R, K in shapes]
    L.moe_mx4_dequantize_experts(pool, sb, slots, n_slots, n, H, F, *(o[shift:] for o in out), XT[wtype])
    for m, o, (R, K) in zip(mats, out, shapes):
        want = ref.values(*ref.quantise(m.double().cpu().numpy().reshape(n * R, K)))
        np.testing.assert_array_equal(o[shift:].double().cpu().numpy().reshape(n * R, K), want)
    assert L.moe_device_status() == 0


def test_quantise_experts_skips_a_slot_out_of_range():
    H, F = 64, 32
    sb = ref.slot_bytes(H, F)
    pool = torch.full((2 * sb,), 0x5A, dtype=torch.uint8, device="cuda")
    w = torch.ones(2 * H * F, device="cuda")
    for bad in (2, -1):
        slots = dev(np.array([bad, 1], np.int32))
        L.moe_mx4_quantize_experts(w, w, w, 0, 2, H, F, pool, sb, slots, 2)
        assert L.moe_device_status() == L.MOE_ERR_INVALID
        assert bool((pool[:sb] == 0x5A).all()) and not bool((pool[sb:] == 0x5A).all())
        out = torch.full((2 * H * F,), 7.0, device="cuda")
        L.moe_mx4_dequantize_experts(pool, sb, slots, 2, 2, H, F, out, out.clone(), out.clone(), 0)
        assert L.moe_device_status() == L.MOE_ERR_INVALID
        assert bool((out[:H * F] == 7.0).all()) and bool((out[H * F:] == 1.0).all())


# ------------------------------------------------------------------ products

class Call:
    """One product call's inputs, buffers and reference."""

    def __init__(self, T, H, F, E, k, seed, ids=None, table=None, n_slots=None, htype="f32"):
        rng = np.random.default_rng(seed)
        self.T, self.H, self.F, self.E, self.k, self.htype = T, H, F, E, k, htype
        self.ex = ref.Experts(rng, E, H, F)
        pool, self.sb = self.ex.pool(table, n_slots)
        self.pool = dev(pool.reshape(-1))
        self.table = None if table is None else dev(np.asarray(table, np.int32))
        self.n_slots = n_slots or E
        self.ids = ids if ids is not None else np.stack(
            [rng.choice(E, k, replace=False) for _ in range(T)]).astype(np.int32)
        self.d_ids = dev(self.ids)
        self.w = rng.uniform(0.05, 1.0, (T, k)).astype(np.float32)
        self.d_w = dev(self.w)
        self.x = ref.quantise(rng.standard_normal((T, H)))
        self.hq = ref.quantise(rng.standard_normal((T * k, F)))
        self.ws = torch.full((L.moe_mx4_expert_workspace(T, H, F, E, k),), 0xC3, dtype=torch.uint8, device="cuda")

    def inputs(self, q):
        return dev(ref.pack(q[0])), dev(q[1])

    def gateup(self, stream=None, h=None, q=None):
        c, s = q or self.inputs(self.x)
        if h is None:
            h = torch.full((self.T * self.k, self.F), 7.0, dtype=DT[self.htype], device="cuda")
        L.moe_mx4_expert_gateup(c, s, self.T, self.H, self.F, self.E, self.k, self.d_ids, self.table, self.n_slots,
                                self.pool, self.sb, h, XT[self.htype], self.ws, self.ws.numel(), stream)
        return h

    def down(self, stream=None, out=None, q=None):
        c, s = q or self.inputs(self.hq)
        if out is None:
            out = torch.full((self.T, self.k, self.H), 7.0, device="cuda")
        L.moe_mx4_expert_down(c, s, self.T, self.H, self.F, self.E, self.k, self.d_ids, self.d_w, self.table,
                              self.n_slots, self.pool, self.sb, out, self.ws, self.ws.numel(), stream)
        return out

    def served(self, r):
        e = self.ids.reshape(-1)[r]
        return 0 <= e < self.E and (self.table is None or 0 <= int(self.table[e]) < self.n_slots)

    def check_gateup(self, h, rows=None):
        h = h.double().cpu().numpy()
        x = ref.values(*self.x)
        for r in rows if rows is not None else range(self.T * self.k):
            if not self.served(r):
                assert (h[r] == 7.0).all(), r
                continue
            want, tol = ref.gateup(x[r // self.k], *self.ex.vals[self.ids.reshape(-1)[r]][:2])
            if self.htype == "bf16":
                tol = tol + ref.BF16_STEP * (np.abs(want) + tol)
            assert (np.abs(h[r] - want) <= tol + 1e-37).all(), (r, np.abs(h[r] - want).max(), tol.max())

    def check_down(self, out, rows=None):
        out = out.double().cpu().numpy().reshape(self.T * self.k, self.H)
        h = ref.values(*self.hq)
        for r in rows if rows is not None else range(self.T * self.k):
            if not self.served(r):
                assert (out[r] == 7.0).all(), r
                continue
            d = self.ex.vals[self.ids.reshape(-1)[r]][2]
            w = float(self.w.reshape(-1)[r])
            tol = w * ref.accumulation(self.F) * (np.abs(d) @ np.abs(h[r])) + ref.F32_STEP * np.abs(w * (d @ h[r]))
            assert (np.abs(out[r] - w * (d @ h[r])) <= tol + 1e-37).all(), r


SHAPES = [(1, 32, 32, 1, 1), (1, 256, 512, 8, 2), (2, 64, 96, 3, 3), (3, 96, 160, 5, 3), (33, 128, 64, 8, 4),
          (5, 288, 192, 256, 8), (77, 160, 224, 4, 2), (1, 2048, 768, 8, 8), (9, 1024, 1408, 4, 2)]


@pytest.mark.parametrize("htype", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,F,E,k", SHAPES)
def test_products_against_64_bits(T, H, F, E, k, htype):
    c = Call(T, H, F, E, k, seed=T * 7 + H, htype=htype)
    c.check_gateup(c.gateup())
    c.check_down(c.down())
    assert L.moe_device_status() == 0


@pytest.mark.parametrize("n", [1, 7, 8, 9, 127, 128, 129, 175, 176, 177, 255, 256, 257, 513, 1000, 1024, 1025, 2047, 2048,
                               2049, 2113])
def test_one_expert_takes_every_route(n):
    """Group lengths around every tile border; the other experts are empty."""
    ids = np.full((n, 1), 2, np.int32)
    c = Call(n, 160, 96, 4, 1, seed=n, ids=ids)
    rows = sorted({0, 1, n // 2, max(0, n - 2), n - 1} | set(range(0, n, 61)))
    rows = [r for r in rows if r < n]
    c.check_gateup(c.gateup(), rows)
    c.check_down(c.down(), rows)


def test_dropped_routes_repeats_and_slot_table():
    rng = np.random.default_rng(5)
    T, E, k = 21, 6, 4
    ids = rng.integers(-1, E, (T, k)).astype(np.int32)  # repeats within a token, -1 among them
    ids[3] = -1
    ids[4] = 2
    c = Call(T, 160, 96, E, k, seed=5, ids=ids, table=rng.permutation(9)[:E], n_slots=9)
    c.check_gateup(c.gateup())
    c.check_down(c.down())
    assert L.moe_device_status() == 0
    none = Call(T, 160, 96, E, k, seed=5, ids=np.full((T, k), -1, np.int32))
    assert bool((none.gateup() == 7.0).all()) and bool((none.down() == 7.0).all())
    assert L.moe_device_status() == 0


@pytest.mark.parametrize("T,k,E", [(300, 4, 5), (1031, 1, 256), (515, 8, 16), (129, 8, 129), (257, 8, 9),
                                   (700, 3, 130)])
def test_many_routes_dropped_and_repeated(T, k, E):
    """More routes than a CTA groups for itself, over few and over many experts, some unused."""
    rng = np.random.default_rng(T)
    ids = rng.integers(-1, max(1, E - 2), (T, k)).astype(np.int32)
    c = Call(T, 96, 64, E, k, seed=T, ids=ids, table=rng.permutation(E + 3)[:E], n_slots=E + 3)
    rows = list(range(0, T * k, 7)) + [T * k - 1]
    c.check_gateup(c.gateup(), rows)
    c.check_down(c.down(), rows)
    assert L.moe_device_status() == 0


@pytest.mark.parametrize("T", [1, 40, 300, 600])
def test_ids_and_slots_out_of_range_are_reported_and_skipped(T):
    k, E = 4, 6
    ids = np.tile(np.array([[0, E, -7, 3]], np.int32), (T, 1))
    c = Call(T, 64, 96, E, k, seed=T, ids=ids)
    for run, check in ((c.gateup, c.check_gateup), (c.down, c.check_down)):
        out = run()
        assert L.moe_device_status() == L.MOE_ERR_INVALID
        check(out)
    ids = np.tile(np.array([[0, 1, 2, 3]], np.int32), (T, 1))
    c = Call(T, 64, 96, E, k, seed=T, ids=ids)
    c.table = dev(np.array([0, -1, 6, 3, 4, 5], np.int32))  # experts 1 and 2 are not resident
    for run, check in ((c.gateup, c.check_gateup), (c.down, c.check_down)):
        out = run()
        assert L.moe_device_status() == L.MOE_ERR_INVALID
        check(out)


def test_nan_scale_poisons_its_row_alone():
    c = Call(9, 128, 64, 4, 2, seed=3)
    c.x[1][4, 2] = 255
    h = c.gateup().cpu().numpy()
    nan = np.isnan(h).all(axis=1)
    assert nan.tolist() == [r // 2 == 4 for r in range(18)]
    assert not np.isnan(h[~nan]).any()


def test_streams_graphs_and_repeats_give_the_same_bits():
    c = Call(50, 256, 192, 8, 4, seed=1)
    q, hq = c.inputs(c.x), c.inputs(c.hq)
    h0, p0 = c.gateup(q=q), c.down(q=hq)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    h1, p1 = torch.full_like(h0, 7.0), torch.full_like(p0, 7.0)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.gateup(h=h1, q=q)
        c.down(out=p1, q=hq)
    side.synchronize()
    assert torch.equal(h0, h1) and torch.equal(p0, p1)
    h2, p2 = torch.full_like(h0, 7.0), torch.full_like(p0, 7.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.gateup(h=h2, q=q)
        c.down(out=p2, q=hq)
    for _ in range(3):
        h2.fill_(7.0)
        p2.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(h0, h2) and torch.equal(p0, p2)
    # two calls in flight at once on two streams, a workspace each
    d = Call(50, 256, 192, 8, 4, seed=1)
    s2 = torch.cuda.Stream()
    h3, h4 = torch.full_like(h0, 7.0), torch.full_like(h0, 7.0)
    torch.cuda.synchronize()
    for _ in range(10):
        c.gateup(side, h3, q)
        d.gateup(s2, h4, q)
    torch.cuda.synchronize()
    assert torch.equal(h0, h3) and torch.equal(h0, h4)


def test_prompt_chain_and_pool():
    """Experts uploaded by a host-managed pool; quantise, gate/up, quantise, down, combine."""
    rng = np.random.default_rng(11)
    T, H, F, E, k = 37, 256, 192, 6, 3
    c = Call(T, H, F, E, k, seed=11)
    sb, n_slots = c.sb, 8
    host = [torch.zeros(sb, dtype=torch.uint8).pin_memory() for _ in range(E)]
    for e in range(E):
        img = ref.image(*c.ex.parts[e])
        host[e][:img.size] = torch.from_numpy(img)
    pool = torch.zeros(n_slots * sb + 256, dtype=torch.uint8, device="cuda")
    pool = pool[(-pool.data_ptr()) % 256:][:n_slots * sb]
    copy = torch.cuda.Stream()
    images = (ctypes.c_void_p * E)(*(t.data_ptr() for t in host))
    desc = L.CacheDesc(qtype=L.MOE_MXFP4, H=H, F=F, n_layers=1, n_experts=E, first_layer=0, n_slots=n_slots,
                       slot_bytes=sb, device_pool=pool.data_ptr(), host_images=images, copy_stream=copy.cuda_stream,
                       device_managed=0)
    cache = L.moe_cache_create(desc)
    slots = np.zeros((T, k), np.int32)
    table = torch.zeros(E, dtype=torch.int32, device="cuda")
    L.moe_cache_ensure(cache, 0, c.ids[:8].ctypes.data, 8, k, slots.ctypes.data, None, table)
    L.moe_cache_ensure(cache, 0, np.arange(E, dtype=np.int32).ctypes.data, 1, E, slots.ctypes.data, None, table)
    L.moe_cache_wait_uploads(cache)
    c.pool, c.table, c.n_slots = pool, table, n_slots
    x = dev(rng.standard_normal((T, H)).astype(np.float32))
    c.x = ref.quantise(x.double().cpu().numpy())
    q = quantise_gpu(x)
    h = c.gateup(q=q)
    c.check_gateup(h)
    hq = quantise_gpu(h)
    c.hq = ref.quantise(h.double().cpu().numpy())
    assert np.array_equal(hq[0].cpu().numpy(), ref.pack(c.hq[0]))
    partial = c.down(q=hq)
    c.check_down(partial)
    y = torch.empty(T, H, device="cuda")
    L.moe_combine(partial, T, k, H, x, y)
    want = x.double() + partial.double().sum(1)
    assert torch.allclose(y.double(), want, rtol=(k + 1) * 2 ** -24 * 4, atol=1e-5)
    L.moe_cache_release(cache)
    torch.cuda.synchronize()
    # a stack's kernels read other images: such a pool is refused
    wr = torch.zeros(H, E, dtype=torch.float16, device="cuda")
    wsb = L.moe_stack_workspace(H, F, L.MOE_Q8_0, E, k, 1, 0)
    sws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    stack = L.StackDesc(qtype=L.MOE_Q8_0, H=H, F=F, E=E, k=k, n_layers=1, n_shared=0,
                        w_router=(ctypes.c_void_p * 1)(wr.data_ptr()), n_groups=1,
                        caches=(ctypes.c_void_p * 1)(cache), slot_bytes=1 << 20, max_T=1, workspace=sws.data_ptr(),
                        ws_bytes=wsb)
    out = ctypes.c_void_p()
    assert L.load().moe_stack_create(ctypes.byref(stack), ctypes.byref(out)) == L.MOE_ERR_UNSUPPORTED
    desc.device_managed = 1
    out = ctypes.c_void_p()
    assert L.load().moe_cache_create(ctypes.byref(desc), ctypes.byref(out)) == L.MOE_ERR_UNSUPPORTED
    L.moe_cache_destroy(cache)


# ------------------------------------------------------------------ the whole layer

class Layer:
    def __init__(self, T, H, F, E, k, seed, xtype="f32", bias=True, extra=True, gain=1.0):
        rng = np.random.default_rng(seed)
        self.T, self.H, self.F, self.E, self.k, self.xtype = T, H, F, E, k, xtype
        self.ex = ref.Experts(rng, E, H, F)
        table = rng.permutation(E + 2)[:E].astype(np.int32)
        pool, self.sb = self.ex.pool(table, E + 2)
        self.pool, self.table, self.n_slots = dev(pool.reshape(-1)), dev(table), E + 2
        self.x = dev((rng.standard_normal((T, H)) * gain).astype(np.float32)).to(DT[xtype])
        self.wr = (rng.standard_normal((H, E)) / H ** 0.5 / gain).astype(np.float16)
        self.d_wr = dev(self.wr)
        self.bias = rng.standard_normal(E).astype(np.float32) if bias else None
        self.extra = dev(rng.standard_normal((T, H)).astype(np.float32)) if extra else None
        self.ws = torch.full((L.moe_mx4_layer_workspace(T, H, F, E, k),), 0xC3, dtype=torch.uint8, device="cuda")

    def run(self, y=None, stream=None, with_ids=True, extra="own"):
        y = torch.full((self.T, self.H), 7.0, device="cuda") if y is None else y
        ids = torch.full((self.T, self.k), -9, dtype=torch.int32, device="cuda") if with_ids else None
        w = torch.full((self.T, self.k), -9.0, device="cuda") if with_ids else None
        L.moe_mx4_layer(self.x, XT[self.xtype], self.T, self.H, self.F, self.E, self.k, self.d_wr,
                        None if self.bias is None else dev(self.bias), self.table, self.n_slots, self.pool, self.sb,
                        self.extra if extra == "own" else extra, y, ids, w, self.ws, self.ws.numel(), stream)
        return y, ids, w

    def check(self, y, ids, w, tokens=None):
        x = self.x.double().cpu().numpy()
        y, ids, w = y.double().cpu().numpy(), ids.cpu().numpy(), w.double().cpu().numpy()
        logits = x @ self.wr.astype(np.float64) + (0 if self.bias is None else self.bias.astype(np.float64))
        order = np.stack([np.lexsort((np.arange(self.E), -l)) for l in logits])
        want_ids = order[:, :self.k]
        assert all(m is not False for m in ids_match(ids, logits, want_ids, self.k))
        for t in tokens if tokens is not None else range(self.T):
            l = logits[t, ids[t]]
            wt = np.exp(l - l.max())
            wt /= wt.sum()
            # logits within 2e-6 max(1, |l|) (the router's own bound), softmax of k terms
            assert np.abs(w[t] - wt).max() <= 4 * 2e-6 * max(1.0, np.abs(l).max()) + 16 * ref.F32_STEP
            want = np.zeros(self.H) if self.extra is None else self.extra[t].double().cpu().numpy()
            tol = (self.k + 1) * 2 * ref.F32_STEP * np.abs(want)
            for j in range(self.k):
                g, u, d = self.ex.vals[ids[t, j]]
                h, th = ref.gateup(x[t], g, u)
                # x to 22 bits of its largest magnitude, h of each 32 columns' largest
                q = 2.0 ** -21 * np.abs(x[t]).max()
                th = th + 1.1 * (np.abs(u @ x[t]) * q * np.abs(g).sum(1) + np.abs(g @ x[t]) * q * np.abs(u).sum(1))
                hb = np.abs(h).reshape(-1, 32).max(1).repeat(32) + th
                th = th + 2.0 ** -20 * hb
                o = d @ h
                want = want + w[t, j] * o
                tol = tol + w[t, j] * (np.abs(d) @ th + ref.accumulation(self.F) * (np.abs(d) @ np.abs(h))) \
                    + (self.k + 4) * 2 * ref.F32_STEP * np.abs(w[t, j] * o)
            err = np.abs(y[t] - want)
            assert (err <= tol + 1e-37).all(), (t, (err / (tol + 1e-37)).max())
            # and as a whole, far inside the type's resolution of a length-H vector
            assert np.linalg.norm(err) <= 1e-5 * np.linalg.norm(want) + 1e-30, np.linalg.norm(err) / np.linalg.norm(want)


LAYERS = [(1, 32, 32, 1, 1), (1, 256, 512, 8, 2), (2, 96, 160, 5, 3), (8, 288, 192, 16, 8), (9, 128, 64, 3, 2),
          (32, 160, 96, 40, 4), (32, 64, 32, 2, 2), (17, 256, 128, 256, 8), (32, 128, 64, 256, 8), (32, 96, 64, 4, 4),
          (8, 4096, 32, 2, 1), (7, 4096, 160, 3, 2), (1, 2048, 768, 16, 8), (3, 1024, 1408, 4, 2)]


@pytest.mark.parametrize("xtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,F,E,k", LAYERS)
def test_layer_against_64_bits(T, H, F, E, k, xtype):
    l = Layer(T, H, F, E, k, seed=T * 31 + H + k, xtype=xtype)
    l.check(*l.run())
    assert L.moe_device_status() == 0


def test_layer_optional_arguments_and_aliased_output():
    l = Layer(5, 128, 96, 6, 3, seed=2, bias=False, extra=False)
    y, ids, w = l.run()
    l.check(y, ids, w)
    y2, _, _ = l.run(with_ids=False)
    assert torch.equal(y, y2)
    l = Layer(5, 128, 96, 6, 3, seed=3)
    y, ids, w = l.run()
    l.check(y, ids, w)
    z = l.extra.clone()
    l.run(y=z, extra=z)
    assert torch.equal(y, z)


def test_layer_unaligned_router_and_tokens():
    """Router weights and tokens on element boundaries only."""
    l = Layer(5, 160, 96, 16, 3, seed=13, xtype="bf16")
    y, ids, w = l.run()
    l.check(y, ids, w)
    wr, x = l.d_wr, l.x
    l.d_wr = torch.cat([wr.new_zeros(1), wr.reshape(-1)])[1:]
    l.x = torch.cat([x.new_zeros(1), x.reshape(-1)])[1:].reshape(x.shape)
    assert l.d_wr.data_ptr() % 16 and l.x.data_ptr() % 16
    y2, ids2, w2 = l.run()
    assert torch.equal(ids, ids2)
    l.check(y2, ids2, w2)


def test_layer_equal_logits_go_to_the_lower_expert():
    l = Layer(3, 128, 64, 40, 8, seed=14, bias=False, extra=False)
    l.d_wr.zero_()
    l.wr = np.zeros_like(l.wr)
    y, ids, w = l.run()
    assert ids.tolist() == [list(range(8))] * 3
    assert torch.allclose(w, torch.full_like(w, 0.125), rtol=2 ** -22, atol=0)
    l.bias = np.zeros(40, np.float32)
    l.bias[[39, 7, 20]] = 1.0
    l.bias[5] = -0.0
    y, ids, w = l.run()
    assert ids.tolist() == [[7, 20, 39, 0, 1, 2, 3, 4]] * 3
    l.check(y, ids, w)


@pytest.mark.parametrize("gain", [1e-18, 1e-6, 1e6, 1e18])
def test_layer_scales_of_x(gain):
    l = Layer(4, 128, 96, 6, 3, seed=4, gain=1.0, extra=False)
    l.x = l.x * gain
    # products of x with itself stay in range: the down weights' sum carries gain^2 at most
    l.bias = np.arange(6, dtype=np.float32) * 8  # the routing does not depend on x's size
    l.d_wr.zero_()
    l.wr = np.zeros_like(l.wr)
    y, ids, w = l.run()
    l.check(y, ids, w)


def test_layer_subnormal_tokens_and_overflowing_h():
    l = Layer(4, 128, 96, 6, 3, seed=4, extra=True)
    l.bias = np.arange(6, dtype=np.float32) * 8
    l.d_wr.zero_()
    x = l.x.clone()
    l.x = x * 1e-41
    y, ids, w = l.run()
    assert torch.equal(y, l.extra)  # products of two such values are zero
    l.x = x * 1e30
    y, ids, w = l.run()
    assert bool(torch.isnan(y).all())
    assert L.moe_device_status() == 0


def test_layer_zero_and_non_finite_tokens():
    l = Layer(6, 128, 96, 4, 2, seed=6, extra=False)
    ok, ids0, w0 = l.run()
    x = l.x.clone()
    x[1] = 0
    x[3, 5] = float("nan")
    x[4, 7] = float("inf")
    l.x = x
    y, ids, w = l.run()
    assert bool((y[1] == 0).all())
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(y[4]).all())
    for t in (0, 2, 5):
        assert torch.equal(y[t], ok[t])


def test_layer_missing_expert_is_reported_and_adds_nothing():
    l = Layer(4, 128, 96, 4, 2, seed=8, extra=True)
    _, ids, w = l.run()
    gone = int(ids[0, 0])
    l.table[gone] = -1
    y, ids2, w2 = l.run()
    assert L.moe_device_status() == L.MOE_ERR_INVALID
    assert torch.equal(ids, ids2)
    w3 = torch.where(ids == gone, torch.zeros_like(w), w)
    l.check_w = None
    x = l.x.double().cpu().numpy()
    for t in range(4):
        want = l.extra[t].double().cpu().numpy()
        for j in range(2):
            g, u, d = l.ex.vals[int(ids[t, j])]
            want = want + float(w3[t, j]) * (d @ ref.gateup(x[t], g, u)[0])
        assert np.linalg.norm(y[t].double().cpu().numpy() - want) <= 1e-5 * np.linalg.norm(want)


def test_layer_streams_graphs_and_repeats_give_the_same_bits():
    l = Layer(8, 256, 192, 16, 4, seed=9)
    d_bias = dev(l.bias)

    def call(m, y, stream=None):
        L.moe_mx4_layer(m.x, XT[m.xtype], m.T, m.H, m.F, m.E, m.k, m.d_wr, d_bias, m.table, m.n_slots, m.pool, m.sb,
                        m.extra, y, None, None, m.ws, m.ws.numel(), stream)

    y0 = torch.full((8, 256), 7.0, device="cuda")
    call(l, y0)
    torch.cuda.synchronize()
    for _ in range(20):  # back to back on one workspace
        y = torch.full_like(y0, 7.0)
        call(l, y)
        assert torch.equal(y, y0)
    m = Layer(8, 256, 192, 16, 4, seed=9)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    y1, y2 = torch.full_like(y0, 7.0), torch.full_like(y0, 7.0)
    torch.cuda.synchronize()
    for _ in range(20):  # two calls in flight at once
        call(l, y1, s1)
        call(m, y2, s2)
    torch.cuda.synchronize()
    assert torch.equal(y1, y0) and torch.equal(y2, y0)
    y3 = torch.full_like(y0, 7.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(l, y3)
        call(l, y3)
    for _ in range(5):
        y3.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y3, y0)
    assert L.moe_device_status() == 0


def test_layer_then_prompt_path_agree_to_four_bits():
    """The same experts serve both paths: the prompt path differs by its 4-bit activations only."""
    l = Layer(16, 256, 192, 8, 2, seed=12, extra=False)
    y, ids, w = l.run()
    T, H, F, E, k = l.T, l.H, l.F, l.E, l.k
    ws = torch.empty(L.moe_mx4_expert_workspace(T, H, F, E, k), dtype=torch.uint8, device="cuda")
    q = quantise_gpu(l.x)
    h = torch.empty(T * k, F, device="cuda")
    L.moe_mx4_expert_gateup(*q, T, H, F, E, k, ids, l.table, l.n_slots, l.pool, l.sb, h, 0, ws, ws.numel())
    hq = quantise_gpu(h)
    part = torch.empty(T, k, H, device="cuda")
    L.moe_mx4_expert_down(*hq, T, H, F, E, k, ids, w, l.table, l.n_slots, l.pool, l.sb, part, ws, ws.numel())
    z = torch.empty(T, H, device="cuda")
    L.moe_combine(part, T, k, H, None, z)
    # an E2M1 step is at most 1/4 of a value in (4, 6] and 1/8 elsewhere above 1: about 0.12 rms of x,
    # twice over in gate * up and once more in h
    assert float((y - z).norm() / y.norm()) < 0.4
