"""MXFP4 on the host: slot images, pack and unpack, and every refusal (no GPU)."""
import ctypes

import numpy as np
import pytest

import mx4_reference as ref
from routed_expert_ffn_gemv_gb300 import _build, _lib as L

MX = L.MOE_MXFP4


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return L.load()


def aligned(n, align=256):
    a = np.zeros(n + align, np.uint8)
    off = (-a.ctypes.data) % align
    return a[off:off + n]


@pytest.mark.parametrize("H,F", [(32, 32), (128, 64), (256, 128), (96, 160), (288, 192)])
def test_pack_is_the_documented_image_and_unpack_inverts_it(lib, H, F):
    rng = np.random.default_rng(H * 1000 + F)
    e = ref.Experts(rng, 1, H, F)
    canon = [ref.canonical(*p) for p in e.parts[0]]
    n = L.moe_slot_image_bytes(MX, H, F)
    img = aligned(n)
    img[:] = 0xFF
    assert L.moe_pack_expert(MX, H, F, *(c.ctypes.data for c in canon), img.ctypes.data) == n
    assert np.array_equal(img, ref.image(*e.parts[0]))
    back = [np.zeros_like(c) for c in canon]
    L.moe_unpack_expert(MX, H, F, img.ctypes.data, *(b.ctypes.data for b in back))
    for a, b in zip(canon, back):
        assert np.array_equal(a, b)


def test_image_is_the_canonical_size_for_whole_tiles(lib):
    for H, F in ((128, 128), (2048, 768), (1024, 512), (2048, 1408)):
        assert L.moe_slot_image_bytes(MX, H, F) == 3 * H * F // 32 * 17


def test_reference_quantiser_known_blocks():
    x = np.zeros((1, 32))
    x[0, :9] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.2]
    codes, scales = ref.quantise(x)
    assert scales[0, 0] == 127  # floor(log2 6) - 2 + 127
    assert codes[0, :9].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8]


def test_other_calls_refuse_the_type(lib):
    b = aligned(4096)
    p = b.ctypes.data
    out = ctypes.c_size_t()
    assert lib.moe_expert_ffn(p, 0, 1, 256, 512, MX, 8, 2, p, p, None, 8, p, 1 << 20, None, 0, p, p, 1 << 20,
                              None) == L.MOE_ERR_INVALID
    assert lib.moe_expert_ffn_noalloc(p, 0, 1, 256, 512, MX, 8, 2, p, p, None, 8, p, 1 << 20, None, 0, p,
                                      None) == L.MOE_ERR_INVALID
    assert lib.moe_stack_workspace(256, 512, MX, 8, 2, 1, 0, ctypes.byref(out)) == L.MOE_ERR_INVALID


def test_quantise_refusals(lib):
    b = aligned(4096)
    p = b.ctypes.data
    bad = L.MOE_ERR_INVALID
    q, d = lib.moe_mx4_quantize, lib.moe_mx4_dequantize
    for f, args in ((q, lambda **k: (k.get("x", p), k.get("t", 0), k.get("rows", 1), k.get("cols", 32),
                                     k.get("ld", 32), k.get("c", p), k.get("s", p), None)),
                    (d, lambda **k: (k.get("c", p), k.get("s", p), k.get("rows", 1), k.get("cols", 32),
                                     k.get("x", p), k.get("t", 0), k.get("ld", 32), None))):
        assert f(*args(rows=0)) == L.MOE_OK
        assert f(*args(rows=-1)) == bad
        assert f(*args(cols=0)) == bad
        assert f(*args(cols=48, ld=48)) == bad
        assert f(*args(ld=31)) == bad
        assert f(*args(t=2)) == bad
        assert f(*args(x=None)) == bad and f(*args(c=None)) == bad and f(*args(s=None)) == bad
        assert f(*args(x=p + 2)) == bad          # fp32 rows on a 2-byte boundary
        assert f(*args(c=p + 8)) == bad
    qe, de = lib.moe_mx4_quantize_experts, lib.moe_mx4_dequantize_experts
    sb = ref.slot_bytes(128, 64)

    def qa(g=p, u=p, w=p, t=0, n=1, H=128, F=64, pool=p, b=sb, slots=None, ns=1):
        return (g, u, w, t, n, H, F, pool, b, slots, ns, None)

    def da(g=p, u=p, w=p, t=0, n=1, H=128, F=64, pool=p, b=sb, slots=None, ns=1):
        return (pool, b, slots, ns, n, H, F, g, u, w, t, None)

    for f, a in ((qe, qa), (de, da)):
        assert f(*a(n=0)) == L.MOE_OK
        for kw in (dict(n=-1), dict(H=100), dict(F=0), dict(t=5), dict(b=sb - 256), dict(b=sb + 16), dict(ns=0),
                   dict(n=2), dict(pool=p + 16), dict(pool=None), dict(g=None), dict(u=None), dict(w=None),
                   dict(g=p + 1)):
            assert f(*a(**kw)) == bad, kw


def test_product_and_layer_refusals(lib):
    b = aligned(4096)
    p = b.ctypes.data
    bad = L.MOE_ERR_INVALID
    sb = ref.slot_bytes(128, 64)
    big = 1 << 40

    def gu(x=p, xs=p, T=1, H=128, F=64, E=4, k=2, ids=p, tab=None, ns=4, pool=p, b=sb, h=p, t=0, ws=p, wb=big):
        return lib.moe_mx4_expert_gateup(x, xs, T, H, F, E, k, ids, tab, ns, pool, b, h, t, ws, wb, None)

    def dn(x=p, xs=p, T=1, H=128, F=64, E=4, k=2, ids=p, tab=None, ns=4, pool=p, b=sb, h=p, w=p, ws=p, wb=big):
        return lib.moe_mx4_expert_down(x, xs, T, H, F, E, k, ids, w, tab, ns, pool, b, h, ws, wb, None)

    def ly(x=p, t=0, T=1, H=128, F=64, E=4, k=2, wr=p, ns=4, pool=p, b=sb, h=p, ws=p, wb=big):
        return lib.moe_mx4_layer(x, t, T, H, F, E, k, wr, None, None, ns, pool, b, None, h, None, None, ws, wb, None)

    for f in (gu, dn, ly):
        assert f(T=0) == L.MOE_OK
        for kw in (dict(T=-1), dict(H=100), dict(F=48), dict(E=0), dict(E=257), dict(k=0), dict(k=5), dict(k=9, E=16),
                   dict(ns=0), dict(pool=None), dict(pool=p + 128), dict(b=sb + 16), dict(b=sb - 256), dict(x=None),
                   dict(h=None), dict(ws=None), dict(ws=p + 16), dict(wb=0)):
            assert f(**kw) == bad, (f.__name__, kw)
    for f in (gu, dn):
        for kw in (dict(xs=None), dict(ids=None), dict(x=p + 8), dict(T=(1 << 23) + 1)):
            assert f(**kw) == bad, (f.__name__, kw)
    assert gu(t=2) == bad and dn(w=None) == bad and dn(h=p + 4) == bad
    assert gu(h=p + 2) == bad and gu(h=p + 1, t=1) == bad
    assert ly(t=2) == bad and ly(wr=None) == bad and ly(T=33) == bad
    out = ctypes.c_size_t()
    assert lib.moe_mx4_expert_workspace(1, 128, 64, 4, 2, None) == bad
    assert lib.moe_mx4_layer_workspace(33, 128, 64, 4, 2, ctypes.byref(out)) == bad
    assert lib.moe_mx4_layer_workspace(32, 128, 64, 4, 2, ctypes.byref(out)) == L.MOE_OK and out.value > 0


def test_layer_refuses_tokens_off_their_elements(lib):
    b = aligned(4096)
    p = b.ctypes.data
    sb = ref.slot_bytes(128, 64)
    for t, x in ((L.MOE_F32, p + 2), (L.MOE_F32, p + 1), (L.MOE_BF16, p + 1)):
        assert lib.moe_mx4_layer(x, t, 1, 128, 64, 4, 2, p, None, None, 4, p, sb, None, p, None, None, p, 1 << 40,
                                 None) == L.MOE_ERR_INVALID, (t, x - p)


def test_layer_refuses_more_tiles_than_a_unit_numbers(lib):
    b = aligned(4096)
    p = b.ctypes.data
    F = (1 << 26) + 32
    sb = (ref.slot_bytes(32, F) + 255) // 256 * 256
    assert lib.moe_mx4_layer(p, L.MOE_F32, 1, 32, F, 4, 2, p, None, None, 4, p, sb, None, p, None, None, p, 1 << 40,
                             None) == L.MOE_ERR_UNSUPPORTED
