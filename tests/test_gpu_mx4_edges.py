"""MXFP4 operators where their precision, launch limits and stream order are at their edges, against
64 bits (tests/mx4_reference.py)."""
import numpy as np
import pytest

import mx4_reference as ref
from routed_expert_ffn_gemv_gb300 import _lib as L

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from test_gpu_mx4 import DT, XT, Layer, clean_status, dev  # noqa: E402,F401


def experts_of(E, H, F, parts):
    """ref.Experts of given (codes, scales) triples, one per expert."""
    e = ref.Experts.__new__(ref.Experts)
    e.E, e.H, e.F, e.parts = E, H, F, parts
    e.vals = [[ref.values(*m) for m in p] for p in parts]
    return e


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


# ------------------------------------------------------------------ precision of the layer's tokens

@pytest.mark.parametrize("xtype", ["f32", "bf16"])
@pytest.mark.parametrize("ratio", [1.0, 45.0, 1e4, 1e6])
@pytest.mark.parametrize("T,H", [(1, 2048), (5, 288), (8, 4096), (12, 1056)])
def test_layer_token_with_a_large_channel(T, H, ratio, xtype):
    """A channel `ratio` times the others, in a block of 32 columns whose weights are zero: the other
    columns keep their 22 bits (of their own block's largest magnitude)."""
    E, F, k = 2, 96, 1
    rng = np.random.default_rng(T + H)
    l = Layer(T, H, F, E, k, seed=T + H, xtype=xtype, extra=False)
    for p in l.ex.parts:
        for m in (0, 1):
            p[m][0][:, 64:96] = 0
    l.ex = experts_of(E, H, F, l.ex.parts)
    pool, l.sb = l.ex.pool(l.table.cpu().numpy(), l.n_slots)
    l.pool = dev(pool.reshape(-1))
    x = l.x.float()
    x[:, 71] = 3.0 * ratio
    l.x = x.to(DT[xtype])
    l.d_wr.zero_()
    l.bias = np.array([0.0, 1.0], np.float32)
    y, ids, w = l.run()
    assert ids.reshape(-1).tolist() == [1] * T
    xs, y = l.x.double().cpu().numpy(), y.double().cpu().numpy()
    g, u, d = l.ex.vals[1]
    for t in range(T):
        h, th = ref.gateup(xs[t], g, u)
        # half a step: a number of 1.71 * 2^21 steps or more stands for the block's largest magnitude
        q = np.abs(xs[t]).reshape(-1, 32).max(1).repeat(32) * 2.0 ** -22
        q[64:96] = 0
        eg, eu = np.abs(g) @ q, np.abs(u) @ q
        th = th + 1.1 * (np.abs(u @ xs[t]) * eg + np.abs(g @ xs[t]) * eu + eg * eu)
        hb = np.abs(h).reshape(-1, 32).max(1).repeat(32) + th
        want = d @ h
        tol = np.abs(d) @ (th + 2.0 ** -22 * hb) + ref.accumulation(F) * (np.abs(d) @ np.abs(h)) + 4 * ref.F32_STEP * np.abs(want)
        err = np.abs(y[t] - want)
        assert (err <= tol).all(), (t, (err / tol).max())
        assert np.linalg.norm(err) <= 2e-6 * np.linalg.norm(want), np.linalg.norm(err) / np.linalg.norm(want)


@pytest.mark.parametrize("T,H,F", [(1, 32, 32), (3, 96, 160), (8, 288, 96), (12, 160, 224), (20, 416, 32)])
def test_layer_takes_any_workspace_contents(T, H, F):
    """Columns past H and F meet weights of zero: what the workspace held before (a NaN scale is 255) must not."""
    l = Layer(T, H, F, 4, 2, seed=H, extra=False)
    y = []
    for fill in (0, 0xFF, 0x7F):
        l.ws.fill_(fill)
        y.append(l.run()[0])
    assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])
    assert not bool(torch.isnan(y[0]).any())


# ------------------------------------------------------------------ SwiGLU of large negative gates

def gate_experts(H, F, gates, up):
    """One expert whose gate rows give gates[f] and up rows `up` for a token of ten ones: sums of a few
    small integers (a power of two), exact in any order; down takes h's column 32 b into row b."""
    gc, gs = np.zeros((F, H), np.uint8), np.full((F, H // 32), 127, np.uint8)
    left = np.abs(gates).astype(np.int64).copy()
    for c in range(10):
        for code, v in ((7, 12), (6, 8), (5, 6), (4, 4), (3, 3), (2, 2), (1, 1)):
            take = (left >= v) & (gc[:, c] == 0)
            gc[take, c] = code
            left[take] -= v
    assert not left.any()
    gc[np.sign(gates) < 0] |= 8 * (gc[np.sign(gates) < 0] > 0).astype(np.uint8)
    gs[:] = 128  # codes times two
    uc, us = np.zeros((F, H), np.uint8), np.full((F, H // 32), 127, np.uint8)
    uc[:, 0] = 2
    us[:, 0] = 127 + up
    dc, ds = np.zeros((H, F), np.uint8), np.full((H, F // 32), 127, np.uint8)
    for b in range(F // 32):
        dc[b, 32 * b] = 2
    return experts_of(1, H, F, [[(gc, gs), (uc, us), (dc, ds)]])


def silu_bound(g, u, htype="f32"):
    """h and the bound of its fp32 evaluation, in half steps (2^-24) of h: exp(-|g| / 2) by a power of two
    good to 2^-22 (4) and its correction (1), squared; a sum (1); a reciprocal good to 2^-23 (2); four products.
    The bf16 form leaves the correction out: the argument's rounding, |g| / 2 log2(e) half steps, and its
    constant's, another half step of it, come to |g| 2^-24 each, twice; then h is rounded to bf16."""
    h = g * (1.0 / (1.0 + np.exp(-g))) * u
    tol = 17 * ref.F32_STEP * np.abs(h)
    if htype == "bf16":
        tol = tol + 4 * np.abs(g) * ref.F32_STEP * np.abs(h)
        tol = tol + ref.BF16_STEP * (np.abs(h) + tol)
    return h, tol


@pytest.mark.parametrize("htype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2100])
def test_product_swiglu_of_every_gate(T, htype):
    H, F = 64, 192
    gates = np.arange(-96, 96).astype(np.float64)
    ex = gate_experts(H, F, gates, 60)
    pool, sb = ex.pool()
    pool = dev(pool.reshape(-1))
    x = np.zeros((T, H))
    x[:, :10] = 1.0
    codes, scales = (np.repeat(a, T, 0) for a in ref.quantise(x[:1]))
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(L.moe_mx4_expert_workspace(T, H, F, 1, 1), dtype=torch.uint8, device="cuda")
    h = torch.full((T, F), 7.0, dtype=DT[htype], device="cuda")
    L.moe_mx4_expert_gateup(dev(ref.pack(codes)), dev(scales), T, H, F, 1, 1, ids, None, 1, pool, sb, h, XT[htype], ws,
                            ws.numel())
    want, tol = silu_bound(gates, 2.0 ** 60, htype)
    got = h.double().cpu().numpy()
    assert (got == got[0]).all()
    err = np.abs(got[0] - want)
    assert (err <= tol).all(), (gates[err > tol], (err / np.maximum(np.abs(want), 1e-300))[err > tol])


@pytest.mark.parametrize("T", [1, 9])
def test_layer_swiglu_of_every_gate(T):
    """A gate to each block of 32 columns of h, so that its digits add 2^-22 of itself at most."""
    gates = np.arange(-96, 32).astype(np.float64)
    H, F = 128, 32 * gates.size
    ex = gate_experts(H, F, gates.repeat(32), 60)
    l = Layer(T, H, 32, 1, 1, seed=1, bias=False, extra=False)
    l.ex, l.F = ex, F
    pool, l.sb = ex.pool(l.table.cpu().numpy(), l.n_slots)
    l.pool = dev(pool.reshape(-1))
    l.x = torch.zeros_like(l.x)
    l.x[:, :10] = 1.0
    l.ws = torch.full((L.moe_mx4_layer_workspace(T, H, F, 1, 1),), 0xC3, dtype=torch.uint8, device="cuda")
    y, _, w = l.run()
    assert bool((w == 1.0).all())
    want, tol = silu_bound(gates, 2.0 ** 60)
    tol = tol + 2.0 ** -22 * np.abs(want)
    got = y.double().cpu().numpy()
    assert (got == got[0]).all()
    err = np.abs(got[0] - want)
    assert (err <= tol).all(), (gates[err > tol], (err / np.maximum(np.abs(want), 1e-300))[err > tol])


# ------------------------------------------------------------------ long rows

@pytest.mark.parametrize("T,H,E", [(32, 48000, 8), (17, 204224, 1), (2, 96000, 3)])
def test_layer_long_router_rows(T, H, E):
    """The first: a little less than 48 KB of shared memory, beside what the kernel declares; the second: the
    longest rows of more than 16 tokens."""
    l = Layer(T, H, 32, E, 1, seed=5, extra=False)
    l.check(*l.run(), tokens=[0, T // 2, T - 1])
    assert L.moe_device_status() == 0


@pytest.mark.parametrize("T,H,E,off", [(1, 4096, 250, 0), (3, 4128, 249, 3), (20, 5120, 251, 1), (16, 1472, 73, 5),
                                       (17, 8192, 130, 2), (4, 32, 1, 1), (2, 64, 7, 7), (32, 30048, 9, 4), (9, 256, 256, 1)])
def test_layer_router_weights_in_several_passes(T, H, E, off):
    """Router rows that are not 16-byte pieces, from any element on: more of them than shared memory holds at a
    time, a few, and fewer than a piece."""
    l = Layer(T, H, 32, E, 1, seed=E, extra=False)
    l.d_wr = torch.cat([l.d_wr.new_zeros(off), l.d_wr.reshape(-1)])[off:]
    assert l.d_wr.data_ptr() % 16 == 2 * off % 16
    l.check(*l.run(), tokens=[0, T - 1])
    assert L.moe_device_status() == 0
