"""The MXFP4 products and layer over many work items, stages and routes, against 64 bits
(tests/mx4_reference.py).  Many experts share a few slots, so that the weights stay small."""
import numpy as np
import pytest

import mx4_reference as ref
from routed_expert_ffn_gemv_gb300 import _lib as L

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from test_gpu_mx4 import DT, XT, Call, Layer, clean_status, dev  # noqa: E402,F401


class SharedExperts:
    """E experts over `distinct` slots (expert e: slot e % distinct), images by moe_pack_expert."""

    def __init__(self, rng, E, H, F, distinct):
        base = ref.Experts(rng, distinct, H, F)
        self.E, self.H, self.F, self.distinct = E, H, F, distinct
        self.base = base
        self.vals = [base.vals[e % distinct] for e in range(E)]
        self.table = (np.arange(E) % distinct).astype(np.int32)

    def pool(self):
        sb = ref.slot_bytes(self.H, self.F)
        out = np.zeros((self.distinct, sb), np.uint8)
        img = np.zeros(sb + 16, np.uint8)
        at = (-img.ctypes.data) % 16
        for e in range(self.distinct):
            canon = [ref.canonical(*m) for m in self.base.parts[e]]
            n = L.moe_pack_expert(L.MOE_MXFP4, self.H, self.F, *(c.ctypes.data for c in canon), img.ctypes.data + at)
            out[e, :n] = img[at:at + n]
        return out, sb


def random_rows(rng, rows, K):
    return (rng.integers(0, 16, (rows, K), dtype=np.uint8), rng.integers(126, 129, (rows, K // 32)).astype(np.uint8))


class SharedCall(Call):
    def __init__(self, T, H, F, E, k, seed, htype="f32", distinct=3, dropped=False):
        rng = np.random.default_rng(seed)
        self.T, self.H, self.F, self.E, self.k, self.htype = T, H, F, E, k, htype
        self.ex = SharedExperts(rng, E, H, F, distinct)
        pool, self.sb = self.ex.pool()
        self.pool, self.table, self.n_slots = dev(pool.reshape(-1)), dev(self.ex.table), distinct
        self.ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
        if dropped:
            self.ids[rng.random((T, k)) < 0.1] = -1
        self.d_ids = dev(self.ids)
        self.w = rng.uniform(0.05, 1.0, (T, k)).astype(np.float32)
        self.d_w = dev(self.w)
        self.x, self.hq = random_rows(rng, T, H), random_rows(rng, T * k, F)
        self.ws = torch.full((L.moe_mx4_expert_workspace(T, H, F, E, k),), 0xFF, dtype=torch.uint8, device="cuda")

    def some(self, n=48):
        R = self.T * self.k
        return sorted({0, 1, R - 1, R - 2} | set(range(0, R, max(1, R // n))))


# several stages of 256 columns and several work items to a CTA (152 of them), the ring's stages used more
# than once; few routes (each CTA groups them: up to 2048) and more; chunks of up to 32 routes (up to 16 an
# expert) and wide ones
LONG = [(2200, 1056, 1312, 16, 2), (1100, 2080, 1056, 40, 2), (300, 1056, 1184, 256, 8), (500, 1312, 1056, 256, 8),
        (250, 1056, 1312, 200, 8), (1000, 1056, 1440, 8, 2), (900, 544, 2592, 128, 3)]


@pytest.mark.parametrize("htype", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,F,E,k", LONG)
def test_products_of_many_stages_and_items(T, H, F, E, k, htype):
    c = SharedCall(T, H, F, E, k, seed=T, htype=htype, dropped=T % 100 == 0)
    c.check_gateup(c.gateup(), c.some())
    if htype == "f32":
        c.check_down(c.down(), c.some())
    assert L.moe_device_status() == 0


@pytest.mark.parametrize("T,tiles,E,k", [(128, 200, 64, 4), (256, 100, 128, 4), (300, 60, 256, 8), (2100, 260, 64, 1)])
def test_products_of_more_items_than_are_looked_up_ahead(T, tiles, E, k):
    """More than 64 work items to a CTA: chunks (an expert at least) by weight tiles."""
    c = SharedCall(T, 32, 64 * tiles, E, k, seed=tiles)
    c.check_gateup(c.gateup(), c.some(24))
    c = SharedCall(T, 128 * tiles, 32, E, k, seed=tiles)
    c.check_down(c.down(), c.some(24))
    assert L.moe_device_status() == 0


@pytest.mark.parametrize("T,E,k", [(300, 256, 8), (1100, 24, 2)])
def test_prompt_chain_in_a_graph(T, E, k):
    """Quantise, gate/up, quantise, down, combine on one stream and one workspace, more routes than a CTA groups
    for itself: captured and replayed, the bits of the calls made one by one."""
    H, F = 288, 160
    c = SharedCall(T, H, F, E, k, seed=E)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()

    def buffers():
        u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
        return dict(xc=u8(T, H // 2), xs=u8(T, H // 32), h=torch.zeros(T * k, F, dtype=torch.bfloat16, device="cuda"),
                    hc=u8(T * k, F // 2), hs=u8(T * k, F // 32), p=torch.zeros(T, k, H, device="cuda"),
                    y=torch.zeros(T, H, device="cuda"))

    def steps(b):
        yield lambda: L.moe_mx4_quantize(x, L.MOE_BF16, T, H, H, b["xc"], b["xs"])
        yield lambda: L.moe_mx4_expert_gateup(b["xc"], b["xs"], T, H, F, E, k, c.d_ids, c.table, c.n_slots, c.pool, c.sb,
                                              b["h"], L.MOE_BF16, c.ws, c.ws.numel())
        yield lambda: L.moe_mx4_quantize(b["h"], L.MOE_BF16, T * k, F, F, b["hc"], b["hs"])
        yield lambda: L.moe_mx4_expert_down(b["hc"], b["hs"], T, H, F, E, k, c.d_ids, c.d_w, c.table, c.n_slots, c.pool,
                                            c.sb, b["p"], c.ws, c.ws.numel())
        yield lambda: L.moe_combine(b["p"], T, k, H, None, b["y"])

    one = buffers()
    for call in steps(one):
        call()
        torch.cuda.synchronize()
    both = buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in steps(both):
            call()
    for _ in range(5):
        for t in both.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(one[n], both[n]) for n in one)
    # and the values, stage by stage
    unpack = lambda t: np.stack((t & 15, t >> 4), -1).reshape(t.shape[0], -1)  # noqa: E731
    c.x = (unpack(one["xc"].cpu().numpy()), one["xs"].cpu().numpy())
    c.hq = (unpack(one["hc"].cpu().numpy()), one["hs"].cpu().numpy())
    c.htype = "bf16"
    c.check_gateup(one["h"], c.some(24))
    c.check_down(one["p"], c.some(24))
    assert torch.allclose(one["y"].double(), one["p"].double().sum(1), rtol=0, atol=float(
        one["p"].abs().double().sum(1).max()) * k * 2.0 ** -23)


@pytest.mark.parametrize("xtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,F,E,k", [(32, 512, 512, 256, 8), (8, 1024, 1536, 64, 8), (20, 288, 1440, 200, 8),
                                       (2, 2080, 4128, 16, 8)])
def test_layer_of_many_units(T, H, F, E, k, xtype):
    """More than eight work units to a CTA: queue, publication and ring slots are used several times."""
    l = Layer(T, H, 32, E, k, seed=T, xtype=xtype) if H < 1024 else Layer(T, H, 32, 8, k, seed=T, xtype=xtype)
    rng = np.random.default_rng(F)
    l.ex, l.F, l.E = SharedExperts(rng, E, H, F, 3), F, E
    pool, l.sb = l.ex.pool()
    l.pool, l.table, l.n_slots = dev(pool.reshape(-1)), dev(l.ex.table), 3
    l.wr = (rng.standard_normal((H, E)) / H ** 0.5).astype(np.float16)
    l.d_wr = dev(l.wr)
    l.bias = rng.standard_normal(E).astype(np.float32)
    l.ws = torch.full((L.moe_mx4_layer_workspace(T, H, F, E, k),), 0xFF, dtype=torch.uint8, device="cuda")
    y, ids, w = l.run()
    l.check(y, ids, w, tokens=sorted({0, T // 2, T - 1}))
    for _ in range(3):
        assert torch.equal(l.run()[0], y)
    assert L.moe_device_status() == 0
