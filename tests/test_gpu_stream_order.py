"""Router calls take the weights and the bias that the stream's previous kernel wrote."""
import pytest

from routed_expert_ffn_gemv_gb300 import _lib as L

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("last", ["weights", "bias"])
@pytest.mark.parametrize("T,H,E,off", [(1, 2048, 128, 0), (8, 1024, 256, 0), (5, 1024, 37, 1), (40, 1024, 64, 0)])
def test_router_inputs_of_the_kernel_before(T, H, E, off, last):
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x = torch.randn(T, H, generator=g, device="cuda")
    wf = torch.randn(H * E, generator=g, device="cuda") / H ** 0.5
    bf = torch.randn(E, generator=g, device="cuda")
    w = torch.zeros(H * E + off, dtype=torch.float16, device="cuda")[off:]
    b = torch.zeros(E, device="cuda")
    k = 4
    ids, wt = torch.zeros(2, T, k, dtype=torch.int32, device="cuda"), torch.zeros(2, T, k, device="cuda")
    logits = torch.zeros(2, T, E, device="cuda")

    def call(i):
        L.moe_router_topk(x, L.MOE_F32, T, H, w, b, E, k, ids[i], wt[i], logits[i])

    w.copy_(wf)
    b.copy_(bf)
    torch.cuda.synchronize()
    call(0)
    torch.cuda.synchronize()
    want = x.double() @ w.reshape(H, E).double() + b.double()
    assert float((logits[0].double() - want).abs().max()) < 1e-4
    for i in range(20):
        w.zero_()
        b.zero_()
        if last == "weights":
            b.copy_(bf)
            w.copy_(wf)
        else:
            w.copy_(wf)
            b.add_(bf)
        call(1)
        assert torch.equal(ids[1], ids[0]) and torch.equal(wt[1], wt[0]) and torch.equal(logits[1], logits[0]), i


def test_router_calls_of_two_threads():
    """Two host threads with routers of different sizes, a stream each."""
    import threading
    errors = []

    def work(H, E, seed):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                g = torch.Generator(device="cuda")
                g.manual_seed(seed)
                x = torch.randn(4, H, generator=g, device="cuda")
                w = (torch.randn(H, E, generator=g, device="cuda") / H ** 0.5).half()
                ids, wt = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, 2, device="cuda")
                for _ in range(500):
                    L.moe_router_topk(x, L.MOE_F32, 4, H, w, None, E, 2, ids, wt, None, s)
                logits = x.double() @ w.double()
            s.synchronize()
            if not torch.equal(torch.topk(logits, 2).indices.int(), ids):
                errors.append("ids")
        except Exception as e:  # handed to the main thread
            errors.append(repr(e))

    threads = [threading.Thread(target=work, args=a) for a in ((2048, 128, 1), (256, 8, 2), (1024, 128, 3))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
