"""The 16-bit products whose rows choose their matrix on the host: refusals before any device work (no GPU)."""
import ctypes

import numpy as np
import pytest

from routed_expert_ffn_gemv_gb300 import _build, _lib as L

BAD, NO = L.MOE_ERR_INVALID, L.MOE_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return L.load()


@pytest.fixture(scope="module")
def ptr():
    a = np.zeros(4096 + 256, np.uint8)
    ptr.keep = a
    return a.ctypes.data + (-a.ctypes.data) % 256


def call(f, defaults, **kw):
    args = dict(defaults, **kw)
    assert args.keys() == defaults.keys()
    return f(*args.values())


def matmul_args(p):
    return dict(x=p, type=L.MOE_BF16, x_rows=4, ldx=64, x_index=None, x_share=1, offsets=p, G=2, R=4, w=p, w_order=0, N=32, K=64,
                act=0, scale=None, y_index=None, y=p, ytype=L.MOE_F32, y_rows=4, ldy=32, s=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(type=L.MOE_F32), BAD), (dict(type=3), BAD), (dict(ytype=3), BAD), (dict(ytype=-1), BAD), (dict(w_order=2), BAD),
    (dict(act=2), BAD), (dict(act=-1), BAD), (dict(G=0), BAD), (dict(G=513), BAD), (dict(R=-1), BAD), (dict(R=(1 << 24) + 1), BAD),
    (dict(N=0), BAD), (dict(K=0), BAD), (dict(N=36, ldy=40), NO), (dict(K=60), NO), (dict(N=65544, ldy=65544), NO),
    (dict(K=65544, ldx=65544), NO), (dict(ldx=56), BAD), (dict(ldx=68), BAD), (dict(ldy=24), BAD), (dict(ldy=36), BAD),
    (dict(ldx=(1 << 32) + 8), BAD), (dict(x_rows=-1), BAD), (dict(y_rows=-1), BAD), (dict(x_rows=0), BAD), (dict(y_rows=0), BAD),
    (dict(act=1, w_order=1), NO), (dict(x=None), BAD), (dict(offsets=None), BAD), (dict(w=None), BAD), (dict(y=None), BAD),
    (dict(R=0, x=None, offsets=None, w=None, y=None), L.MOE_OK),
])
def test_matmul_refusals(lib, ptr, kw, rc):
    assert call(lib.moe_grouped_matmul, matmul_args(ptr), **kw) == rc


def test_matmul_refuses_misaligned_buffers_and_no_share(lib, ptr):
    for name in ("x", "w", "y"):
        assert call(lib.moe_grouped_matmul, matmul_args(ptr), **{name: ptr + 8}) == BAD
    assert call(lib.moe_grouped_matmul, matmul_args(ptr), scale=ptr + 2) == BAD
    assert call(lib.moe_grouped_matmul, matmul_args(ptr), x_index=ptr, x_share=0) == BAD


def grad_args(p):
    return dict(x=p, type=L.MOE_F16, x_rows=4, ldx=64, x_index=None, x_share=1, dy=p, dy_rows=4, lddy=32, dy_index=None, offsets=p,
                G=2, R=4, N=32, K=64, accumulate=0, dw=p, wtype=L.MOE_F32, s=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(type=L.MOE_F32), BAD), (dict(wtype=3), BAD), (dict(accumulate=2), BAD), (dict(G=0), BAD), (dict(G=513), BAD),
    (dict(R=-1), BAD), (dict(R=(1 << 24) + 1), BAD), (dict(N=36, lddy=40), NO), (dict(K=4), NO), (dict(ldx=56), BAD),
    (dict(lddy=24), BAD), (dict(lddy=36), BAD), (dict(x=None), BAD), (dict(dy=None), BAD), (dict(dw=None), BAD),
    (dict(offsets=None), BAD), (dict(x_rows=0), BAD), (dict(dy_rows=0), BAD), (dict(R=0, accumulate=1, x=None, dy=None), L.MOE_OK),
])
def test_weight_gradient_refusals(lib, ptr, kw, rc):
    assert call(lib.moe_grouped_weight_grad, grad_args(ptr), **kw) == rc


def test_weight_gradient_refuses_misaligned_buffers(lib, ptr):
    for name in ("x", "dy", "dw"):
        assert call(lib.moe_grouped_weight_grad, grad_args(ptr), **{name: ptr + 8}) == BAD
    assert call(lib.moe_grouped_weight_grad, grad_args(ptr), x_index=ptr, x_share=0) == BAD


def lora_args(p):
    return dict(x=p, type=L.MOE_BF16, T=4, ldx=64, w=p, N=32, K=64, adapter=p, n_adapters=2, a=p, b=p, rank=8, scale=None, y=p,
                ytype=L.MOE_BF16, ldy=32, workspace=p, ws_bytes=1 << 20, s=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(type=L.MOE_F32), BAD), (dict(ytype=3), BAD), (dict(T=-1), BAD), (dict(T=(1 << 24) + 1), BAD), (dict(rank=0), BAD),
    (dict(rank=12), NO), (dict(rank=264), NO), (dict(n_adapters=0), BAD), (dict(N=36, ldy=40), NO), (dict(K=60), NO),
    (dict(N=65544, ldy=65544), NO), (dict(ldx=56), BAD), (dict(ldy=24), BAD), (dict(ldy=36), BAD), (dict(ws_bytes=511), BAD),
    (dict(workspace=None), BAD), (dict(x=None), BAD), (dict(w=None), BAD), (dict(adapter=None), BAD), (dict(a=None), BAD),
    (dict(b=None), BAD), (dict(y=None), BAD), (dict(T=0, x=None, w=None, y=None, workspace=None), L.MOE_OK),
])
def test_lora_refusals(lib, ptr, kw, rc):
    assert call(lib.moe_lora_matmul, lora_args(ptr), **kw) == rc


def test_lora_refuses_misaligned_buffers(lib, ptr):
    for name in ("x", "w", "a", "b", "y"):
        assert call(lib.moe_lora_matmul, lora_args(ptr), **{name: ptr + 8}) == BAD
    assert call(lib.moe_lora_matmul, lora_args(ptr), workspace=ptr + 128) == BAD


def test_group_rows_refusals(lib, ptr):
    f = lib.moe_group_rows
    assert f(None, 4, 2, ptr, ptr, None, 0, None) == BAD
    assert f(ptr, 4, 2, None, ptr, None, 0, None) == BAD
    assert f(ptr, 4, 2, ptr, None, None, 0, None) == BAD
    assert f(ptr, -1, 2, ptr, ptr, None, 0, None) == BAD
    assert f(ptr, 4, 0, ptr, ptr, None, 0, None) == BAD
    assert f(ptr, 4, 513, ptr, ptr, None, 0, None) == BAD
    n = 1 << 18
    need = L.moe_group_rows_workspace(n, 512)
    assert need > 0
    assert f(ptr, n, 512, ptr, ptr, None, need, None) == BAD
    assert f(ptr, n, 512, ptr, ptr, ptr, need - 1, None) == BAD
    assert f(ptr, n, 512, ptr, ptr, ptr + 2, need, None) == BAD


def test_workspaces(lib):
    out = ctypes.c_size_t()
    assert L.moe_group_rows_workspace(32768, 512) == 0
    assert lib.moe_group_rows_workspace((1 << 24) + 1, 2, ctypes.byref(out)) == BAD
    assert lib.moe_group_rows_workspace(4, 2, None) == BAD
    assert lib.moe_lora_workspace(4, 8, None) == BAD
    most = 0
    for T in (1, 2, 31, 64, 65, 4096):
        n = L.moe_lora_workspace(T, 64)
        assert n > most
        most = n
    assert L.moe_lora_workspace(4096, 8) <= L.moe_lora_workspace(4096, 64) <= L.moe_lora_workspace(4096, 256)


def test_other_calls_refuse_fp16_rows(lib, ptr):
    """MOE_F16 is a type of these products only."""
    assert lib.moe_router_topk(ptr, L.MOE_F16, 1, 64, ptr, None, 4, 1, ptr, ptr, None, None) == BAD
    assert lib.moe_mx4_quantize(ptr, L.MOE_F16, 1, 32, 32, ptr, ptr, None) == BAD
    assert lib.moe_expert_ffn(ptr, L.MOE_F16, 1, 64, 64, 0, 4, 1, ptr, ptr, None, 4, ptr, 1 << 20, None, 0, ptr, ptr, 1 << 20,
                              None) == BAD
