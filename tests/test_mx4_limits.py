"""MXFP4 on the host: limits of sizes (no GPU)."""
import ctypes

import numpy as np
import pytest

import mx4_reference as ref
from routed_expert_ffn_gemv_gb300 import _build, _lib as L


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return L.load()


@pytest.fixture(scope="module")
def ptr():
    a = np.zeros(4096 + 256, np.uint8)
    ptr.keep = a
    return a.ctypes.data + (-a.ctypes.data) % 256


def layer(lib, p, T, H, F, E, k=1):
    """A layer call whose sizes are refused before anything is read."""
    return lib.moe_mx4_layer(p, L.MOE_F32, T, H, F, E, k, p, None, None, 1, p, ref.slot_bytes(H, F), None, p, None, None, p,
                             1 << 50, None)


@pytest.mark.parametrize("T,E", [(1, 1), (16, 8), (16, 256), (17, 1), (32, 8), (32, 250)])
def test_layer_refuses_rows_past_the_routers_shared_memory(lib, ptr, T, E):
    most = (409600 if T <= 16 else 204800) - 72 * ((E + 7) // 8 * 8)
    H = most // 32 * 32 + 32
    assert layer(lib, ptr, T, H, 32, E) == L.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("E,k", [(1, 1), (8, 8), (96, 8), (128, 1), (129, 8), (256, 3), (256, 8)])
def test_workspaces_grow_with_the_call(lib, E, k):
    """A workspace of a larger call serves every smaller one of the same experts."""
    most = 0
    for T in list(range(1, 700)) + [1000, 1023, 1024, 2047, 2048, 2049, 4095, 4096, 20000]:
        n = L.moe_mx4_expert_workspace(T, 160, 96, E, k)
        assert n >= most, T
        most = n
    for H, F in ((32, 32), (128, 96), (160, 64)):
        assert L.moe_mx4_expert_workspace(20000, H, F, E, k) <= most
    most = 0
    for T in range(1, L.MOE_DECODE_MAX_T + 1):
        n = L.moe_mx4_layer_workspace(T, 160, 96, E, k)
        assert n >= most, T
        most = n


def cache_desc(ptr, **kw):
    images = (ctypes.c_void_p * 4)(*[ptr] * 4)
    d = L.CacheDesc(qtype=L.MOE_MXFP4, H=128, F=64, n_layers=1, n_experts=4, first_layer=0, n_slots=4,
                    slot_bytes=ref.slot_bytes(128, 64), device_pool=ptr, host_images=images)
    for k, v in kw.items():
        setattr(d, k, v)
    d.keep = images
    return d


@pytest.mark.parametrize("admit_after", [2, 7])
def test_pool_refuses_admission_of_experts_that_only_stay_on_the_host(lib, ptr, admit_after):
    """A bypassed expert would be read from its pinned image, which no MXFP4 call does."""
    out = ctypes.c_void_p()
    d = cache_desc(ptr, admit_after=admit_after)
    assert lib.moe_cache_create(ctypes.byref(d), ctypes.byref(out)) == L.MOE_ERR_UNSUPPORTED
    assert not out.value


@pytest.mark.parametrize("H,F", [(32, (1 << 28) + 32), ((1 << 28) + 32, 32), (32, (1 << 31) - 32), ((1 << 31) - 32, 64)])
def test_calls_refuse_rows_past_their_offsets(lib, ptr, H, F):
    """A row of h of 2^29 fp32 elements has more bytes than the kernels' row offsets, and (2^31 rounded up to a
    tile) is no int."""
    out, sb = ctypes.c_size_t(), 1 << 46
    un = L.MOE_ERR_UNSUPPORTED
    assert lib.moe_mx4_expert_workspace(4, H, F, 4, 2, ctypes.byref(out)) == un
    assert lib.moe_mx4_layer_workspace(4, H, F, 4, 2, ctypes.byref(out)) == un
    assert lib.moe_mx4_expert_gateup(ptr, ptr, 4, H, F, 4, 2, ptr, None, 4, ptr, sb, ptr, L.MOE_F32, ptr, sb, None) == un
    assert lib.moe_mx4_expert_down(ptr, ptr, 4, H, F, 4, 2, ptr, ptr, None, 4, ptr, sb, ptr, ptr, sb, None) == un
    assert lib.moe_mx4_layer(ptr, L.MOE_F32, 4, H, F, 4, 2, ptr, None, None, 4, ptr, sb, None, ptr, None, None, ptr, sb,
                             None) == un
    assert lib.moe_mx4_expert_workspace(4, 32, 1 << 28, 4, 2, ctypes.byref(out)) == L.MOE_OK


def test_image_size_of_the_longest_rows(lib):
    """Rows rounded up to a tile do not wrap."""
    n = (1 << 31) - 32
    assert L.moe_slot_image_bytes(L.MOE_MXFP4, 32, n) == ((1 << 25) + (1 << 24)) * 8704
    assert L.moe_slot_image_bytes(L.MOE_MXFP4, n, 32) == ((1 << 24) + (1 << 24)) * 8704
