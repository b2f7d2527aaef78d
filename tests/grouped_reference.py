"""Plain 64-bit forms of the products whose rows choose their matrix, with bounds on what fp32 sums may differ by.

A product of 16-bit values is exact in fp32.  A sum of n of them in fp32, in any order, each addition off by at most a
unit in the last place (2^-23 of the partial sum, whichever way it rounds), is off by at most (n + 16) 2^-23 of the
sum of the magnitudes: that sum is computed beside each product.
"""
import numpy as np
import torch

from routed_expert_ffn_gemv_gb300 import _lib as L

TYPES = {"f32": (L.MOE_F32, torch.float32), "bf16": (L.MOE_BF16, torch.bfloat16), "f16": (L.MOE_F16, torch.float16)}
# half a step of a type, relative, and its smallest step halved
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}


def code(t):
    return TYPES[t][0]


def dtype(t):
    return TYPES[t][1]


def group(ids, G):
    """offsets [G + 1] and rows [n] of int ids, counted one group at a time."""
    ids = np.asarray(ids)
    offsets, rows = [0], []
    for g in range(G):
        mine = np.nonzero(ids == g)[0].tolist()
        rows += mine
        offsets.append(len(rows))
    return np.array(offsets, np.int32), np.array(rows + [-1] * (ids.size - len(rows)), np.int32)


def rounded(value, err, out):
    """Bound on a result of magnitude |value| that is off by `err` before it is rounded to `out`."""
    return err + HALF[out] * (value.abs() + err) + TINY[out]


def product(x, w):
    """x [n, K] times w [N, K] transposed, in 64 bits, and the bound on an fp32 sum."""
    x, w = x.double(), w.double()
    return x @ w.T, (x.shape[1] + 16) * 2.0 ** -23 * (x.abs() @ w.abs().T)


def swiglu(g, eg, u, eu):
    """silu(g) * u and its bound: |silu'| <= 1.1, and 17 units of 2^-24 for its evaluation in fp32."""
    s = g * torch.sigmoid(g)
    h = s * u
    err = 1.1 * eg * (u.abs() + eu) + s.abs() * eu
    return h, err + 17 * 2.0 ** -24 * (h.abs() + err) + 2.0 ** -126


def check(got, value, bound, what=""):
    """Every finite element within its bound."""
    d = (got.double() - value).abs()
    bad = ~(d <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), float((d / bound)[bad].max()), bad.nonzero()[:4].tolist())
