"""MXFP4 in plain numpy, 64 bits: the format, slot images and the routed experts' products."""
import numpy as np

VALUES = np.array([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
VALUES = np.concatenate([VALUES, -VALUES])
F32_STEP = 2.0 ** -24   # half a step of fp32, relative
BF16_STEP = 2.0 ** -8   # half a step of bf16, relative


def quantise(x):
    """Codes [.., K] and scale bytes [.., K/32] (uint8) of x, the nearest code by distance, ties to
    the even code."""
    x = np.asarray(x)
    b = x.astype(np.float64).reshape(-1, 32)
    codes = np.zeros(b.shape, np.uint8)
    scales = np.zeros(b.shape[0], np.uint8)
    for i, row in enumerate(b):
        if not np.isfinite(row).all():
            scales[i] = 255
            continue
        amax = np.abs(row).max()
        s = 0
        if amax > 0:
            s = max(0, int(np.frexp(amax)[1]) - 1 - 2 + 127)
        scales[i] = s
        v = np.abs(row) * 2.0 ** (127 - s)
        d = np.abs(v[:, None] - VALUES[None, :8])
        best = d.min(axis=1, keepdims=True)
        tie = d == best
        c = np.where(tie[:, ::2].any(axis=1), 2 * tie[:, ::2].argmax(axis=1), tie.argmax(axis=1))
        codes[i] = c + 8 * np.signbit(row)
    return codes.reshape(x.shape), scales.reshape(*x.shape[:-1], x.shape[-1] // 32)


def values(codes, scales):
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (VALUES[codes].reshape(*scales.shape, 32) * s[..., None]).reshape(codes.shape)


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def canonical(codes, scales):
    """Canonical 17-byte blocks of rows [R, K] as a flat byte array."""
    R, K = codes.shape
    out = np.zeros((R, K // 32, 17), np.uint8)
    out[:, :, 0] = scales
    out[:, :, 1:] = pack(codes).reshape(R, K // 32, 16)
    return out.reshape(-1)


def image(gate, up, down):
    """The documented slot image, byte by byte, of (codes, scales) triples."""
    F, H = gate[0].shape
    HB, FB, FT, HT = -(-H // 128), -(-F // 128), -(-F // 64), -(-H // 128)
    out = np.zeros((FT * HB + HT * FB) * 8704, np.uint8)

    def put(base, B, tile_row, codes, scales):
        p = pack(codes)
        for b in range(codes.size // 32):
            tb = base + ((tile_row // 128) * B + b // 4) * 8704
            r, c = tile_row % 128, b % 4
            at = tb + 64 * r + 16 * (c ^ ((r // 2) % 4))
            out[at:at + 16] = p[16 * b:16 * b + 16]
            out[tb + 8192 + 16 * (r % 32) + 4 * (r // 32) + c] = scales[b]

    for f in range(F):
        put(0, HB, f // 64 * 128 + f % 64, gate[0][f], gate[1][f])
        put(0, HB, f // 64 * 128 + f % 64 + 64, up[0][f], up[1][f])
    for h in range(H):
        put(FT * HB * 8704, FB, h, down[0][h], down[1][h])
    return out


def slot_bytes(H, F):
    n = (-(-F // 64) * -(-H // 128) + -(-H // 128) * -(-F // 128)) * 8704
    return -(-n // 256) * 256


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-np.clip(x, -700, 700)))


def accumulation(K):
    """Relative bound, per unit of sum |w x|, of an fp32 sum of K exact products taken at most 32 at
    a time: one rounding (or truncation: a whole step) per 32 products and 64 more in joining."""
    return (K / 32 + 64) * 2 * F32_STEP


def gateup(x, gate, up):
    """h and an elementwise bound of an fp32 evaluation's error, for one token and one expert.
    |silu'| <= 1.1; exp, division and the two products add at most eight roundings of h."""
    g, u = gate @ x, up @ x
    ag, au = np.abs(gate) @ np.abs(x), np.abs(up) @ np.abs(x)
    h = g * sigmoid(g) * u
    a = accumulation(x.size)
    return h, 1.1 * np.abs(u) * a * ag + np.abs(g * sigmoid(g)) * a * au + 1.1 * a * a * ag * au + 8 * F32_STEP * np.abs(h)


class Experts:
    """E random experts: codes and scales of each matrix, values, and the pool's images."""

    def __init__(self, rng, E, H, F, spread=2):
        self.E, self.H, self.F = E, H, F
        self.parts, self.vals = [], []
        for _ in range(E):
            p, v = [], []
            for R, K in ((F, H), (F, H), (H, F)):
                codes = rng.integers(0, 16, (R, K), dtype=np.uint8)
                # 2^-3 .. 2^-3+spread around the size that keeps a product of K terms near one
                scales = rng.integers(0, spread + 1, (R, K // 32)) + 124 - int(np.log2(K)) // 2
                p.append((codes, scales.astype(np.uint8)))
                v.append(values(*p[-1]))
            self.parts.append(p)
            self.vals.append(v)

    def pool(self, table=None, n_slots=None):
        sb = slot_bytes(self.H, self.F)
        out = np.full((n_slots or self.E, sb), 0xA5, np.uint8)
        for e in range(self.E):
            img = image(*self.parts[e])
            out[e if table is None else table[e], :img.size] = img
        return out, sb
