"""What the microscaled 4-bit (MXFP4) operators compute, at the sizes they are measured at.

Each case names one of the library's operators and its sizes:

  quantize   rows of activations to MXFP4 and back        (moe_mx4_quantize, moe_mx4_dequantize)
  experts    a layer's expert weights to slot images, back (moe_mx4_quantize_experts, ..._dequantize_experts)
  gateup     the routed experts' gate/up product + SwiGLU  (moe_mx4_expert_gateup)
  down       the routed experts' weighted down product     (moe_mx4_expert_down)
  layer      router, top-k, expert FFN and combine          (moe_mx4_layer)

``run`` computes a case either in plain torch operations (``own`` false) or through the library.
Layer shapes are the library's own configurations (Granite-, Qwen3-30B-A3B- and
DeepSeek-16B-shaped: H, F, E, k) and ragged sizes around them.
"""
import math
import random

import numpy as np
import torch

own = False

# The eight magnitudes of an E2M1 code, in code order (bit 3 of a code is the sign).
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_F32, _BF16 = 0, 1


def listed():
    return [
        # a decode step's activations: latency
        {"name": "quantize-8x2048-bf16", "op": "quantize", "rows": 8, "cols": 2048, "pad": 0, "dtype": "bf16"},
        # a prompt's activations, rows of a wider buffer
        {"name": "quantize-4096x2048-bf16", "op": "quantize", "rows": 4096, "cols": 2048, "pad": 64, "dtype": "bf16"},
        # loading a Granite-shaped layer's checkpoint weights
        {"name": "experts-32-h1024-f512-bf16", "op": "experts", "n": 32, "H": 1024, "F": 512, "dtype": "bf16"},
        # loading a Qwen-shaped layer from fp32 weights
        {"name": "experts-128-h2048-f768-f32", "op": "experts", "n": 128, "H": 2048, "F": 768, "dtype": "f32"},
        # a single token through a Qwen-shaped layer
        {"name": "gateup-1-qwen", "op": "gateup", "T": 1, "H": 2048, "F": 768, "E": 128, "k": 8, "dtype": "f32"},
        # a ragged small batch, DeepSeek-shaped
        {"name": "gateup-77-deepseek", "op": "gateup", "T": 77, "H": 2048, "F": 1408, "E": 64, "k": 2, "dtype": "bf16"},
        # a long prompt, Qwen-shaped
        {"name": "gateup-4096-qwen", "op": "gateup", "T": 4096, "H": 2048, "F": 768, "E": 128, "k": 8, "dtype": "bf16"},
        # a ragged decode batch, Granite-shaped
        {"name": "down-19-granite", "op": "down", "T": 19, "H": 1024, "F": 512, "E": 32, "k": 8},
        # a long prompt, Qwen-shaped
        {"name": "down-4096-qwen", "op": "down", "T": 4096, "H": 2048, "F": 768, "E": 128, "k": 8},
        # a single sequence's decode step, Granite-shaped
        {"name": "layer-1-granite", "op": "layer", "T": 1, "H": 1024, "F": 512, "E": 32, "k": 8, "dtype": "f32"},
        # eight sequences' decode step, Qwen-shaped
        {"name": "layer-8-qwen", "op": "layer", "T": 8, "H": 2048, "F": 768, "E": 128, "k": 8, "dtype": "bf16"},
        # the largest decode batch, DeepSeek-shaped
        {"name": "layer-32-deepseek", "op": "layer", "T": 32, "H": 2048, "F": 1408, "E": 64, "k": 2, "dtype": "f32"},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "experts", "gateup", "down", "layer"])
    dtype = rng.choice(["f32", "bf16"])
    H, F = 32 * rng.randint(8, 64), 32 * rng.randint(4, 24)
    E = _log_uniform(rng, 8, 128)
    k = rng.randint(1, 8)
    if op == "quantize":
        return {"op": op, "rows": _log_uniform(rng, 1, 4096), "cols": 32 * _log_uniform(rng, 1, 64),
                "pad": 8 * rng.randint(0, 8), "dtype": dtype}
    if op == "experts":
        return {"op": op, "n": _log_uniform(rng, 1, 128), "H": H, "F": F, "dtype": dtype}
    if op == "layer":
        return {"op": op, "T": _log_uniform(rng, 1, 32), "H": H, "F": F, "E": E, "k": k, "dtype": dtype}
    T = _log_uniform(rng, 1, 4096)
    if op == "down":
        return {"op": op, "T": T, "H": H, "F": F, "E": E, "k": k}
    return {"op": op, "T": T, "H": H, "F": F, "E": E, "k": k, "dtype": dtype}


# ------------------------------------------------------------------------------ the format, plain

def _quantise(x):
    """MXFP4 of rows x [..., K], K a multiple of 32: codes [..., K] and E8M0 scale bytes
    [..., K/32], uint8.  The scale is 2^(floor(log2 max|x|) - 2), codes round to nearest even."""
    blocks = x.float().reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    amax = blocks.abs().amax(-1)
    exponent = torch.frexp(amax).exponent - 1  # floor(log2 amax); -1 for amax 0
    byte = torch.where(amax > 0, exponent - 2 + 127, torch.zeros_like(exponent)).clamp(0, 254)
    v = torch.ldexp(blocks.double(), (127 - byte).double().unsqueeze(-1)).abs()
    code = ((v > 0.25).int() + (v >= 0.75).int() + (v > 1.25).int() + (v >= 1.75).int()
            + (v > 2.5).int() + (v >= 3.5).int() + (v > 5.0).int())
    code = torch.where(torch.signbit(blocks), code + 8, code)
    return code.reshape(x.shape).to(torch.uint8), byte.to(torch.uint8)


def _dequantise(codes, scales):
    """fp32 values of unpacked codes [..., K] and scale bytes [..., K/32]."""
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float32, device=codes.device)
    v = table[codes.int()].reshape(*scales.shape, 32)
    return torch.ldexp(v, (scales.float() - 127.0).unsqueeze(-1)).reshape(codes.shape)


def _pack(codes):
    """Two codes to a byte, the even element in the low nibble."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _unpack(packed):
    return torch.stack((packed & 15, packed >> 4), -1).reshape(*packed.shape[:-1], packed.shape[-1] * 2)


def _tiles(codes, scales):
    """Packed codes [n, R, K/2] and scales [n, R, K/32] of n matrices in the slot image's order:
    128-row tiles of 128-column blocks of 8704 bytes (see moe_mx4_quantize_experts)."""
    n, R, Kb = codes.shape
    G, B = -(-R // 128), -(-Kb // 64)
    c = codes.new_zeros(n, G * 128, B * 64)
    c[:, :R, :Kb] = codes
    s = scales.new_zeros(n, G * 128, B * 4)
    s[:, :R, :Kb // 16] = scales
    c = c.reshape(n, G, 128, B, 4, 16).permute(0, 1, 3, 2, 4, 5)
    row = torch.arange(128, device=c.device)
    place = torch.arange(4, device=c.device)[None, :] ^ ((row[:, None] >> 1) & 3)
    c = c[:, :, :, row[:, None], place, :].reshape(n, G, B, 8192)
    s = s.reshape(n, G, 4, 32, B, 4).permute(0, 1, 4, 3, 2, 5).reshape(n, G, B, 512)
    return torch.cat((c, s), -1).reshape(n, -1)


def _images(gate, up, down):
    """Slot images [n, bytes] of experts given as (packed codes, scales) pairs: gate and up rows
    interleaved by 64, then down."""
    n, F = gate[0].shape[:2]

    def both(a, b):
        T = -(-F // 64)
        z = a.new_zeros(n, 2, T * 64, a.shape[-1])
        z[:, 0, :F], z[:, 1, :F] = a, b
        return z.reshape(n, 2, T, 64, -1).transpose(1, 2).reshape(n, T * 128, -1)

    return torch.cat((_tiles(both(gate[0], up[0]), both(gate[1], up[1])), _tiles(*down)), 1)


# ------------------------------------------------------------------------------ inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _weights(g, n, R, K):
    """n matrices [R, K] of the size a trained projection has, as packed codes and scales."""
    w = torch.randn(n, R, K, generator=g, device="cuda") / math.sqrt(K)
    codes, scales = _quantise(w)
    return _pack(codes), scales


def _routes(g, T, E, k):
    """Router logits with the spread and the popularity skew of the layers' routers."""
    rank = torch.randperm(E, generator=g, device="cuda") + 1
    logits = 3.0 * torch.randn(T, E, generator=g, device="cuda") - 1.1 * rank.float().log()
    top = torch.topk(logits, k, dim=1)
    return top.indices.int().contiguous(), torch.softmax(top.values, 1).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op = case["op"]
    s = {"case": case, "stream": torch.cuda.current_stream().cuda_stream}
    if op == "quantize":
        rows, cols, dt = case["rows"], case["cols"], _dtype(case)
        wide = torch.randn(rows, cols + case["pad"], generator=g, device="cuda").to(dt)
        s["x"] = wide[:, :cols]
        s["codes"] = torch.empty(rows, cols // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(rows, cols // 32, dtype=torch.uint8, device="cuda")
        s["y"] = torch.empty(rows, cols, dtype=dt, device="cuda")
        return s
    H, F = case["H"], case["F"]
    if op == "experts":
        n, dt = case["n"], _dtype(case)
        shapes = {"gate": (n, F, H), "up": (n, F, H), "down": (n, H, F)}
        for name, shape in shapes.items():
            s[name] = (torch.randn(shape, generator=g, device="cuda") / math.sqrt(shape[2])).to(dt)
            s["out_" + name] = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        s["slot_bytes"] = _slot_bytes(H, F)
        s["pool"] = torch.empty(n * s["slot_bytes"], dtype=torch.uint8, device="cuda")
        return s
    T, E, k = case["T"], case["E"], min(case["k"], case["E"])
    s["k"] = k
    s["gate"], s["up"], s["down"] = _weights(g, E, F, H), _weights(g, E, F, H), _weights(g, E, H, F)
    # the experts' slots in their pool, in the order of their uploads
    s["table"] = torch.randperm(E, generator=g, device="cuda").int()
    s["slot_bytes"] = _slot_bytes(H, F)
    pool = torch.zeros(E, s["slot_bytes"], dtype=torch.uint8, device="cuda")
    image = _images(s["gate"], s["up"], s["down"])
    pool[s["table"].long(), :image.shape[1]] = image
    s["pool"] = pool.reshape(-1)
    if op == "layer":
        s["x"] = torch.randn(T, H, generator=g, device="cuda").to(_dtype(case))
        s["w_router"] = (torch.randn(H, E, generator=g, device="cuda") * H ** -0.25).half()
        rank = torch.randperm(E, generator=g, device="cuda") + 1
        s["bias"] = -1.1 * rank.float().log()
        s["extra"] = torch.randn(T, H, generator=g, device="cuda")
        s["y"] = torch.empty(T, H, device="cuda")
        return s
    s["ids"], s["weights"] = _routes(g, T, E, k)
    if op == "gateup":
        codes, s["scales"] = _quantise(torch.randn(T, H, generator=g, device="cuda"))
        s["h"] = torch.empty(T * k, F, dtype=_dtype(case), device="cuda")
    else:
        a = torch.randn(T * k, F, generator=g, device="cuda")
        codes, s["scales"] = _quantise(a * torch.sigmoid(a) * torch.randn(T * k, F, generator=g, device="cuda"))
        s["partial"] = torch.empty(T, k, H, device="cuda")
    s["codes"] = _pack(codes)
    return s


def _slot_bytes(H, F):
    """A slot image's size, rounded up to the pools' 256 bytes."""
    blocks = -(-F // 64) * -(-H // 128) + -(-H // 128) * -(-F // 128)
    return -(-blocks * 8704 // 256) * 256


# ------------------------------------------------------------------------------ one pass

def _grouped(x, of, ids, w):
    """Per route r with expert ids[r]: w[expert] @ x[of[r]], as one batched product over the
    experts in use, their rows padded to the fullest one.  w: codes and scales of [E, R, K]."""
    used, expert = torch.unique(ids.long(), return_inverse=True)
    order = torch.argsort(expert, stable=True)
    count = torch.bincount(expert, minlength=used.numel())
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device) - (count.cumsum(0) - count)[expert[order]]
    rows = x.new_zeros(used.numel(), int(count.max()), x.shape[1])
    rows[expert, place] = x[of]
    values = _dequantise(_unpack(w[0][used]), w[1][used])
    return torch.bmm(rows, values.transpose(1, 2))[expert, place]


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "quantize":
        codes, scales = _quantise(s["x"])
        return _dequantise(codes, scales).to(s["x"].dtype)
    if op == "experts":
        gate, up, down = _quantise(s["gate"]), _quantise(s["up"]), _quantise(s["down"])
        return {"gate": _dequantise(*gate).bfloat16(), "up": _dequantise(*up).bfloat16(),
                "down": _dequantise(*down).bfloat16()}
    T, k = case["T"], s["k"]
    routes = torch.arange(T * k, device="cuda")
    if op == "down":
        h = _dequantise(_unpack(s["codes"]), s["scales"])
        return (_grouped(h, routes, s["ids"].reshape(-1), s["down"]) * s["weights"].reshape(-1, 1)).reshape(T, k, -1)
    if op == "gateup":
        x, ids = _dequantise(_unpack(s["codes"]), s["scales"]), s["ids"].reshape(-1)
    else:
        x = s["x"].float()
        logits = s["x"].double() @ s["w_router"].double() + s["bias"].double()
        top = torch.sort(logits, dim=1, descending=True, stable=True)
        chosen, ids = top.values[:, :k], top.indices[:, :k].reshape(-1)
        weights = torch.exp(chosen - chosen[:, :1])
        weights = (weights / weights.sum(1, keepdim=True)).float()
    gate, up = _grouped(x, routes // k, ids, s["gate"]), _grouped(x, routes // k, ids, s["up"])
    h = gate / (1.0 + torch.exp(-gate)) * up
    if op == "gateup":
        return h.to(_dtype(case))
    partial = _grouped(h, routes, ids, s["down"]).reshape(T, k, -1)
    return s["extra"] + (partial * weights.unsqueeze(-1)).sum(1)


def _run_own(s):
    from routed_expert_ffn_gemv_gb300 import _lib as L
    case, st = s["case"], s["stream"]
    op = case["op"]
    if op == "quantize":
        rows, cols, t = case["rows"], case["cols"], _BF16 if case["dtype"] == "bf16" else _F32
        L.moe_mx4_quantize(s["x"], t, rows, cols, cols + case["pad"], s["codes"], s["scales"], st)
        L.moe_mx4_dequantize(s["codes"], s["scales"], rows, cols, s["y"], t, cols, st)
        return s["y"]
    H, F = case["H"], case["F"]
    if op == "experts":
        n, t = case["n"], _BF16 if case["dtype"] == "bf16" else _F32
        L.moe_mx4_quantize_experts(s["gate"], s["up"], s["down"], t, n, H, F, s["pool"], s["slot_bytes"], None, n, st)
        L.moe_mx4_dequantize_experts(s["pool"], s["slot_bytes"], None, n, n, H, F, s["out_gate"], s["out_up"],
                                     s["out_down"], _BF16, st)
        return {"gate": s["out_gate"], "up": s["out_up"], "down": s["out_down"]}
    T, E, k = case["T"], case["E"], s["k"]
    if "workspace" not in s:  # kept with the other buffers
        size = L.moe_mx4_layer_workspace(T, H, F, E, k) if op == "layer" else L.moe_mx4_expert_workspace(T, H, F, E, k)
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    ws = s["workspace"]
    if op == "layer":
        L.moe_mx4_layer(s["x"], _BF16 if case["dtype"] == "bf16" else _F32, T, H, F, E, k, s["w_router"], s["bias"],
                        s["table"], E, s["pool"], s["slot_bytes"], s["extra"], s["y"], None, None, ws, ws.numel(), st)
        return s["y"]
    if op == "gateup":
        L.moe_mx4_expert_gateup(s["codes"], s["scales"], T, H, F, E, k, s["ids"], s["table"], E, s["pool"],
                                s["slot_bytes"], s["h"], _BF16 if case["dtype"] == "bf16" else _F32, ws, ws.numel(), st)
        return s["h"]
    L.moe_mx4_expert_down(s["codes"], s["scales"], T, H, F, E, k, s["ids"], s["weights"], s["table"], E, s["pool"],
                          s["slot_bytes"], s["partial"], ws, ws.numel(), st)
    return s["partial"]


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


def work(case):
    op = case["op"]
    if op == "quantize":
        n, size = case["rows"] * case["cols"], 2 if case["dtype"] == "bf16" else 4
        # the rows in, codes and scales out, then those in and the values out
        return {"bytes": n * 2 * size + 2 * n * 17 / 32, "flops": 0}
    H, F = case["H"], case["F"]
    if op == "experts":
        n, size = 3 * case["n"] * H * F, 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * (size + 2) + 2 * n * 17 / 32, "flops": 0}
    T, E, k = case["T"], case["E"], min(case["k"], case["E"])
    routes = T * k
    # experts in use with independent uniform routes: what the weights' reads come to
    active = E * (1.0 - (1.0 - k / E) ** T)
    if op == "gateup":
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": active * 2 * H * F * 17 / 32 + T * H * 17 / 32 + routes * F * size, "flops": 4 * routes * H * F}
    if op == "down":
        return {"bytes": active * H * F * 17 / 32 + routes * F * 17 / 32 + routes * H * 4, "flops": 2 * routes * H * F}
    size = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": active * 3 * H * F * 17 / 32 + H * E * 2 + T * H * (size + 8),
            "flops": 6 * routes * H * F + 2 * T * H * E}


# ------------------------------------------------------------------------------ in 64 bits

def _exact_values(packed, scales):
    """float64 values of packed codes, from the bit fields (sign, two exponent bits, one mantissa
    bit; exponent 0 is subnormal)."""
    nib = torch.stack((packed & 15, packed >> 4), -1).flatten(-2).to(torch.int64)
    e, m = (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(e == 0, m * 0.5, (1.0 + 0.5 * m) * (2.0 ** (e - 1).double()))
    v = torch.where(nib >= 8, -mag, mag)
    return v * (2.0 ** (scales.double() - 127.0)).repeat_interleave(32, -1)


def _exact_mx4(x):
    """float64 MXFP4 round trip of x by the nearest of the fifteen values, ties to the even code."""
    b = x.double().reshape(-1, 32)
    amax = b.abs().amax(1, keepdim=True)
    e = torch.floor(torch.log2(amax.clamp_min(2.0 ** -149)))
    e = torch.where(2.0 ** e > amax, e - 1, e)          # a rounded log2 must not pass a power of two
    e = torch.where(2.0 ** (e + 1) <= amax, e + 1, e)
    scale = 2.0 ** (e - 2).clamp(-127, 127)
    v = (b / scale).abs().clamp_max(6.0)
    # steps of 0.5 below 2, 1 below 4, 2 above; torch.round takes ties to even multiples
    step = torch.where(v < 2.0, 0.5, torch.where(v < 4.0, 1.0, 2.0)).double()
    return (torch.round(v / step) * step * torch.sign(b) * scale).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_mx4(s["x"].contiguous())
    if op == "experts":
        return {name: _exact_mx4(s[name]) for name in ("gate", "up", "down")}
    T, k = case["T"], s["k"]
    if op == "layer":
        x = s["x"].double()
        logits = x @ s["w_router"].double() + s["bias"].double()
        ids = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :k]
        weights = torch.softmax(torch.gather(logits, 1, ids), 1)
    else:
        x = _exact_values(s["codes"], s["scales"])
        ids, weights = s["ids"].long(), s["weights"].double()
    out = torch.zeros(T * k, case["F"] if op == "gateup" else case["H"], dtype=torch.float64, device="cuda")
    flat = ids.reshape(-1)
    for e in torch.unique(flat).tolist():
        r = (flat == e).nonzero().reshape(-1)
        h = x[r] if op == "down" else x[r // k]
        if op != "down":
            a = h @ _exact_values(s["gate"][0][e], s["gate"][1][e]).T
            b = h @ _exact_values(s["up"][0][e], s["up"][1][e]).T
            h = a * torch.sigmoid(a) * b
        if op != "gateup":
            h = (h @ _exact_values(s["down"][0][e], s["down"][1][e]).T) * weights.reshape(-1)[r, None]
        out[r] = h
    if op == "gateup":
        return out
    out = out.reshape(T, k, -1)
    return out if op == "down" else s["extra"].double() + out.sum(1)
