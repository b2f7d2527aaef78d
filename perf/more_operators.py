"""What the products whose rows choose their matrix compute, at the sizes they are measured at.

Each case names one of the library's operators and its sizes:

  group   the rows of each group from the rows' group ids       (moe_group_rows)
  matmul  products of ragged groups of rows, a matrix each:     (moe_grouped_matmul)
          the routed experts' gate/up with SwiGLU, their weighted down product, an input gradient
  grad    the matrices' gradient                                (moe_grouped_weight_grad)
  lora    a shared projection plus each token's low-rank adapter (moe_lora_matmul)

``run`` computes a case either in plain torch operations (``own`` false) or through the library.
Layer shapes are the library's own configurations (Granite-, Qwen3-30B-A3B- and
DeepSeek-16B-shaped: H, F, E, k) and ragged sizes around them.
"""
import math

import torch

own = False

_TYPES = {"f32": (0, torch.float32), "bf16": (1, torch.bfloat16), "f16": (2, torch.float16)}
_NK, _KN = 0, 1               # order of a matrix: [N][K] or [K][N]
_NONE, _SWIGLU = 0, 1         # what is done to a product's rows


def listed():
    return [
        # one token's routes: latency
        {"name": "group-8-qwen", "op": "group", "T": 1, "E": 128, "k": 8, "drop": 0.0},
        # a long prompt's routes, the light ones dropped by the router's threshold
        {"name": "group-32768-qwen", "op": "group", "T": 4096, "E": 128, "k": 8, "drop": 0.05},
        # a single token's gate/up product, Qwen-shaped
        {"name": "gateup-1-qwen", "op": "matmul", "form": "gateup", "T": 1, "H": 2048, "F": 768, "E": 128, "k": 8,
         "drop": 0.0, "dtype": "bf16", "out": "bf16"},
        # a ragged decode batch's down product, Granite-shaped
        {"name": "down-19-granite", "op": "matmul", "form": "down", "T": 19, "H": 1024, "F": 512, "E": 32, "k": 8,
         "drop": 0.05, "dtype": "f16", "out": "f32"},
        # a ragged small batch, DeepSeek-shaped
        {"name": "gateup-77-deepseek", "op": "matmul", "form": "gateup", "T": 77, "H": 2048, "F": 1408, "E": 64,
         "k": 2, "drop": 0.0, "dtype": "f16", "out": "f16"},
        # a long prompt's gate/up product, Qwen-shaped
        {"name": "gateup-4096-qwen", "op": "matmul", "form": "gateup", "T": 4096, "H": 2048, "F": 768, "E": 128,
         "k": 8, "drop": 0.0, "dtype": "bf16", "out": "bf16"},
        # the gradient of that product's input in a training step
        {"name": "dx-4096-qwen", "op": "matmul", "form": "dx", "T": 4096, "H": 2048, "F": 768, "E": 128, "k": 8,
         "drop": 0.0, "dtype": "bf16", "out": "bf16"},
        # the gradient of a small micro-batch's down matrices, Granite-shaped
        {"name": "grad-509-granite", "op": "grad", "form": "down", "T": 509, "H": 1024, "F": 512, "E": 32, "k": 8,
         "drop": 0.05, "dtype": "f16", "out": "f32"},
        # the gradient of the gate/up matrices, Qwen-shaped
        {"name": "grad-4096-qwen", "op": "grad", "form": "gateup", "T": 4096, "H": 2048, "F": 768, "E": 128, "k": 8,
         "drop": 0.0, "dtype": "bf16", "out": "bf16"},
        # one request's decode step through the shared experts' gate/up projection, DeepSeek-shaped
        {"name": "lora-1-r16", "op": "lora", "requests": 1, "T": 1, "K": 2048, "N": 2816, "adapters": 4, "rank": 16,
         "dtype": "bf16", "out": "bf16"},
        # 32 requests' decode step, nearly every one with an adapter of its own
        {"name": "lora-32-r64", "op": "lora", "requests": 32, "T": 32, "K": 2048, "N": 2816, "adapters": 48,
         "rank": 64, "dtype": "f16", "out": "f32"},
        # prompts of 24 requests in one batch
        {"name": "lora-4096-r32", "op": "lora", "requests": 24, "T": 4096, "K": 2048, "N": 2816, "adapters": 16,
         "rank": 32, "dtype": "bf16", "out": "bf16"},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["group", "matmul", "matmul", "grad", "lora", "lora"])
    T, dtype = _log_uniform(rng, 1, 4096), rng.choice(["bf16", "f16"])
    out = rng.choice(["f32", dtype])
    if op == "lora":
        return {"op": op, "requests": _log_uniform(rng, 1, min(T, 256)), "T": T, "K": 8 * rng.randint(16, 256),
                "N": 8 * rng.randint(16, 352), "adapters": _log_uniform(rng, 1, 64), "rank": 8 * _log_uniform(rng, 1, 16),
                "dtype": dtype, "out": out}
    E = _log_uniform(rng, 8, 128)
    case = {"op": op, "T": T, "E": E, "k": rng.randint(1, 8), "drop": rng.choice([0.0, 0.05])}
    if op == "group":
        return case
    case.update(H=8 * rng.randint(16, 256), F=8 * rng.randint(8, 96), dtype=dtype, out=out,
                form=rng.choice(["gateup", "down", "dx"] if op == "matmul" else ["gateup", "down"]))
    return case


# ------------------------------------------------------------------------------ inputs

def _route(g, T, E, k, drop):
    """Routes of T tokens with the spread and the popularity skew of the layers' routers: expert ids
    (-1 where the weight is below `drop`) and weights, [T, k]."""
    rank = torch.randperm(E, generator=g, device="cuda") + 1
    logits = 3.0 * torch.randn(T, E, generator=g, device="cuda") - 1.1 * rank.float().log()
    top = torch.topk(logits, k, dim=1)
    weights = torch.softmax(top.values, 1)
    keep = weights >= drop
    return torch.where(keep, top.indices, -1).int().contiguous(), torch.where(keep, weights, 0.0).contiguous()


def _group(ids, G):
    """First position of each group and the entries in the order of their groups, -1 behind the last."""
    ids = ids.reshape(-1).long()
    key = torch.where((ids >= 0) & (ids < G), ids, G)
    order = torch.argsort(key, stable=True)
    offsets = torch.zeros(G + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.bincount(key, minlength=G + 1)[:G].cumsum(0)
    position = torch.arange(ids.numel(), device=ids.device)
    return offsets.int(), torch.where(position < offsets[G], order, -1).int()


def _requests(g, T, n):
    """Which of n requests each of T tokens belongs to: runs of tokens of ragged lengths, none empty."""
    cuts = torch.randperm(T - 1, generator=g, device="cuda")[:n - 1] + 1 if n > 1 else []
    first = torch.zeros(T, dtype=torch.int64, device="cuda")
    first[cuts] = 1
    return first.cumsum(0)


def _rand(g, dtype, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, T = case["op"], case["T"]
    s = {"case": case, "stream": torch.cuda.current_stream().cuda_stream}
    if op == "lora":
        dt, ot = _TYPES[case["dtype"]][1], _TYPES[case["out"]][1]
        K, N, n, r = case["K"], case["N"], case["adapters"], case["rank"]
        request = _requests(g, T, case["requests"])
        # a request in eight uses the shared projection alone
        of = torch.randint(0, n, (case["requests"],), generator=g, device="cuda")
        of = torch.where(torch.rand(case["requests"], generator=g, device="cuda") < 0.125, -1, of)
        s["adapter"] = of[request].int().contiguous()
        s["x"] = _rand(g, dt, T, K)
        s["w"] = _rand(g, dt, N, K, scale=K ** -0.5)
        s["a"] = _rand(g, dt, n, r, K, scale=K ** -0.5)
        s["b"] = _rand(g, dt, n, N, r, scale=r ** -0.5)
        s["scale"] = 2.0 ** torch.randint(-2, 2, (n,), generator=g, device="cuda").float()
        s["y"] = torch.zeros(T, N, dtype=ot, device="cuda")
        return s
    E, k = case["E"], min(case["k"], case["E"])
    s["k"] = k
    s["ids"], s["weights"] = _route(g, T, E, k, case["drop"])
    R = T * k
    if op == "group":
        s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        s["rows"] = torch.zeros(R, dtype=torch.int32, device="cuda")
        return s
    dt, ot = _TYPES[case["dtype"]][1], _TYPES[case["out"]][1]
    H, F, form = case["H"], case["F"], case["form"]
    s["offsets"], s["rows"] = _group(s["ids"], E)
    if op == "grad":
        # activations and the products' gradients, each in the order in which the forward pass left them
        if form == "gateup":
            s["x"], s["dy"] = _rand(g, dt, T, H), _rand(g, dt, R, 2 * F, scale=0.1)
        else:
            s["x"], s["dy"] = _rand(g, dt, R, F), _rand(g, dt, R, H, scale=0.1)
        s["dw"] = torch.zeros(E, s["dy"].shape[1], s["x"].shape[1], dtype=ot, device="cuda")
        return s
    if form == "gateup":
        s["x"], s["w"] = _rand(g, dt, T, H), _rand(g, dt, E, 2 * F, H, scale=H ** -0.5)
        s["y"] = torch.zeros(R, F, dtype=ot, device="cuda")
    elif form == "down":
        a = torch.randn(R, F, generator=g, device="cuda")
        s["x"] = (a * torch.sigmoid(a) * torch.randn(R, F, generator=g, device="cuda")).to(dt)
        s["w"] = _rand(g, dt, E, H, F, scale=F ** -0.5)
        s["y"] = torch.zeros(T, k, H, dtype=ot, device="cuda")
    else:
        s["x"], s["w"] = _rand(g, dt, R, 2 * F, scale=0.1), _rand(g, dt, E, 2 * F, H, scale=H ** -0.5)
        s["y"] = torch.zeros(T, k, H, dtype=ot, device="cuda")
    return s


# ------------------------------------------------------------------------------ one pass

def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "group":
        return _group(s["ids"], case["E"])
    if op == "lora":
        x, adapter = s["x"].float(), s["adapter"]
        y = x @ s["w"].float().T
        for a in torch.unique(adapter).tolist():
            if a >= 0:
                t = (adapter == a).nonzero().reshape(-1)
                y[t] += s["scale"][a] * ((x[t] @ s["a"][a].float().T) @ s["b"][a].float().T)
        return y.to(s["y"].dtype)
    E, k, form = case["E"], s["k"], case["form"]
    offsets, rows = s["offsets"].tolist(), s["rows"].long()
    if op == "grad":
        dw = torch.zeros_like(s["dw"])
        for e in range(E):
            if offsets[e + 1] > offsets[e]:
                i = slice(offsets[e], offsets[e + 1])
                x = s["x"][rows[i] // k] if form == "gateup" else s["x"][i]
                dy = s["dy"][i] if form == "gateup" else s["dy"][rows[i]]
                dw[e] = (dy.float().T @ x.float()).to(dw.dtype)
        return dw
    y = torch.zeros_like(s["y"])
    flat = y.reshape(-1, y.shape[-1])
    for e in range(E):
        if offsets[e + 1] == offsets[e]:
            continue
        i = slice(offsets[e], offsets[e + 1])
        w = s["w"][e].float()
        if form == "gateup":
            p = s["x"][rows[i] // k].float() @ w.T
            gate, up = p[:, :case["F"]], p[:, case["F"]:]
            flat[i] = (gate / (1.0 + torch.exp(-gate)) * up).to(y.dtype)
        elif form == "down":
            p = s["x"][i].float() @ w.T
            flat[rows[i]] = (p * s["weights"].reshape(-1)[rows[i]].unsqueeze(1)).to(y.dtype)
        else:
            flat[rows[i]] = (s["x"][i].float() @ w).to(y.dtype)
    return y


def _run_own(s):
    from routed_expert_ffn_gemv_gb300 import _lib as L
    case, st = s["case"], s["stream"]
    op, T = case["op"], case["T"]
    if op == "lora":
        K, N, n, r = case["K"], case["N"], case["adapters"], case["rank"]
        if "workspace" not in s:  # kept with the other buffers
            s["workspace"] = torch.empty(L.moe_lora_workspace(T, r), dtype=torch.uint8, device="cuda")
        L.moe_lora_matmul(s["x"], _TYPES[case["dtype"]][0], T, K, s["w"], N, K, s["adapter"], n, s["a"], s["b"], r,
                          s["scale"], s["y"], _TYPES[case["out"]][0], N, s["workspace"], s["workspace"].numel(), st)
        return s["y"]
    E, k = case["E"], s["k"]
    R = T * k
    if op == "group":
        if "workspace" not in s:
            s["workspace"] = torch.empty(L.moe_group_rows_workspace(R, E), dtype=torch.uint8, device="cuda")
        L.moe_group_rows(s["ids"], R, E, s["offsets"], s["rows"], s["workspace"], s["workspace"].numel(), st)
        return s["offsets"], s["rows"]
    H, F, form = case["H"], case["F"], case["form"]
    t, o, rows = _TYPES[case["dtype"]][0], _TYPES[case["out"]][0], s["rows"]
    if form in ("down", "dx") and op == "matmul" and case["drop"]:
        s["y"].zero_()  # dropped routes write no row, and the next pass drops others
    if op == "grad":
        if form == "gateup":
            L.moe_grouped_weight_grad(s["x"], t, T, H, rows, k, s["dy"], R, 2 * F, None, s["offsets"], E, R, 2 * F, H, 0,
                                      s["dw"], o, st)
        else:
            L.moe_grouped_weight_grad(s["x"], t, R, F, None, 1, s["dy"], R, H, rows, s["offsets"], E, R, H, F, 0,
                                      s["dw"], o, st)
        return s["dw"]
    if form == "gateup":
        L.moe_grouped_matmul(s["x"], t, T, H, rows, k, s["offsets"], E, R, s["w"], _NK, F, H, _SWIGLU, None, None,
                             s["y"], o, R, F, st)
    elif form == "down":
        L.moe_grouped_matmul(s["x"], t, R, F, None, 1, s["offsets"], E, R, s["w"], _NK, H, F, _NONE, s["weights"],
                             rows, s["y"], o, R, H, st)
    else:
        L.moe_grouped_matmul(s["x"], t, R, 2 * F, None, 1, s["offsets"], E, R, s["w"], _KN, H, 2 * F, _NONE, None,
                             rows, s["y"], o, R, H, st)
    return s["y"]


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


def work(case):
    op, T = case["op"], case["T"]
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if op == "lora":
        K, N, n, r = case["K"], case["N"], case["adapters"], case["rank"]
        # adapters in use with independent uniform requests, one request in eight without
        used = n * (1.0 - (1.0 - 0.875 / n) ** case["requests"])
        return {"bytes": size[case["dtype"]] * (N * K + T * K + used * r * (K + N)) + size[case["out"]] * T * N + 4 * T,
                "flops": 2 * T * N * K + 0.875 * 2 * T * r * (K + N)}
    E, k = case["E"], min(case["k"], case["E"])
    R = T * k
    if op == "group":
        return {"bytes": 8 * R + 4 * (E + 1), "flops": 0}
    H, F, form = case["H"], case["F"], case["form"]
    # groups in use with independent uniform routes: what the matrices' reads come to
    used = E * (1.0 - (1.0 - k / E) ** T)
    b, o = size[case["dtype"]], size[case["out"]]
    if op == "grad":
        if form == "gateup":
            return {"bytes": b * (T * H + R * 2 * F) + o * E * 2 * F * H, "flops": 4 * R * F * H}
        return {"bytes": b * R * (F + H) + o * E * F * H, "flops": 2 * R * F * H}
    if form == "gateup":
        return {"bytes": b * (used * 2 * F * H + T * H) + o * R * F, "flops": 4 * R * F * H}
    if form == "down":
        return {"bytes": b * (used * F * H + R * F) + o * R * H + 4 * R, "flops": 2 * R * F * H}
    return {"bytes": b * (used * 2 * F * H + R * 2 * F) + o * R * H, "flops": 4 * R * F * H}


# ------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    op, T = case["op"], case["T"]
    if op == "group":
        return None  # whole numbers: nothing is rounded
    s = prepare(case, seed)
    if op == "lora":
        y = torch.empty(T, case["N"], dtype=torch.float64, device="cuda")
        w = s["w"].double()
        for a in range(-1, case["adapters"]):
            mine = s["adapter"] == a
            x = s["x"][mine].double()
            total = w if a < 0 else w + s["scale"][a].double() * (s["b"][a].double() @ s["a"][a].double())
            if x.shape[0]:
                y[mine] = x @ total.T
        return y
    E, k, F, form = case["E"], s["k"], case["F"], case["form"]
    expert = s["ids"].reshape(-1)
    # positions of the routes of each expert among the grouped rows, counted rather than sorted
    first, out = 0, torch.zeros(s["dw" if op == "grad" else "y"].shape, dtype=torch.float64, device="cuda")
    flat = out.reshape(-1, out.shape[-1])
    for e in range(E):
        route = (expert == e).nonzero().reshape(-1)
        place = first + torch.arange(route.numel(), device="cuda")
        first += route.numel()
        if not route.numel():
            continue
        if op == "grad" and form == "gateup":
            out[e] = torch.einsum("in,ik->nk", s["dy"][place].double(), s["x"][route // k].double())
        elif op == "grad":
            out[e] = torch.einsum("in,ik->nk", s["dy"][route].double(), s["x"][place].double())
        elif form == "gateup":
            x = s["x"][route // k].double()
            gate, up = x @ s["w"][e, :F].double().T, x @ s["w"][e, F:].double().T
            flat[place] = gate * torch.sigmoid(gate) * up
        elif form == "down":
            flat[route] = (s["x"][place].double() @ s["w"][e].double().T) * s["weights"].reshape(-1)[route, None].double()
        else:
            flat[route] = s["x"][place].double() @ s["w"][e].double()
    return out
