"""Cases of the INT8 linear, the router and the whole MoE layer.

Operators:
  quant    bf16 [T, K] -> int8 codes with one scale per token
  linear   int8 tokens x int8 weights, scales per token and per output channel
  dynamic  the same product from bf16 tokens, quantised within the call
  router   logits, scores, top-k ids and route weights of [T, H] tokens
  moe      router + routed experts (block-quantized) + INT8 shared expert, bf16 out

Sizes are those of the layer this library is built around (hidden 4096, 256 experts,
intermediate 2048, top-6), of its 4096 x 4096 dense linear, and generic ones.
"""
import math

import torch

own = False

DEV = "cuda"
FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # codes of a prompt's tokens before several linears that share them
        {"name": "quant_t2048", "op": "quant", "T": 2048, "cols": 4096},
        # one decoding session: an attention projection
        {"name": "dynamic_t1", "op": "dynamic", "T": 1, "rows": 4096, "cols": 4096, "bias": False, "out": "bf16"},
        # sixteen decoding sessions, fp32 out with a bias
        {"name": "dynamic_t16", "op": "dynamic", "T": 16, "rows": 2048, "cols": 4096, "bias": True, "out": "f32"},
        # a short ragged batch with odd sizes
        {"name": "linear_t100_odd", "op": "linear", "T": 100, "rows": 5003, "cols": 4112, "bias": False, "out": "bf16"},
        # a prompt through the 4096 x 4096 projection, tokens quantised in the call
        {"name": "dynamic_t2048", "op": "dynamic", "T": 2048, "rows": 4096, "cols": 4096, "bias": False, "out": "bf16"},
        # the largest product: many prompts at once
        {"name": "linear_t8192", "op": "linear", "T": 8192, "rows": 8192, "cols": 8192, "bias": False, "out": "bf16"},
        # the router of one decoding session
        {"name": "router_t1", "op": "router", "T": 1, "H": 4096, "E": 256, "K": 6, "score": "sqrtsoftplus", "norm": True, "bias": True},
        # the router of a prompt
        {"name": "router_t2048", "op": "router", "T": 2048, "H": 4096, "E": 256, "K": 6, "score": "sqrtsoftplus", "norm": True, "bias": True},
        # one token through the whole layer
        {"name": "moe_t1", "op": "moe", "T": 1, "H": 4096, "I": 2048, "E": 256, "K": 6, "gu": "mxfp4", "dn": "mxfp4",
         "shared": 2048, "score": "sqrtsoftplus", "norm": True, "bias": True},
        # four sessions
        {"name": "moe_t4", "op": "moe", "T": 4, "H": 4096, "I": 2048, "E": 256, "K": 6, "gu": "mxfp4", "dn": "mxfp4",
         "shared": 2048, "score": "sqrtsoftplus", "norm": True, "bias": True},
        # one token, the 4-bit / 2-bit mix
        {"name": "moe_t1_nvfp4_q2k", "op": "moe", "T": 1, "H": 4096, "I": 2048, "E": 256, "K": 6, "gu": "nvfp4", "dn": "q2_k",
         "shared": 2048, "score": "sigmoid", "norm": True, "bias": True},
        # sixteen sessions
        {"name": "moe_t16", "op": "moe", "T": 16, "H": 4096, "I": 2048, "E": 256, "K": 6, "gu": "mxfp4", "dn": "mxfp4",
         "shared": 2048, "score": "softmax", "norm": False, "bias": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "linear", "dynamic", "router", "moe", "moe"])
    if op == "quant":
        return {"op": op, "T": _log(rng, 1, 8192), "cols": 16 * _log(rng, 4, 512)}
    if op in ("linear", "dynamic"):
        return {"op": op, "T": _log(rng, 1, 8192), "rows": _log(rng, 64, 8192), "cols": 16 * _log(rng, 8, 512),
                "bias": rng.random() < 0.5, "out": rng.choice(["bf16", "f32"])}
    score, norm, bias = rng.choice(["softmax", "sigmoid", "sqrtsoftplus"]), rng.random() < 0.5, rng.random() < 0.5
    if op == "router":
        return {"op": op, "T": _log(rng, 1, 4096), "H": 8 * _log(rng, 32, 1024), "E": _log(rng, 8, 512),
                "K": rng.randint(1, 8), "score": score, "norm": norm, "bias": bias}
    gu, dn = rng.choice([("mxfp4", "mxfp4"), ("mxfp4", "mxfp4"), ("nvfp4", "q2_k"), ("nvfp4", "mxfp4"), ("mxfp4", "q2_k")])
    return {"op": op, "T": _log(rng, 1, 16), "H": 512 * rng.randint(1, 8), "I": 512 * rng.randint(1, 4),
            "E": _log(rng, 8, 256), "K": rng.randint(1, 6), "gu": gu, "dn": dn,
            "shared": rng.choice([0, 16 * _log(rng, 8, 128)]), "score": score, "norm": norm, "bias": bias}


# ------------------------------------------------------------------ inputs


def _tokens(g, T, K):
    """Hidden states: normal, every token with a scale of its own and a few large channels."""
    x = torch.randn((T, K), generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn((T, 1), generator=g, device=DEV))
    x[:, torch.randint(0, K, (max(1, K // 256),), generator=g, device=DEV)] *= 6.0
    return x.to(torch.bfloat16)


def _int8_weight(g, rows, cols):
    """A linear's weights after symmetric quantisation: near-normal codes, a scale per row."""
    q = (torch.randn((rows, cols), generator=g, device=DEV) * 32.0).round().clamp(-127, 127).to(torch.int8)
    s = (0.5 + torch.rand((rows,), generator=g, device=DEV)) / (32.0 * math.sqrt(cols))
    return q, s


def _bytes(g, *shape):
    return torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)


def _block_weight(g, fmt, n, rows, cols):
    """Expert planes as the library stores them (data, scales, scale_2 or None)."""
    if fmt == "mxfp4":
        return _bytes(g, n, rows, cols // 2), torch.randint(119, 124, (n, rows, cols // 32), generator=g, device=DEV, dtype=torch.uint8), None
    if fmt == "nvfp4":
        sc = torch.randint(0x08, 0x29, (n, rows, cols // 16), generator=g, device=DEV, dtype=torch.uint8)
        return _bytes(g, n, rows, cols // 2), sc, 0.25 + 0.5 * torch.rand((n,), generator=g, device=DEV)
    d = ((0.5 + torch.rand((n, rows, cols // 256, 2), generator=g, device=DEV)) * 0.004).to(torch.float16)
    sc = torch.cat([_bytes(g, n, rows, cols // 256, 16), d.view(torch.uint8)], dim=-1)
    return _bytes(g, n, rows, cols // 256, 64), sc, None


def _router_weight(g, case):
    w = (torch.randn((case["E"], case["H"]), generator=g, device=DEV) / math.sqrt(case["H"])).to(torch.bfloat16)
    b = 0.1 * torch.randn((case["E"],), generator=g, device=DEV) if case["bias"] else None
    return w, b


SCALE = 1.5  # the routed experts' factor


def _inputs(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, s = case["op"], {}
    if op in ("quant", "linear", "dynamic"):
        s["x"] = _tokens(g, case["T"], case["cols"])
        if op != "quant":
            s["wq"], s["ws"] = _int8_weight(g, case["rows"], case["cols"])
            s["b"] = torch.randn((case["rows"],), generator=g, device=DEV) if case["bias"] else None
        if op == "linear":
            s["xq"], s["xs"] = _quantize(s.pop("x"))
        return s
    s["x"] = _tokens(g, case["T"], case["H"])
    s["rw"], s["rb"] = _router_weight(g, case)
    if op == "moe":
        E, H, I = case["E"], case["H"], case["I"]
        s["gate"] = _block_weight(g, case["gu"], E, I, H)
        s["up"] = _block_weight(g, case["gu"], E, I, H)
        s["down"] = _block_weight(g, case["dn"], E, H, I)
        if case["shared"]:
            s["sgate"], s["sup"] = _int8_weight(g, case["shared"], H), _int8_weight(g, case["shared"], H)
            s["sdown"] = _int8_weight(g, H, case["shared"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        s.update(_handles(case, s))
    return s


def _handles(case, s):
    """What a program keeps between calls: descriptors, workspaces, output buffers."""
    import bit_quantized_moe_dequant_amd as mq

    h, op, T = {"mq": mq}, case["op"], case["T"]

    def weight(name, fmt, n, rows, cols):
        data, scales = s[name][:2]
        s2 = s[name][2] if len(s[name]) > 2 else None
        return mq.Weight(mq.FMT_BY_NAME[fmt], rows, cols, n, data.view(torch.uint8).reshape(-1), scales.view(torch.uint8).reshape(-1), s2)

    if op == "quant":
        h["q"] = torch.empty((T, case["cols"]), dtype=torch.int8, device=DEV)
        h["s"] = torch.empty((T,), device=DEV)
        return h
    if op in ("linear", "dynamic"):
        s["lin"] = (s["wq"], s["ws"])
        h["w"] = weight("lin", "int8", 1, case["rows"], case["cols"])
        h["y"] = torch.empty((T, case["rows"]), dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32, device=DEV)
        return h
    h["router"] = mq.Router(s["rw"], case["K"], scoring=case["score"], normalize=case["norm"], scale=SCALE, bias=s["rb"])
    h["ids"] = torch.empty((T, case["K"]), dtype=torch.int32, device=DEV)
    h["wts"] = torch.empty((T, case["K"]), device=DEV)
    if op == "moe":
        E, H, I, S = case["E"], case["H"], case["I"], case["shared"]
        layer = mq.Layer(H, I, E, case["K"], weight("gate", case["gu"], E, I, H), weight("up", case["gu"], E, I, H), weight("down", case["dn"], E, H, I))
        shared = mq.SharedExpert(weight("sgate", "int8", 1, S, H), weight("sup", "int8", 1, S, H), weight("sdown", "int8", 1, H, S)) if S else None
        h["moe"] = mq.MoeLayer(layer, h["router"], shared)
        h["y"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    return h


# ------------------------------------------------------------------ the passes


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    mq, op = s["mq"], s["case"]["op"]
    if op == "quant":
        return mq.quantize_int8(s["x"], q=s["q"], scale=s["s"])
    if op == "linear":
        return mq.linear_int8(s["w"], s["xq"], s["xs"], bias=s["b"], y=s["y"])
    if op == "dynamic":
        return mq.linear_int8_dynamic(s["w"], s["x"], bias=s["b"], y=s["y"])
    if op == "router":
        return mq.router_topk(s["router"], s["x"], ids=s["ids"], rw=s["wts"])
    return mq.moe_forward(s["moe"], s["x"], y=s["y"], ids=s["ids"], rw=s["wts"])


def _quantize(x):
    """Codes and scales by the operator's fp32 rule: s = max / 127, q = round(x / s)."""
    x = x.float()
    a = x.abs().amax(dim=1, keepdim=True)
    s = a / torch.full_like(a, 127.0)
    q = torch.where(s > 0, torch.round(x / s), torch.zeros_like(x)).clamp(-127, 127)
    return q.to(torch.int8), s[:, 0]


def _int8_product(xq, xs, wq, ws, b):
    y = (xq.float() @ wq.float().t()) * xs[:, None] * ws[None, :]
    return y if b is None else y + b


def _scores(logits, kind):
    if kind == "softmax":
        e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
        return e / e.sum(dim=1, keepdim=True)
    if kind == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    return torch.sqrt(torch.clamp(logits, min=0.0) + torch.log1p(torch.exp(-logits.abs())))


def _route(case, s):
    """Ids and weights, in 64 bits: the order of near-equal scores decides who is chosen."""
    score = _scores(s["x"].double() @ s["rw"].double().t(), case["score"])
    key = score if s["rb"] is None else score + s["rb"].double()
    ids = torch.sort(key, dim=1, descending=True, stable=True)[1][:, : case["K"]]
    w = torch.gather(score, 1, ids)
    if case["norm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return ids.to(torch.int32), (w * SCALE).float()


def _fp4(data):
    """e2m1 codes, low nibble first, as fp32."""
    table = torch.tensor([s * v for s in (1.0, -1.0) for v in FP4], device=DEV)
    return torch.stack((table[(data & 15).int()], table[(data >> 4).int()]), dim=-1).flatten(-2)


def _decode(fmt, w, ids):
    """The chosen experts' matrices, fp32 [len(ids), rows, cols]."""
    data, sc = w[0][ids], w[1][ids]
    if fmt == "mxfp4":
        return (_fp4(data).unflatten(-1, (-1, 32)) * torch.exp2(sc.float() - 127.0).unsqueeze(-1)).flatten(-2)
    if fmt == "nvfp4":
        scale = sc.view(torch.float8_e4m3fn).float() * w[2][ids][:, None, None]
        return (_fp4(data).unflatten(-1, (-1, 16)) * scale.unsqueeze(-1)).flatten(-2)
    d = sc[..., 16:].contiguous().view(torch.float16).float()
    shifts = torch.arange(0, 8, 2, device=DEV, dtype=torch.uint8)[:, None]
    q = ((data.unflatten(-1, (2, 1, 32)) >> shifts) & 3).flatten(-3).unflatten(-1, (16, 16)).float()
    sub = sc[..., :16]
    a, m = d[..., 0:1] * (sub & 15).float(), d[..., 1:2] * (sub >> 4).float()
    return (a.unsqueeze(-1) * q - m.unsqueeze(-1)).flatten(-3)


def _swiglu(g, u):
    return g / (1.0 + torch.exp(-g)) * u


def _experts(case, s, ids, rw):
    pairs = ids.flatten().long()
    x = s["x"].float().repeat_interleave(case["K"], dim=0).unsqueeze(-1)
    g = torch.matmul(_decode(case["gu"], s["gate"], pairs), x).squeeze(-1)
    u = torch.matmul(_decode(case["gu"], s["up"], pairs), x).squeeze(-1)
    o = torch.matmul(_decode(case["dn"], s["down"], pairs), _swiglu(g, u).unsqueeze(-1)).squeeze(-1)
    return (o.unflatten(0, (case["T"], case["K"])) * rw.unsqueeze(-1)).sum(dim=1)


def _run_plain(s):
    case = s["case"]
    if case["op"] == "quant":
        return _quantize(s["x"])
    if case["op"] in ("linear", "dynamic"):
        xq, xs = _quantize(s["x"]) if case["op"] == "dynamic" else (s["xq"], s["xs"])
        y = _int8_product(xq, xs, s["wq"], s["ws"], s["b"])
        return y.to(torch.bfloat16) if case["out"] == "bf16" else y
    ids, rw = _route(case, s)
    if case["op"] == "router":
        return ids, rw
    y = _experts(case, s, ids, rw)
    if case["shared"]:
        xq, xs = _quantize(s["x"])
        h = _swiglu(_int8_product(xq, xs, *s["sgate"], None), _int8_product(xq, xs, *s["sup"], None))
        y = y + _int8_product(*_quantize(h), *s["sdown"], None)
    return y.to(torch.bfloat16), ids, rw


# ------------------------------------------------------------------ work and 64-bit values

BYTES = {"mxfp4": 17 / 32, "nvfp4": 9 / 16, "q2_k": 84 / 256}


def work(case):
    T, op = case["T"], case["op"]
    if op == "quant":
        return {"bytes": T * case["cols"] * 3 + 4 * T, "flops": 4 * T * case["cols"]}
    if op in ("linear", "dynamic"):
        rows, cols = case["rows"], case["cols"]
        x = T * cols * (2 if op == "dynamic" else 1) + (4 * T if op == "linear" else 0)
        y = T * rows * (2 if case["out"] == "bf16" else 4)
        return {"bytes": rows * cols + 4 * rows + (4 * rows if case["bias"] else 0) + x + y, "flops": 2 * T * rows * cols}
    E, H, K = case["E"], case["H"], case["K"]
    b, f = 2 * E * H + (4 * E if case["bias"] else 0) + 2 * T * H + 8 * T * K, 2 * T * E * H
    if op == "moe":
        I, S = case["I"], case["shared"]
        touched = E * (1.0 - (1.0 - min(K, E) / E) ** T)  # expected under even routing
        b += touched * I * H * (2 * BYTES[case["gu"]] + BYTES[case["dn"]]) + 3 * S * H + 4 * (2 * S + H if S else 0) + 2 * T * H
        f += 6 * T * K * I * H + 6 * T * S * H
    return {"bytes": b, "flops": f}


def exact(case, seed):
    """The definitions in 64 bits, expert by expert. The codes and scales of a token are defined
    by their fp32 rule, so those two steps are taken in it."""
    s = _inputs(case, seed)
    op = case["op"]

    def codes(x32):
        a = x32.abs().amax(dim=1)
        sc = torch.div(a, torch.full_like(a, 127.0))
        safe = torch.where(sc == 0, torch.ones_like(sc), sc)
        return torch.clamp(torch.round(torch.div(x32, safe[:, None])), -127, 127).double(), sc.double()

    def product(q, sc, wq, ws, b):
        y = torch.empty((q.shape[0], wq.shape[0]), dtype=torch.float64, device=DEV)
        for r in range(0, wq.shape[0], 1024):  # a block of channels at a time
            y[:, r:r + 1024] = q @ wq[r:r + 1024].double().t()
        y = y * sc[:, None] * ws.double()
        return y if b is None else y + b.double()

    if op == "quant":
        q, sc = codes(s["x"].float())
        return None, sc
    if op == "linear":
        return product(s["xq"].double(), s["xs"].double(), s["wq"], s["ws"], s["b"])
    if op == "dynamic":
        return product(*codes(s["x"].float()), s["wq"], s["ws"], s["b"])

    x = s["x"].double()
    z = torch.stack([(x * w.double()).sum(dim=1) for w in s["rw"]], dim=1)
    if case["score"] == "softmax":
        p = torch.softmax(z, dim=1)
    elif case["score"] == "sigmoid":
        p = torch.sigmoid(z)
    else:
        p = torch.sqrt(torch.logaddexp(z, torch.zeros_like(z)))
    key = p + s["rb"].double() if s["rb"] is not None else p
    ids = torch.argsort(key, dim=1, descending=True, stable=True)[:, : case["K"]]
    w = p.gather(1, ids)
    w = SCALE * (w / w.sum(dim=1, keepdim=True) if case["norm"] else w)
    if op == "router":
        return None, w

    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=DEV)

    def matrix(fmt, planes, e):
        data, sc = planes[0][e], planes[1][e]
        if fmt in ("mxfp4", "nvfp4"):
            both = torch.stack([data & 15, data >> 4], dim=2).reshape(data.shape[0], -1).long()
            v = lut[both & 7] * (1.0 - 2.0 * (both >> 3).double())
            if fmt == "mxfp4":
                return v * torch.ldexp(torch.ones((), dtype=torch.float64, device=DEV), sc.long() - 127).repeat_interleave(32, dim=1)
            return v * sc.view(torch.float8_e4m3fn).double().repeat_interleave(16, dim=1) * planes[2][e].double()
        rows, blocks = data.shape[0], data.shape[1]
        d = sc[:, :, 16:].contiguous().view(torch.float16).double()
        out = torch.empty((rows, blocks, 256), dtype=torch.float64, device=DEV)
        for j in range(16):  # sub-blocks of 16 weights
            half, sh, off = j // 8, 2 * ((j % 8) // 2), 16 * (j % 2)
            q = ((data[:, :, 32 * half + off: 32 * half + off + 16] >> sh) & 3).double()
            lo, hi = (sc[:, :, j] & 15).double(), (sc[:, :, j] >> 4).double()
            out[:, :, 16 * j: 16 * j + 16] = (d[:, :, 0] * lo)[..., None] * q - (d[:, :, 1] * hi)[..., None]
        return out.reshape(rows, -1)

    y = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device=DEV)
    for e in sorted(set(ids.flatten().tolist())):
        t, k = (ids == e).nonzero(as_tuple=True)
        g, u = x[t] @ matrix(case["gu"], s["gate"], e).t(), x[t] @ matrix(case["gu"], s["up"], e).t()
        h = g * torch.sigmoid(g) * u
        y[t] += w[t, k][:, None] * (h @ matrix(case["dn"], s["down"], e).t())
    if case["shared"]:
        q, sc = codes(s["x"].float())
        g, u = product(q, sc, *s["sgate"], None), product(q, sc, *s["sup"], None)
        y += product(*codes((g * torch.sigmoid(g) * u).float()), *s["sdown"], None)
    return y, None, w
