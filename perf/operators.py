"""Cases of the epilogue matmul and of the mixture-of-experts operators.

``run`` computes each operator in its plain form (elementary torch
operations in fp32) or, where ``own`` is true, with the calls that a user
makes of ``mlp_matmul_amd``.  The operators:

``linear``   y = act(X . W^T + bias) + residual
``route``    top-k experts of every token, their softmax weights, and the
             tokens grouped by expert (offsets, order, place)
``gate_up``  h = SiLU(x . G_e^T) * (x . U_e^T) over rows grouped by expert
``down``     Y = x . D_e^T over rows grouped by expert
``layer``    routing, gate/up, down and the weighted sum over a token's
             experts, plus the residual

Weights are bf16 or in the direct-palette form of ``include/unweight.h``
(sign/mantissa bytes, 4-bit indices of the 16 most frequent exponents, raw
exponents of the 64-element groups that hold another one).  The matrices of
all experts are one matrix of experts*rows rows.  Shapes are those of the
repository's MLP and attention workloads and generic splits of them.
"""
import math

import torch

own = False

SIGMA, P_OUT, S_OUT = 0.02, 5e-4, 0.5     # weight spread, share and spread of its outliers (workloads.py)
F32, BF16 = torch.float32, torch.bfloat16
KINDS = {"linear": 1, "route": 2, "gate_up": 3, "down": 4, "layer": 5}


# ---------------------------------------------------------------- the cases
def linear(rows, cols, batch, pal, bias=False, act="none", residual=False, bf16_out=True):
    return {"op": "linear", "rows": rows, "cols": cols, "batch": batch, "pal": pal, "bias": bias, "act": act,
            "residual": residual, "bf16_out": bf16_out}


def route(tokens, experts, top_k, renorm=True, bf16=False, padding=0.0):
    return {"op": "route", "tokens": tokens, "experts": experts, "top_k": top_k, "renorm": renorm, "bf16": bf16,
            "padding": padding}


def experts_case(op, tokens, experts, top_k, ffn, hidden, pal, skew=0.5, padding=0.0):
    return {"op": op, "tokens": tokens, "experts": experts, "top_k": top_k, "ffn": ffn, "hidden": hidden, "pal": pal,
            "skew": skew, "padding": padding}


def listed():
    return [
        # one token through a key/value projection with a bias: the smallest product, launch latency counts
        dict(linear(1024, 4096, 1, True, bias=True), name="linear 1x1024x4096 palette"),
        # a decode batch through the down projection, added to the residual stream
        dict(linear(4096, 14336, 16, True, residual=True), name="linear 16x4096x14336 pal"),
        # a mid-size odd batch through a wide uncompressed first MLP matrix with its bias and GELU
        dict(linear(14336, 4096, 77, False, bias=True, act="gelu_tanh"), name="linear 77x14336x4096 bf16"),
        # an odd-length prompt through a square projection, everything in the epilogue, fp32 result
        dict(linear(4096, 4096, 2049, True, bias=True, act="silu", residual=True, bf16_out=False),
             name="linear 2049x4096x4096 pal"),
        # routing of a decode batch, and of a long prompt with padded tokens over many experts
        dict(route(8, 64, 6), name="route 8 of 64"),
        dict(route(16384, 256, 8, padding=0.05), name="route 16384 of 256"),
        # gate/up of a single token: two experts' weights are read once
        dict(experts_case("gate_up", 1, 8, 2, 3584, 4096, True), name="gate_up 1 palette"),
        # a decode batch over uncompressed experts: a few tokens an expert, the weights' bytes bound it
        dict(experts_case("gate_up", 33, 16, 2, 1792, 4096, False), name="gate_up 33 bf16"),
        # a prompt: the matrix units bound it
        dict(experts_case("gate_up", 4001, 8, 2, 3584, 4096, True), name="gate_up 4001 palette"),
        # many small experts, very uneven, some without a token
        dict(experts_case("down", 1500, 32, 4, 1024, 2048, False, skew=2.0), name="down 1500 bf16"),
        # the whole layer for one token, and for a mid-size batch with padded tokens
        dict(experts_case("layer", 1, 8, 2, 3584, 4096, True), name="layer 1 palette"),
        dict(experts_case("layer", 600, 16, 4, 1024, 2048, False, padding=0.1), name="layer 600 bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["linear", "linear", "route", "gate_up", "gate_up", "down", "layer", "layer"])
    pal = rng.random() < 0.6
    if kind == "linear":
        rows, cols = _log(rng, 64, 16000), 64 * _log(rng, 2, 224)
        batch = _log(rng, 1, min(4096, max(2, int(2e11 / (2 * rows * cols)))))
        return linear(rows, cols, batch, pal, rng.random() < 0.5, rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]),
                      rng.random() < 0.5, rng.random() < 0.6)
    if kind == "route":
        experts = _log(rng, 4, 300)
        return route(_log(rng, 1, 16384), experts, rng.randint(1, min(8, experts)), rng.random() < 0.7,
                     rng.random() < 0.5, rng.choice([0.0, 0.1]))
    experts = _log(rng, 4, 48)
    top_k = rng.randint(1, min(6, experts))
    hidden = 64 * _log(rng, 8, 64)
    ffn = 64 * _log(rng, 4, max(5, min(56, int(1e8 / (64 * experts * hidden)))))
    most = int(2.5e11 / (2 * top_k * ffn * hidden * {"gate_up": 2, "down": 1, "layer": 3}[kind]))
    tokens = _log(rng, 1, max(2, min(6000, most)))
    return experts_case(kind, tokens, experts, top_k, ffn, hidden, pal, rng.choice([0.0, 0.5, 2.0]),
                        rng.choice([0.0, 0.1]))


# --------------------------------------------------------------- the inputs
def _generator(case, seed, stream):
    return torch.Generator("cuda").manual_seed(seed * 64 + KINDS[case["op"]] * 8 + stream)


def _weights(g, rows, cols):
    """bf16 [rows, cols]: N(0, 0.02) with outliers, as the repository's workloads draw them."""
    w = torch.randn(rows, cols, device="cuda", generator=g).mul_(SIGMA)
    n = max(1, int(w.numel() * P_OUT))
    at = torch.randint(w.numel(), (n,), device="cuda", generator=g)
    w.view(-1).index_fill_(0, at, S_OUT * 0.75)
    return w.to(BF16)


def _planes(w):
    """The direct-palette form of bf16 [rows, cols]: what a program holds on the GPU for a compressed matrix."""
    rows, cols = w.shape
    bits = w.view(torch.int16).reshape(-1)
    e = (bits >> 7).to(torch.uint8)                              # the exponent byte (the sign's bit falls off)
    sm = ((bits >> 8).to(torch.uint8) & 0x80) | (bits.to(torch.uint8) & 0x7F)
    palette = torch.sort(torch.bincount(e, minlength=256), descending=True, stable=True)[1][:16].to(torch.uint8)
    index_of = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    index_of[palette.long()] = torch.arange(16, dtype=torch.uint8, device="cuda")
    index = index_of[e.int()].view(-1, 64)
    verbatim = (index == 255).any(1)
    vexp = e.view(-1, 64)[verbatim].reshape(-1)
    index = torch.where(verbatim[:, None], 0, index).view(-1, 2)
    nib = index[:, 0] | (index[:, 1] << 4)
    groups = verbatim.numel()
    flags = torch.zeros(-(-groups // 64) * 64, dtype=torch.int64, device="cuda")
    flags[:groups] = verbatim
    flags = flags.view(-1, 64)
    bitmap = (flags << torch.arange(64, device="cuda")).sum(1)
    vbase = torch.zeros(flags.shape[0] + 1, dtype=torch.int32, device="cuda")
    vbase[1:] = flags.sum(1).cumsum(0)

    def padded(t):
        raw = t.contiguous().view(torch.uint8)
        return torch.cat([raw, raw.new_zeros(-raw.numel() % 16 + 16)])

    return {"rows": rows, "cols": cols, "palette": palette, "sm": padded(sm), "nib": padded(nib), "vexp": padded(vexp),
            "bitmap": padded(bitmap), "tile_vbase": padded(vbase), "verbatim": int(vexp.numel()) // 64}


def _matrix(case, g, rows, cols, experts=1):
    """A weight as a program keeps it: bf16 [experts, rows, cols], or the planes of [experts*rows, cols] and the
    framework's handle on them (the addresses of the same planes; nothing is computed or laid out for it)."""
    w = _weights(g, experts * rows, cols)
    if not case["pal"]:
        return {"w": w.view(experts, rows, cols)}
    m = {"planes": _planes(w)}
    if own:
        from mlp_matmul_amd import DeviceMatrix
        p = m["planes"]
        m["handle"] = DeviceMatrix.from_sections(p["rows"], p["cols"], p["palette"].tolist(), p["verbatim"],
                                                 {k: p[k] for k in ("sm", "nib", "vexp", "bitmap", "tile_vbase")})
    return m


def _logits(case, g):
    t, e = case["tokens"], case["experts"]
    l = torch.randn(t, e, device="cuda", generator=g)
    l += case.get("skew", 0.5) * torch.randn(e, device="cuda", generator=g)      # some experts are popular
    if case["padding"]:
        l[torch.rand(t, device="cuda", generator=g) < case["padding"]] = -math.inf
    return l.to(BF16) if case.get("bf16") else l


def _rows(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g).to(BF16)


def _inputs(case, seed):
    """Everything but the weights."""
    g = _generator(case, seed, 1)
    s = {}
    if case["op"] == "linear":
        s["x"] = _rows(g, case["batch"], case["cols"])
        s["bias"] = torch.randn(case["rows"], device="cuda", generator=g) if case["bias"] else None
        s["residual"] = _rows(g, case["batch"], case["rows"]) if case["residual"] else None
        return s
    s["logits"] = _logits(case, g)
    if case["op"] == "route":
        return s
    if case["op"] == "layer":
        s["x"] = _rows(g, case["tokens"], case["hidden"])
        s["residual"] = _rows(g, case["tokens"], case["hidden"])
        return s
    s["route"] = _route(s["logits"], case["top_k"], True)
    s["offsets"], s["order"] = s["route"][2], s["route"][3]
    n = int(s["offsets"][-1])
    s["order"] = s["order"][:n].contiguous()
    if case["op"] == "gate_up":
        s["x"] = _rows(g, case["tokens"], case["hidden"])
    else:
        s["x"] = _rows(g, n, case["ffn"])
    return s


def _shapes(case):
    """(rows, cols, experts) of the case's weights, in their order."""
    if case["op"] == "linear":
        return [(case["rows"], case["cols"], 1)]
    f, h, e = case.get("ffn"), case.get("hidden"), case["experts"]
    return {"route": [], "gate_up": [(f, h, e)] * 2, "down": [(h, f, e)],
            "layer": [(f, h, e)] * 2 + [(h, f, e)]}[case["op"]]


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    s["m"] = [_matrix(case, _generator(case, seed, 2 + i), *shape) for i, shape in enumerate(_shapes(case))]
    return s


# --------------------------------------------------------- the plain forms
def _plain_weight(m, rows, cols, only=None):
    """fp32 [experts, rows, cols] of a weight, or of the experts ``only`` (an index tensor)."""
    if "w" in m:
        return (m["w"] if only is None else m["w"][only]).to(F32)
    p = m["planes"]
    total = p["rows"] * p["cols"]
    groups = total // 64
    per = rows * cols
    bits = p["bitmap"][:-(-groups // 64) * 8].view(torch.int64)
    flags = ((bits[:, None] >> torch.arange(64, device="cuda")) & 1).reshape(-1)[:groups]
    slot = flags.cumsum(0) - flags
    sm, nib = p["sm"][:total].view(-1, per), p["nib"][:total // 2].view(-1, per // 2)
    flags, slot = flags.view(-1, per // 64), slot.view(-1, per // 64)
    if only is not None:
        sm, nib, flags, slot = sm[only], nib[only], flags[only], slot[only]
    index = torch.stack([nib & 15, nib >> 4], -1).view(-1)
    e = p["palette"][index.int()].view(-1, 64)
    at = flags.reshape(-1).nonzero()[:, 0]
    e[at] = p["vexp"][:p["verbatim"] * 64].view(-1, 64)[slot.reshape(-1)[at]]
    sm = sm.reshape(-1).to(torch.int32)
    bits = ((sm & 0x80) << 24) | (e.view(-1).to(torch.int32) << 23) | ((sm & 0x7F) << 16)
    return bits.view(F32).view(-1, rows, cols)


def _act(v, act):
    if act == "relu":
        return torch.where(v < 0, 0.0, v)
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _route(logits, top_k, renorm):
    l = logits.to(F32)
    tokens, experts = l.shape
    value, ids = torch.sort(l, dim=1, descending=True, stable=True)
    top = torch.where(value[:, :1] == -math.inf, 0.0, value[:, :1])
    part = torch.exp(value - top)
    chosen = part[:, :top_k]
    total = (chosen if renorm else part).sum(1, keepdim=True)
    alive = value[:, :top_k] > -math.inf
    weights = torch.where(alive, chosen / total, 0.0)
    ids = torch.where(alive, ids[:, :top_k], -1).to(torch.int32)
    key = torch.where(ids < 0, experts, ids).view(-1)
    key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(experts + 1, device=key.device, dtype=key.dtype)).to(torch.int32)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    place = torch.where(ids.view(-1) < 0, -1, place).view(tokens, top_k).to(torch.int32)
    order = torch.where(key == experts, -1, order).to(torch.int32)
    return ids, weights, offsets, order, place


def _expert_of(offsets, n):
    return torch.searchsorted(offsets[1:].contiguous(), torch.arange(n, device="cuda", dtype=torch.int32), right=True)


def _grouped(x, ms, rows, cols, offsets):
    """[x_s . W_e(s)^T for each of ms]: x fp32 [n, cols] sorted by expert.  Few rows: each row's own matrix is
    gathered; else every expert's rows are padded to the same number and multiplied in one batch."""
    n, experts = x.shape[0], offsets.numel() - 1
    e = _expert_of(offsets, n)
    if n <= experts // 2:
        return [torch.bmm(_plain_weight(m, rows, cols, e), x[:, :, None])[:, :, 0] for m in ms]
    at = torch.arange(n, device="cuda") - offsets[e]
    most = int((offsets[1:] - offsets[:-1]).max())
    padded = x.new_zeros(experts, most, cols)
    padded[e, at] = x
    return [torch.bmm(padded, _plain_weight(m, rows, cols).transpose(1, 2).contiguous())[e, at] for m in ms]


def _plain(s):
    c = s["case"]
    if c["op"] == "linear":
        v = s["x"].to(F32) @ _plain_weight(s["m"][0], c["rows"], c["cols"])[0].t()
        if s["bias"] is not None:
            v = v + s["bias"]
        v = _act(v, c["act"])
        if s["residual"] is not None:
            v = v + s["residual"].to(F32)
        return v.to(BF16 if c["bf16_out"] else F32)
    if c["op"] == "route":
        return _route(s["logits"], c["top_k"], c["renorm"])
    if c["op"] == "down":
        return _grouped(s["x"].to(F32), s["m"], c["hidden"], c["ffn"], s["offsets"])[0]
    if c["op"] == "gate_up":
        x = s["x"].to(F32)[(s["order"] // c["top_k"]).long()]
        g, u = _grouped(x, s["m"], c["ffn"], c["hidden"], s["offsets"])
        return (_act(g, "silu") * u).to(BF16)
    ids, weights, offsets, order, place = _route(s["logits"], c["top_k"], True)
    n = int(offsets[-1])
    x = s["x"].to(F32)[(order[:n] // c["top_k"]).long()]
    g, u = _grouped(x, s["m"][:2], c["ffn"], c["hidden"], offsets)
    y = _grouped(_act(g, "silu") * u, s["m"][2:], c["hidden"], c["ffn"], offsets)[0]
    y = torch.cat([y, y.new_zeros(1, c["hidden"])])              # place -1 reads the zeros at the end
    v = (y[place.long()] * weights[:, :, None]).sum(1) + s["residual"].to(F32)
    return v.to(BF16)


# ------------------------------------------------------ the framework's calls
def _own(s):
    import mlp_matmul_amd as uw
    c = s["case"]
    w = [m["handle"] if "handle" in m else m["w"] for m in s["m"]]
    if c["op"] == "linear":
        return uw.linear(w[0][0] if "w" in s["m"][0] else w[0], s["x"], bias=s["bias"], act=c["act"],
                         residual=s["residual"], out_dtype=BF16 if c["bf16_out"] else F32)
    if c["op"] == "route":
        r = uw.moe_route(s["logits"], c["top_k"], renormalize=c["renorm"])
        return r.ids, r.weights, r.offsets, r.order, r.place
    if c["op"] == "down":
        return uw.gemm_grouped(w[0], s["x"], s["offsets"])
    if c["op"] == "gate_up":
        return uw.moe_gate_up(w[0], w[1], s["x"], s["offsets"], s["order"], c["top_k"])
    return uw.moe_layer(w[0], w[1], w[2], s["x"], s["logits"], c["top_k"], residual=s["residual"], out_dtype=BF16)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------- the definition
def exact(case, seed):
    """The definitions in 64 bits on the drawn bf16 weights themselves, expert by expert."""
    s = _inputs(case, seed)
    ws = [_weights(_generator(case, seed, 2 + i), e * r, c).view(e, r, c) for i, (r, c, e) in enumerate(_shapes(case))]
    if case["op"] == "linear":
        y = torch.mm(s["x"].double(), ws[0][0].double().t())
        y = y if s["bias"] is None else y + s["bias"].double()
        c = y.clone()
        if case["act"] == "relu":
            y = y.clamp_min(0)
        elif case["act"] == "silu":
            y = c * torch.sigmoid(c)
        elif case["act"] == "gelu":
            y = c * torch.special.ndtr(c)
        elif case["act"] == "gelu_tanh":
            y = c * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (c + 0.044715 * c ** 3))
        return y if s["residual"] is None else y + s["residual"].double()
    k, experts = case["top_k"], case["experts"]
    l = s["logits"].double()
    p = torch.softmax(l.nan_to_num(nan=-math.inf, neginf=-1e300), 1)
    p = torch.where(l.isneginf(), 0.0, p)
    ids = torch.argsort(-l, dim=1, stable=True)[:, :k]
    w = p.gather(1, ids)
    dead = l.gather(1, ids).isneginf()
    if case.get("renorm", True):
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    w = torch.where(dead, 0.0, w)
    if case["op"] == "route":
        return None, w, None, None, None
    flat = torch.where(dead, -1, ids).reshape(-1)
    rows = [(flat == e).nonzero()[:, 0] for e in range(experts)]       # sorted rows of expert e, as flat slots
    if case["op"] == "down":
        parts, at = [], 0
        for e, r in enumerate(rows):
            parts.append(s["x"][at:at + r.numel()].double() @ ws[0][e].double().t())
            at += r.numel()
        return torch.cat(parts)
    x = s["x"].double()
    h = [torch.nn.functional.silu(x[r // k] @ ws[0][e].double().t()) * (x[r // k] @ ws[1][e].double().t())
         for e, r in enumerate(rows)]
    if case["op"] == "gate_up":
        return torch.cat(h)
    y = s["residual"].double()
    for e, r in enumerate(rows):
        y.index_add_(0, r // k, (h[e] @ ws[2][e].double().t()) * w.reshape(-1)[r, None])
    return y


# --------------------------------------------------------------- what it costs
def work(case):
    """Bytes and operations that a pass cannot do without (weights of the experts with tokens, each read once)."""
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        return {"bytes": t * e * (2 if case["bf16"] else 4) + t * k * 16 + 4 * (e + 1), "flops": t * e}
    per = 1.5 + P_OUT * 64 + 9 / 4096 if case["pal"] else 2.0    # sm + nibbles + verbatim exponents + tables
    if case["op"] == "linear":
        r, c, b = case["rows"], case["cols"], case["batch"]
        n = r * c * per + 2 * b * c + b * r * (2 if case["bf16_out"] else 4)
        n += 4 * r * case["bias"] + 2 * b * r * case["residual"]
        return {"bytes": n, "flops": 2 * b * r * c}
    t, e, k, f, h = (case[i] for i in ("tokens", "experts", "top_k", "ffn", "hidden"))
    slots = t * k * (1 - case["padding"])
    used = e * (1 - (1 - k / e) ** (t * (1 - case["padding"])))  # experts that get a token, evenly routed
    mats = {"gate_up": 2, "down": 1, "layer": 3}[case["op"]]
    n = mats * used * f * h * per
    n += {"gate_up": 2 * t * h + 2 * slots * f, "down": 2 * slots * f + 4 * slots * h,
          "layer": 6 * t * h + 4 * t * e}[case["op"]]
    return {"bytes": n, "flops": 2 * slots * f * h * mats}
