"""Cases of the microscaled 4-bit operators and of the scored router.

``run`` computes each operator in its plain form (elementary torch
operations, in fp32, or fp64 where a value decides a choice) or, where
``own`` is true, with the calls that a user makes of ``mlp_matmul_amd``.  The
operators:

``quantize``  bf16 to microscaled 4-bit numbers and back to the values they stand for
``linear``    y = act(X . W^T + bias) + residual with W in 4 bits; X is bf16, or
              quantised to 4 bits first (``x4``)
``route``     experts of every token by sigmoid or softmax scores: a bias that
              counts for the choice alone, groups of experts, top-k, renormalised
              and scaled weights, and the tokens grouped by expert
``gate_up``   h = SiLU(x . G_e^T) * (x . U_e^T) over rows grouped by expert, G and
              U in 4 bits, x as linear's X
``layer``     scored routing, gate/up, down and the weighted sum over a token's
              experts, plus the residual; weights in 4 bits

The format: 32 numbers of a row share a power of two, 2^(s-127) with s an
unsigned byte (255: not a number), each is one of +-{0, 0.5, 1, 1.5, 2, 3, 4,
6} times it in four bits (sign, two exponent bits, one mantissa bit), the
even column in the low half of its byte.  Quantising takes s from the block's
largest magnitude, 2^(s-127) = 2^(floor(log2 max) - 2), and rounds to nearest,
ties to even, up to 6.  Shapes are those of the repository's workloads and
generic splits of them.
"""
import math

import torch

own = False

SIGMA, P_OUT, OUTLIER = 0.02, 5e-4, 0.375     # weight spread, share and size of its outliers (workloads.py)
F32, F64, BF16, U8 = torch.float32, torch.float64, torch.bfloat16, torch.uint8
KINDS = {"quantize": 1, "linear": 2, "route": 3, "gate_up": 4, "layer": 5}


# ---------------------------------------------------------------- the cases
def quantize(rows, cols):
    return {"op": "quantize", "rows": rows, "cols": cols}


def linear(rows, cols, batch, x4, bias=False, act="none", residual=False, bf16_out=True):
    return {"op": "linear", "rows": rows, "cols": cols, "batch": batch, "x4": x4, "bias": bias, "act": act,
            "residual": residual, "bf16_out": bf16_out}


def route(tokens, experts, top_k, score, groups, top_groups, group_top=2, bias=True, renorm=True, scale=1.0, bf16=False,
          padding=0.0):
    return {"op": "route", "tokens": tokens, "experts": experts, "top_k": top_k, "score": score, "groups": groups,
            "top_groups": top_groups, "group_top": group_top, "bias": bias, "renorm": renorm, "scale": scale,
            "bf16": bf16, "padding": padding}


def experts_case(op, tokens, experts, top_k, ffn, hidden, x4, groups=1, top_groups=1, skew=0.5, padding=0.0):
    """The router of these is a sigmoid's with a bias, groups by their two best, renormalised and scaled."""
    return {**route(tokens, experts, top_k, "sigmoid", groups, top_groups, scale=2.5, padding=padding), "op": op,
            "ffn": ffn, "hidden": hidden, "x4": x4, "skew": skew}


def listed():
    return [
        # a few tokens' activations on their way into a 4-bit product: latency counts
        dict(quantize(4, 4096), name="quantize 4x4096"),
        # a whole MLP matrix at load time: the memory bounds it
        dict(quantize(14336, 4096), name="quantize 14336x4096"),
        # one token through a key/value projection with a bias: the smallest product
        dict(linear(1024, 4096, 1, False, bias=True), name="linear 1x1024x4096"),
        # a decode batch through the down projection, added to the residual stream
        dict(linear(4096, 14336, 16, False, residual=True, bf16_out=False), name="linear 16x4096x14336"),
        # an odd-length prompt through a wide first MLP matrix with its bias and GELU, bf16 activations
        dict(linear(14336, 4096, 777, False, bias=True, act="gelu_tanh"), name="linear 777x14336x4096"),
        # a long prompt through the same matrix with its activations in 4 bits too: the matrix units bound it
        dict(linear(14336, 4096, 4097, True), name="linear 4097x14336x4096 x4"),
        # routing of a decode batch, and of a long prompt with padded tokens over many experts in groups
        dict(route(16, 64, 6, "sigmoid", 4, 2), name="route 16 of 64"),
        dict(route(16384, 256, 8, "sigmoid", 8, 4, scale=2.5, padding=0.05), name="route 16384 of 256"),
        # gate/up of a decode batch over many experts: a few tokens an expert, the weights' bytes bound it
        dict(experts_case("gate_up", 40, 64, 6, 1408, 2048, False, 8, 4), name="gate_up 40 of 64"),
        # a prompt over large experts, activations in 4 bits
        dict(experts_case("gate_up", 4001, 8, 2, 3584, 4096, True), name="gate_up 4001 of 8 x4"),
        # the whole layer for one token, and for a mid-size batch with padded tokens over uneven experts
        dict(experts_case("layer", 1, 64, 6, 1408, 2048, False, 8, 4), name="layer 1 of 64"),
        dict(experts_case("layer", 600, 32, 4, 1024, 2048, False, 4, 2, skew=1.0, padding=0.1), name="layer 600 of 32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["quantize", "linear", "linear", "linear", "route", "gate_up", "gate_up", "layer", "layer"])
    x4 = rng.random() < 0.4
    if kind == "quantize":
        cols = 32 * _log(rng, 2, 448)
        return quantize(_log(rng, 1, max(2, min(20000, 58000000 // cols))), cols)
    if kind == "linear":
        rows, cols = _log(rng, 64, 16000), 32 * _log(rng, 4, 448)
        batch = _log(rng, 1, min(4097, max(2, int(4e11 / (2 * rows * cols)))))
        return linear(rows, cols, batch, x4, rng.random() < 0.5, rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]),
                      rng.random() < 0.5, rng.random() < 0.6)
    groups = rng.choice([1, 1, 2, 4, 8])
    top_groups = rng.randint(1, groups)
    if kind == "route":
        per = _log(rng, 4, 320) // groups + 1
        return route(_log(rng, 1, 16384), groups * per, rng.randint(1, min(8, top_groups * per)),
                     rng.choice(["sigmoid", "softmax"]), groups, top_groups, rng.choice([1, 2]), rng.random() < 0.7,
                     rng.random() < 0.7, rng.choice([1.0, 2.5]), rng.random() < 0.5, rng.choice([0.0, 0.1]))
    per = max(1, _log(rng, 4, 64) // groups)
    experts, hidden = groups * per, 32 * _log(rng, 16, 128)
    top_k = rng.randint(1, min(6, top_groups * per))
    ffn = 32 * _log(rng, 8, max(9, min(112, int(1.1e8 / (32 * experts * hidden)))))
    most = int(2.2e11 / (2 * top_k * ffn * hidden * {"gate_up": 2, "layer": 3}[kind]))
    tokens = _log(rng, 1, max(2, min(6000, most)))
    return experts_case(kind, tokens, experts, top_k, ffn, hidden, x4 and kind == "gate_up", groups, top_groups,
                        rng.choice([0.0, 0.5, 1.0]), rng.choice([0.0, 0.1]))


# --------------------------------------------------------------- the inputs
def _generator(case, seed, stream):
    return torch.Generator("cuda").manual_seed(seed * 64 + KINDS[case["op"]] * 8 + stream)


def _weights(g, rows, cols):
    """bf16 [rows, cols]: N(0, 0.02) with outliers, as the repository's workloads draw them."""
    w = torch.randn(rows, cols, device="cuda", generator=g).mul_(SIGMA)
    at = torch.randint(w.numel(), (max(1, int(w.numel() * P_OUT)),), device="cuda", generator=g)
    w.view(-1).index_fill_(0, at, OUTLIER)
    return w.to(BF16)


def _matrix(g, rows, cols):
    """A weight as a program keeps it: codes [rows, cols/2] and scales [rows, cols/32] (rows of them 16 bytes apart
    or a multiple), and the framework's handle on the same two tensors."""
    codes, scales = _quantize(_weights(g, rows, cols))
    room = torch.zeros(rows, -(-scales.shape[1] // 16) * 16, dtype=U8, device="cuda")
    room[:, :scales.shape[1]] = scales
    m = {"codes": codes, "scales": room[:, :scales.shape[1]]}
    if own:
        from mlp_matmul_amd import Mx4Matrix
        m["handle"] = Mx4Matrix(m["codes"], m["scales"])
    return m


def _rows(g, *shape):
    """Activations: a few columns are far larger than the others."""
    x = torch.randn(*shape, device="cuda", generator=g)
    x *= torch.where(torch.rand(shape[-1], device="cuda", generator=g) < 0.01, 8.0, 1.0)
    return x.to(BF16)


def _logits(case, g):
    t, e = case["tokens"], case["experts"]
    l = torch.randn(t, e, device="cuda", generator=g)
    l += case.get("skew", 0.5) * torch.randn(e, device="cuda", generator=g)      # some experts are popular
    if case["padding"]:
        l[torch.rand(t, device="cuda", generator=g) < case["padding"]] = -math.inf
    return l.to(BF16) if case["bf16"] else l


def _inputs(case, seed):
    """Everything but the weights."""
    g = _generator(case, seed, 1)
    s = {}
    if case["op"] == "quantize":
        s["x"] = _rows(g, case["rows"], case["cols"])
        return s
    if case["op"] == "linear":
        s["x"] = _rows(g, case["batch"], case["cols"])
        s["bias"] = torch.randn(case["rows"], device="cuda", generator=g) if case["bias"] else None
        s["residual"] = _rows(g, case["batch"], case["rows"]) if case["residual"] else None
        return s
    s["logits"] = _logits(case, g)
    s["balance"] = 0.1 * torch.randn(case["experts"], device="cuda", generator=g) if case["bias"] else None
    if case["op"] == "route":
        return s
    s["x"] = _rows(g, case["tokens"], case["hidden"])
    if case["op"] == "layer":
        s["residual"] = _rows(g, case["tokens"], case["hidden"])
        return s
    _, _, s["offsets"], order, _ = _route(s["logits"], s["balance"], case)
    s["order"] = order[:int(s["offsets"][-1])].contiguous()
    return s


def _shapes(case):
    """(rows, cols, experts) of the case's weights, in their order."""
    if case["op"] == "linear":
        return [(case["rows"], case["cols"], 1)]
    f, h, e = case.get("ffn"), case.get("hidden"), case.get("experts")
    return {"quantize": [], "route": [], "gate_up": [(f, h, e)] * 2, "layer": [(f, h, e)] * 2 + [(h, f, e)]}[case["op"]]


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    s["m"] = [_matrix(_generator(case, seed, 2 + i), e * r, c) for i, (r, c, e) in enumerate(_shapes(case))]
    return s


# --------------------------------------------------------- the plain forms
def _quantize(x):
    """codes [rows, cols/2] and scales [rows, cols/32], uint8."""
    rows, cols = x.shape
    x = x.to(F32).view(rows, cols // 32, 32)
    exponent = (x.abs().amax(2).view(torch.int32) >> 23) & 255
    scale = (exponent - 2).clamp(0, 254)
    up = torch.where(scale == 254, 2.0 ** -127, ((254 - scale) << 23).view(F32))      # 2^(127 - scale)
    v = x * up[:, :, None]
    a = v.abs()
    code = ((a > 0.25).to(U8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)).to(U8)
    code |= torch.signbit(v).to(U8) << 3
    code = code.view(rows, cols // 2, 2)
    return code[:, :, 0] | (code[:, :, 1] << 4), scale.to(U8)


def _values(codes, scales):
    """fp32 [rows, cols] that codes and scales stand for."""
    rows, blocks = scales.shape
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    table = torch.cat([table, -table])
    v = table[torch.stack([codes & 15, codes >> 4], -1).view(rows, blocks, 32).int()]
    s = scales.to(torch.int32)
    s = torch.where(s == 0, 2.0 ** -127, (s << 23).view(F32))
    return (v * s[:, :, None]).view(rows, blocks * 32)


def _activations(x, x4):
    return _values(*_quantize(x)) if x4 else x.to(F32)


def _plain_weight(m, experts, only=None):
    """fp32 [experts, rows, cols] of a weight, or of the experts ``only`` (an index tensor)."""
    codes, scales = m["codes"].view(experts, -1, m["codes"].shape[1]), m["scales"]
    scales = scales.reshape(experts, -1, scales.shape[1])
    if only is not None:
        codes, scales = codes[only], scales[only]
    n, rows, half = codes.shape
    return _values(codes.reshape(n * rows, half), scales.reshape(n * rows, -1)).view(n, rows, half * 2)


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


def _route(logits, balance, c):
    """Scores are rounded to fp32 and their sums with the bias, and the groups', are fp32's: they decide."""
    l = logits.to(F64)
    tokens, experts = l.shape
    alive = l > -math.inf
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-l))
    else:
        top = l.amax(1, keepdim=True)
        part = torch.where(alive, torch.exp(l - torch.where(top == -math.inf, 0.0, top)), 0.0)
        score = torch.where(alive, part / part.sum(1, keepdim=True), 0.0)
    score = score.to(F32)
    key = torch.where(alive, score if balance is None else score + balance, -math.inf)
    if c["groups"] > 1:
        per = experts // c["groups"]
        best = torch.sort(key.view(tokens, c["groups"], per), dim=2, descending=True)[0]
        group = best[:, :, 0]
        if c["group_top"] == 2 and per > 1:
            group = torch.where(best[:, :, 1] > -math.inf, group + best[:, :, 1], group)
        chosen = torch.sort(group, dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
        allowed = torch.zeros(tokens, c["groups"], dtype=torch.bool, device=key.device).scatter_(1, chosen, True)
        key = torch.where(allowed.repeat_interleave(per, 1), key, -math.inf)
    value, ids = torch.sort(key, dim=1, descending=True, stable=True)
    value, ids = value[:, :c["top_k"]], ids[:, :c["top_k"]]
    live = value > -math.inf
    weights = torch.where(live, score.gather(1, ids), 0.0).to(F64)
    if c["renorm"]:
        total = weights.sum(1, keepdim=True)
        weights = torch.where(total > 0, weights / total, 0.0)
    weights = (weights * c["scale"]).to(F32)
    ids = torch.where(live, ids, -1).to(torch.int32)
    bin_of = torch.where(ids < 0, experts, ids).view(-1)
    bin_of, order = torch.sort(bin_of, stable=True)
    offsets = torch.searchsorted(bin_of, torch.arange(experts + 1, device=key.device, dtype=torch.int32)).to(torch.int32)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    place = torch.where(ids.view(-1) < 0, -1, place).view(tokens, -1).to(torch.int32)
    order = torch.where(bin_of == experts, -1, order).to(torch.int32)
    return ids, weights, offsets, order, place


def _grouped(x, ms, offsets):
    """[x_s . W_e(s)^T for each of ms]: x fp32 [n, cols] sorted by expert.  Few rows: each row's own matrix is
    gathered; else every expert's rows are padded to the same number and multiplied in one batch."""
    n, experts = x.shape[0], offsets.numel() - 1
    e = torch.searchsorted(offsets[1:].contiguous(), torch.arange(n, device="cuda", dtype=torch.int32), right=True)
    if n <= experts // 2:
        return [torch.bmm(_plain_weight(m, experts, e), x[:, :, None])[:, :, 0] for m in ms]
    at = torch.arange(n, device="cuda") - offsets[e]
    padded = x.new_zeros(experts, int((offsets[1:] - offsets[:-1]).max()), x.shape[1])
    padded[e, at] = x
    return [torch.bmm(padded, _plain_weight(m, experts).transpose(1, 2).contiguous())[e, at] for m in ms]


def _plain(s):
    c = s["case"]
    if c["op"] == "quantize":
        return _values(*_quantize(s["x"])).to(BF16)
    if c["op"] == "linear":
        v = _activations(s["x"], c["x4"]) @ _plain_weight(s["m"][0], 1)[0].t()
        if s["bias"] is not None:
            v = v + s["bias"]
        v = _act(v, c["act"])
        if s["residual"] is not None:
            v = v + s["residual"].to(F32)
        return v.to(BF16 if c["bf16_out"] else F32)
    if c["op"] == "route":
        return _route(s["logits"], s["balance"], c)
    if c["op"] == "gate_up":
        x = _activations(s["x"], c["x4"])[(s["order"] // c["top_k"]).long()]
        g, u = _grouped(x, s["m"], s["offsets"])
        return (_act(g, "silu") * u).to(BF16)
    ids, weights, offsets, order, place = _route(s["logits"], s["balance"], c)
    n = int(offsets[-1])
    x = s["x"].to(F32)[(order[:n] // c["top_k"]).long()]
    g, u = _grouped(x, s["m"][:2], offsets)
    y = _grouped(_act(g, "silu") * u, s["m"][2:], offsets)[0]
    y = torch.cat([y, y.new_zeros(1, c["hidden"])])              # place -1 reads the zeros at the end
    return ((y[place.long()] * weights[:, :, None]).sum(1) + s["residual"].to(F32)).to(BF16)


# ------------------------------------------------------ the framework's calls
def _own(s):
    import mlp_matmul_amd as uw
    c = s["case"]
    w = [m["handle"] for m in s["m"]]
    if c["op"] == "quantize":
        return uw.mx4_dequantize(uw.mx4_quantize(s["x"]), out_dtype=BF16)
    if c["op"] == "linear":
        x = uw.mx4_quantize(s["x"]) if c["x4"] else s["x"]
        return uw.linear(w[0], x, bias=s["bias"], act=c["act"], residual=s["residual"],
                         out_dtype=BF16 if c["bf16_out"] else F32)
    if c["op"] == "gate_up":
        x = uw.mx4_quantize(s["x"]) if c["x4"] else s["x"]
        return uw.moe_gate_up(w[0], w[1], x, s["offsets"], s["order"], c["top_k"])
    r = uw.moe_route_scored(s["logits"], c["top_k"], score=c["score"], bias=s["balance"], groups=c["groups"],
                            top_groups=c["top_groups"], group_top=c["group_top"], renormalize=c["renorm"],
                            scale=c["scale"])
    if c["op"] == "route":
        return r.ids, r.weights, r.offsets, r.order, r.place
    return uw.moe_experts(w[0], w[1], w[2], s["x"], r, residual=s["residual"], out_dtype=BF16)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------- the definition
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _nearest(x):
    """What quantising bf16 [rows, cols] leaves of it, fp64: the nearest number of each block's grid, of two equally
    near ones that with the even code."""
    b = x.double().reshape(-1, 32)
    top = b.abs().amax(1, keepdim=True)
    half = torch.frexp(top)[0]                                   # top = half 2^e, half in [0.5, 1): top / half is a power of two
    step = torch.where(top > 0, top / half / 8, 1.0).clamp_min(2.0 ** -127)
    a = b.abs() / step
    best, gap = torch.zeros_like(a), a.clone()
    for i, v in enumerate(GRID[1:], 1):
        d = (a - v).abs()
        closer = (d < gap) | ((d == gap) & (i % 2 == 0))
        best, gap = torch.where(closer, v, best), torch.where(closer, d, gap)
    return (torch.copysign(best, b) * step).view(x.shape)


def exact(case, seed):
    """The definitions in 64 bits on the drawn bf16 weights, quantised here, expert by expert."""
    s = _inputs(case, seed)
    if case["op"] == "quantize":
        return _nearest(s["x"])
    ws = [_nearest(_weights(_generator(case, seed, 2 + i), e * r, c)).view(e, r, c)
          for i, (r, c, e) in enumerate(_shapes(case))]
    x = (_nearest(s["x"]) if case.get("x4") else s["x"].double()) if "x" in s else None
    if case["op"] == "linear":
        y = torch.mm(x, ws[0][0].t())
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
    k, experts, groups = case["top_k"], case["experts"], case["groups"]
    l = s["logits"].double()
    dead = l.isneginf()
    score = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l.clamp_min(-1e300), 1).masked_fill(dead, 0)
    key = score.float() + (0 if s["balance"] is None else s["balance"])
    key = key.masked_fill(dead, -math.inf)
    if groups > 1:
        best = torch.topk(key.view(-1, groups, experts // groups), min(case["group_top"], experts // groups), dim=2)[0]
        total = best.nan_to_num(neginf=0.0).sum(2).masked_fill(best[:, :, 0].isneginf(), -math.inf)
        out = torch.argsort(-total, dim=1, stable=True)[:, case["top_groups"]:]
        key.view(-1, groups, experts // groups)[torch.arange(key.shape[0], device="cuda")[:, None], out] = -math.inf
    ids = torch.argsort(-key, dim=1, stable=True)[:, :k]
    dead = key.gather(1, ids).isneginf()
    w = score.gather(1, ids).masked_fill(dead, 0)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    w = w * case["scale"]
    if case["op"] == "route":
        return None, w, None, None, None
    flat = torch.where(dead, -1, ids).reshape(-1)
    rows = [(flat == e).nonzero()[:, 0] for e in range(experts)]       # sorted rows of expert e, as flat slots
    h = [torch.nn.functional.silu(x[r // k] @ ws[0][e].t()) * (x[r // k] @ ws[1][e].t()) for e, r in enumerate(rows)]
    if case["op"] == "gate_up":
        return torch.cat(h)
    y = s["residual"].double()
    for e, r in enumerate(rows):
        y.index_add_(0, r // k, (h[e] @ ws[2][e].t()) * w.reshape(-1)[r, None])
    return y


# --------------------------------------------------------------- what it costs
def work(case):
    """Bytes and operations that a pass cannot do without (weights of the experts with tokens, each read once; 4-bit
    activations are read as bf16 once, what they become is kept on chip at best)."""
    per = 0.5 + 1 / 32
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (4 + per), "flops": n}
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        return {"bytes": t * e * (2 if case["bf16"] else 4) + t * k * 16 + 4 * (2 * e + 1), "flops": t * e}
    if case["op"] == "linear":
        r, c, b = case["rows"], case["cols"], case["batch"]
        n = r * c * per + 2 * b * c + b * r * (2 if case["bf16_out"] else 4)
        return {"bytes": n + 4 * r * case["bias"] + 2 * b * r * case["residual"], "flops": 2 * b * r * c}
    t, e, k, f, h = (case[i] for i in ("tokens", "experts", "top_k", "ffn", "hidden"))
    live = t * (1 - case["padding"])
    used = e * (1 - (1 - k / e) ** live)                         # experts that get a token, evenly routed
    mats = {"gate_up": 2, "layer": 3}[case["op"]]
    n = mats * used * f * h * per + {"gate_up": 2 * t * h + 2 * live * k * f, "layer": 6 * t * h + 4 * t * e}[case["op"]]
    return {"bytes": n, "flops": 2 * live * k * f * h * mats}
