"""Plain definitions in 64 bits of the microscaled 4-bit format and of the
scored router, on the CPU."""
import numpy as np
import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def quantize_ref(x):
    """(codes [rows, cols/2], scales [rows, cols/32]) uint8 of x [rows, cols]."""
    rows, cols = x.shape
    b = x.detach().double().cpu().reshape(rows, cols // 32, 32)
    finite = torch.isfinite(b).all(2)
    b = torch.where(finite[:, :, None], b, 0.0)
    top = b.abs().amax(2)
    e = torch.frexp(top)[1].long() - 1                                   # floor(log2 top)
    s = torch.where(top > 0, (e - 2 + 127).clamp(0, 254), 0)
    v = b.abs() / torch.ldexp(torch.ones_like(top), s - 127)[:, :, None]
    gap = (v[..., None] - GRID).abs()
    near = gap == gap.amin(-1, keepdim=True)
    even = torch.arange(8) % 2 == 0
    pick = torch.where((near & even).any(-1), (near & even).to(torch.int8).argmax(-1), near.to(torch.int8).argmax(-1))
    code = pick.to(torch.uint8) | (torch.signbit(b).to(torch.uint8) << 3)
    code = torch.where(finite[:, :, None], code, 0).to(torch.uint8).view(rows, cols // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), torch.where(finite, s, 255).to(torch.uint8)


def values_ref(codes, scales):
    """fp64 [rows, cols]; NaN where the scale is 255."""
    codes, scales = codes.cpu(), scales.cpu()
    rows, blocks = scales.shape
    table = torch.cat([GRID, -GRID])
    v = table[torch.stack([codes & 15, codes >> 4], -1).view(rows, blocks, 32).long()]
    f = torch.where(scales == 255, float("nan"), torch.ldexp(torch.ones(rows, blocks, dtype=torch.float64), scales.long() - 127))
    return (v * f[:, :, None]).view(rows, blocks * 32)


def route_ref(logits, top_k, score, bias, groups, top_groups, group_top, renormalize, scale):
    """(ids, weights fp64, offsets, order, place) token by token."""
    l = logits.detach().double().cpu().numpy()
    l = np.where(l == np.inf, np.finfo(np.float32).max, l)
    dead = ~(l > -np.inf)
    tokens, experts = l.shape
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            s64 = 1 / (1 + np.exp(-np.where(dead, 0, l)))
        else:
            z = np.where(dead, -np.inf, l)
            top = z.max(1, keepdims=True, initial=-np.inf)
            p = np.exp(np.where(dead, -np.inf, z - np.where(np.isinf(top), 0, top)))
            s64 = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
    s = s64.astype(np.float32)
    key = s if bias is None else s + bias.detach().float().cpu().numpy()
    key = np.where(dead | ~(key > -np.inf), -np.inf, np.minimum(key, np.finfo(np.float32).max)).astype(np.float32)
    per = experts // groups
    ids = np.full((tokens, top_k), -1, np.int32)
    weights = np.zeros((tokens, top_k))
    for t in range(tokens):
        k = key[t].copy()
        if groups > 1:
            g = -np.sort(-k.reshape(groups, per), 1)
            both = g[:, 0].copy()
            if group_top == 2 and per > 1:
                two = g[:, 1] > -np.inf
                with np.errstate(over="ignore"):
                    both[two] = np.minimum(g[two, 0] + g[two, 1], np.finfo(np.float32).max)
            out = np.argsort(-both, kind="stable")[top_groups:]
            k.reshape(groups, per)[out] = -np.inf
        best = np.argsort(-k, kind="stable")[:top_k]
        best = best[k[best] > -np.inf]
        ids[t, :len(best)] = best
        w = s[t, best].astype(np.float64)
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else w * 0
        weights[t, :len(best)] = w * scale
    flat = ids.reshape(-1)
    order = np.argsort(np.where(flat < 0, experts, flat), kind="stable").astype(np.int32)
    n = int((flat >= 0).sum())
    place = np.full(flat.shape, -1, np.int32)
    place[order[:n]] = np.arange(n)
    order[n:] = -1
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[flat >= 0], minlength=experts))]).astype(np.int32)
    return ids, weights, offsets, order, place.reshape(tokens, top_k)
