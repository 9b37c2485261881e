"""GPU tests of routing by scores and of the experts' part of a layer against
plain definitions in 64 bits.

Which experts are chosen is decided by fp32 numbers that the definition fixes, so
that ids, offsets, order and place are equal.  A weight is a rounded score (half
a step, 2^-24), a sum of at most 16 of them, a division and a product, each off by
2^-24 at most: within 20 * 2^-24 of itself.
"""
import numpy as np
import pytest

import mlp_matmul_amd as uw
from tests.gpu_util import print_case
from tests.mx4_cases import ROUTES
from tests.mx4_util import route_ref
from tests.test_gpu_experts import activate, f64, make_weight, torch_cuda  # noqa: F401
from tests.test_gpu_mx4 import weight

pytestmark = pytest.mark.gpu


def compare(torch, logits, top_k, what, **kw):
    print_case(what)
    a = dict(score="sigmoid", bias=None, groups=1, top_groups=1, group_top=2, renormalize=True, scale=1.0)
    a.update(kw)
    r = uw.moe_route_scored(logits, top_k, **a)
    ids, weights, offsets, order, place = route_ref(logits, top_k, *(a[k] for k in (
        "score", "bias", "groups", "top_groups", "group_top", "renormalize", "scale")))
    for got, want, name in ((r.ids, ids, "ids"), (r.offsets, offsets, "offsets"), (r.order, order, "order"),
                            (r.place, place, "place")):
        assert np.array_equal(got.cpu().numpy(), want), f"{what}: {name}"
    w = r.weights.double().cpu().numpy()
    assert (np.abs(w - weights) <= 20 * 2.0 ** -24 * np.abs(weights) + 1e-37).all(), what
    return r


def logits_of(torch, seed, tokens, experts, pad=0, bf16=False):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(tokens, experts + pad, generator=g) * 2
    return (l.to(torch.bfloat16) if bf16 else l).cuda()[:, :experts]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("tokens,experts,top_k,groups,top_groups", ROUTES)
def test_routing(torch_cuda, tokens, experts, top_k, groups, top_groups, score):
    torch = torch_cuda
    for i, (biased, group_top, renorm, scale) in enumerate(((True, 2, True, 2.5), (False, 1, False, 1.0), (True, 1, True, 1.0))):
        l = logits_of(torch, tokens + i, tokens, experts, pad=i, bf16=i == 2)
        bias = torch.randn(experts, generator=torch.Generator().manual_seed(i)).cuda() * 0.2 if biased else None
        compare(torch, l, top_k, f"scored {tokens} of {experts} top {top_k} groups {groups}/{top_groups} {score} {i}",
                score=score, bias=bias, groups=groups, top_groups=top_groups, group_top=group_top, renormalize=renorm,
                scale=scale)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_ties_and_padding(torch_cuda, score):
    """Equal scores (few values, and scores that meet at 0 and 1), tokens and groups without experts, NaN, infinities
    and a bias of -inf."""
    torch = torch_cuda
    inf = float("inf")
    g = torch.Generator().manual_seed(3)
    l = torch.randint(-2, 3, (300, 48), generator=g).float()
    l[0] = -inf
    l[1] = 100.0
    l[2] = -200.0
    l[3] = torch.linspace(90, 120, 48)
    l[4, 5:] = -inf
    l[5, :24] = float("nan")
    l[6, 7], l[6, 9] = inf, inf
    l[7] = torch.linspace(-inf, 1, 48) if score == "sigmoid" else 3.0e38
    l[8:60][torch.rand(52, 48, generator=g) < 0.7] = -inf
    l[9] = -inf
    l[9, 47] = 0.5
    l[299] = -inf
    bias = torch.randint(-1, 2, (48,), generator=g).float() * 0.25
    bias[13], bias[14] = -inf, float("nan")
    for groups, top_groups, group_top in ((1, 1, 1), (8, 4, 2), (6, 1, 1), (4, 2, 2)):
        for b in (None, bias.cuda()):
            for tokens in (60, 300):
                compare(torch, l[:tokens].cuda(), 6, f"ties {score} {groups}/{top_groups} bias={b is not None} {tokens}", score=score,
                        bias=b, groups=groups, top_groups=top_groups, group_top=group_top, renormalize=groups != 6)


@pytest.mark.parametrize("experts,groups", [(40, 10), (64, 16), (128, 16), (128, 2), (200, 5), (256, 8), (256, 4), (512, 16), (512, 8)])
def test_group_ties(torch_cuda, experts, groups):
    """Groups whose keys are equal, among them those of experts 64 apart and more, and groups of a few experts: the lowest
    index goes first.  Few different logits, so that most keys are equal."""
    torch = torch_cuda
    inf = float("inf")
    g = torch.Generator().manual_seed(experts + groups)
    per = experts // groups
    l = torch.randint(-1, 2, (220, experts), generator=g).float()
    l[0] = 1.0
    l[1] = -200.0
    l[2, :experts - per] = -inf                            # the last group alone
    l[3] = torch.arange(experts).flip(0).float() / experts
    l[4:40][torch.rand(36, experts, generator=g) < 0.9] = -inf
    l[40:80, ::per] = 2.0                                  # every group's best key is the same
    l[219] = -inf
    bias = torch.randint(-1, 2, (experts,), generator=g).float() * 0.25
    for score in ("sigmoid", "softmax"):
        for group_top in (1, 2):
            for b in (None, bias.cuda()):
                for top_groups in sorted({1, groups // 2, groups - 1}):
                    for tokens in (9, 220):
                        compare(torch, l[:tokens].cuda(), min(6, top_groups * per),
                                f"group ties {experts}/{groups} top {top_groups} of {group_top} {score} bias={b is not None} {tokens}",
                                score=score, bias=b, groups=groups, top_groups=top_groups, group_top=group_top)


def test_neighbouring_scores(torch_cuda):
    """Logits one step of fp32 apart, and far tails: which score is larger after its rounding decides."""
    torch = torch_cuda
    for centre in (-90.0, -20.0, -3.0, 0.0, 1.0, 9.0, 16.0):
        base = np.float32(centre)
        vals = [base]
        for _ in range(63):
            vals.append(np.nextafter(vals[-1], np.float32(1e9), dtype=np.float32))
        l = torch.tensor(np.array([np.random.default_rng(i).permutation(vals) for i in range(100)])).cuda()
        for score in ("sigmoid", "softmax"):
            compare(torch, l, 8, f"neighbours of {centre} {score}", score=score, groups=4, top_groups=2)


def test_long_prompt(torch_cuda):
    torch = torch_cuda
    l = logits_of(torch, 5, 5000, 256)
    l[::37] = -float("inf")
    bias = torch.randn(256, generator=torch.Generator().manual_seed(1)).cuda() * 0.1
    compare(torch, l, 8, "scored 5000 of 256", bias=bias, groups=8, top_groups=4, scale=2.5)
    # more tokens than blocks of 64
    big = torch.randn(70000, 12, generator=torch.Generator().manual_seed(2)).cuda()
    compare(torch, big, 3, "scored 70000 of 12", groups=3, top_groups=2)


# ------------------------------------------------------------ the experts on a routing
def experts_ref(torch, x, ws, ids, weights, residual):
    """(sum_j w_j down(h_j) + residual with h in 64 bits, a bound on the error), fp64: h is rounded to bf16, half a
    step of 2^-8 each, and the fp32 sums' errors are (K + 8) 2^-23 of the absolute values'."""
    y = torch.zeros_like(x) if residual is None else f64(residual)
    err = y.abs() * 2.0 ** -23
    for j in range(ids.shape[1]):
        for t in range(ids.shape[0]):
            e = int(ids[t, j])
            if e < 0:
                continue
            g, u, d = (w[e] for w in ws)
            a, b = g @ x[t], u @ x[t]
            ea, eb = ((x.shape[1] + 8) * 2.0 ** -23 * (w.abs() @ x[t].abs()) for w in (g, u))
            s = activate(torch, a, "silu")
            h = s * b
            es = 1.13 * ea + 2.0 ** -20 * (a.abs() + s.abs())
            eh = es * (b.abs() + eb) + s.abs() * eb + 2.0 ** -8 * h.abs() * 1.01
            w = float(weights[t, j])
            y[t] += w * (d @ h)
            err[t] += abs(w) * (d.abs() @ (eh + (d.shape[1] + 40) * 2.0 ** -23 * h.abs()))
    return y, err


FORMS = ("bf16", "palette", "mx4")


def three_weights(torch, form, experts, F, H, seed):
    made = []
    for i, (r, c) in enumerate(((F, H), (F, H), (H, F))):
        if form == "mx4":
            m, v = weight(torch, seed + i, experts * r, c)
            made.append((m, v.view(experts, r, c)))
        else:
            made.append(make_weight(torch, seed + i, experts, r, c, form == "palette"))
    return [m for m, _ in made], [v for _, v in made]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("tokens,experts,top_k,groups,top_groups,F,H", [(1, 8, 2, 2, 1, 128, 192), (1, 64, 6, 8, 4, 64, 128),
                                                                       (40, 12, 3, 4, 2, 192, 64), (150, 4, 2, 1, 1, 64, 320)])
def test_experts(torch_cuda, form, tokens, experts, top_k, groups, top_groups, F, H):
    torch = torch_cuda
    if form == "mx4" and tokens > 1:
        F, H = F + 32, H + 32                              # odd numbers of blocks
    what = f"experts {form} {tokens} of {experts} {F}x{H}"
    print_case(what)
    ws, vs = three_weights(torch, form, experts, F, H, tokens)
    X = torch.randn(tokens, H, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    l = logits_of(torch, 8, tokens, experts)
    if tokens > 1:
        l[tokens // 2] = -float("inf")
    bias = torch.randn(experts, generator=torch.Generator().manual_seed(2)).cuda() * 0.1
    r = uw.moe_route_scored(l, top_k, bias=bias, groups=groups, top_groups=top_groups, scale=1.5)
    for residual, kind in ((None, torch.float32), (X, torch.bfloat16)):
        out = uw.moe_experts(*ws, X, r, residual=residual, out_dtype=kind)
        want, err = experts_ref(torch, f64(X), vs, r.ids.cpu(), f64(r.weights), residual)
        half = torch.finfo(kind).eps / 2
        off = (f64(out) - want).abs() > err + (want.abs() + err) * half + 1e-30
        assert out.dtype == kind and not bool(off.any()), f"{what}: {int(off.sum())} off"
    # in place of the residual, and of X
    y = X.clone()
    uw.moe_experts(*ws, y, r, residual=y, out=y)
    assert torch.equal(y, out), what


@pytest.mark.parametrize("E,k,F,H", [(1, 1, 32, 32), (8, 2, 160, 96), (130, 16, 64, 256), (70, 16, 32, 2080), (6, 3, 4128, 2496),
                                     (512, 4, 96, 544), (6, 3, 4128, 32), (2, 2, 192, 64)])
def test_one_token(torch_cuda, E, k, F, H):
    """Its experts are summed in the down projection's kernel, or where sums are long in one of their own; also with
    slots that have no expert."""
    torch = torch_cuda
    print_case(f"one token, {k} of {E} experts of {F}x{H}")
    ws, vs = three_weights(torch, "mx4", E, F, H, E)
    X = torch.randn(1, H, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    l = logits_of(torch, 8, 1, E)
    for some in (E, max(1, k - 1)):
        l[0, some:] = -float("inf")
        r = uw.moe_route_scored(l, k, scale=1.5)
        assert int((r.ids >= 0).sum()) == min(k, some)
        for residual, kind in ((None, torch.float32), (X, torch.bfloat16)):
            out = uw.moe_experts(*ws, X, r, residual=residual, out_dtype=kind)
            want, err = experts_ref(torch, f64(X), vs, r.ids.cpu(), f64(r.weights), residual)
            limit = err + (want.abs() + err) * (torch.finfo(kind).eps / 2) + 1e-30
            assert not bool(((f64(out) - want).abs() > limit).any())
    l[:] = -float("inf")
    r = uw.moe_route_scored(l, k)
    assert torch.equal(uw.moe_experts(*ws, X, r, residual=X), X.float())
    assert not bool(uw.moe_experts(*ws, X, r).any())


def test_one_token_on_a_bad_routing(torch_cuda):
    """Places and offsets that no router returns: nothing outside is read, slots whose row no expert holds count nothing."""
    torch = torch_cuda
    print_case("one token, bad routing")
    E, k, F, H = 5, 4, 96, 160
    ws, vs = three_weights(torch, "mx4", E, F, H, 2)
    X = torch.randn(1, H, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()

    def made(offsets, place):
        i32 = dict(dtype=torch.int32, device="cuda")
        return uw.Routing(None, torch.tensor([[0.5, 0.25, 1.0, 2.0]], device="cuda"), torch.tensor(offsets, **i32),
                          torch.arange(4, **i32), torch.tensor([place], **i32))

    # rows 0 and 1 of expert 1, row 2 of expert 3
    r = made([0, 0, 2, 2, 3, 3], [1, 2 ** 31 - 1, -7, 2])
    want, err = experts_ref(torch, f64(X), vs, torch.tensor([[1, -1, -1, 3]]), f64(r.weights), None)
    out = uw.moe_experts(*ws, X, r)
    assert bool(((f64(out) - want).abs() <= err + (want.abs() + err) * 2.0 ** -24).all())
    for offsets in ([0, 9, -4, 2 ** 31 - 1, 1, 0], [4, 3, 2, 1, 0, -1], [-2 ** 31] * 6, [2 ** 31 - 1] * 6):
        assert uw.moe_experts(*ws, X, made(offsets, [0, 1, 2, 3])).shape == (1, H)


@pytest.mark.parametrize("form", ["bf16", "palette"])
def test_experts_is_the_layer(torch_cuda, form):
    """On moe_route's routing the result is moe_layer's, bit for bit (from two tokens on)."""
    torch = torch_cuda
    print_case(f"experts against layer {form}")
    ws, _ = three_weights(torch, form, 6, 64, 128, 3)
    X = torch.randn(50, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    l = logits_of(torch, 8, 50, 6)
    assert torch.equal(uw.moe_experts(*ws, X, uw.moe_route(l, 2), residual=X), uw.moe_layer(*ws, X, l, 2, residual=X))
