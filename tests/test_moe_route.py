"""moe_route, moe_route_backward and moe_sort against their definitions.

The choice is compared as whole numbers with that of scores in 64 bits; weights and
gradients are fp32.  Errors: an exponential is off by 2 ulp and its argument by
|l - top| 2^-24, at most 30 2^-24 where the result is not below 1e-13 of the
largest; sums of at most 512 terms in chains of 21; quotients: 100 2^-24 of a
weight bounds them all.  Gradients add the difference g - c, off by 100 2^-24 of the
larger |g|."""
import ctypes
import math

import pytest
import torch

import fp4_quantization_gb300 as mxq
from fp4_quantization_gb300 import _lib
from layer_util import guarded

gpu = pytest.mark.gpu
U = 2.0 ** -24
SIG, RENORM, GMAX = 2048, 4096, 8192


def scores64(l, sigmoid):
    if sigmoid:
        return 1 / (1 + torch.exp(-l))
    top = l.amax(-1, keepdim=True)
    s = torch.exp(l - torch.where(top > -math.inf, top, 0))
    return s / s.sum(-1, keepdim=True).clamp(min=1e-300)


def route64(logits, k, flags, bias=None, groups=1, kept=1, scale=1.0):
    """Experts and weights from the definition, in 64 bits."""
    l = logits.double()
    T, E = l.shape
    free = l > -math.inf
    if bias is not None:
        free = free & (bias > -math.inf)
    s = scores64(l, bool(flags & SIG))
    key = torch.where(free, s if bias is None else s + bias.double(), -math.inf)
    if groups > 1 and kept < groups:
        two = key.view(T, groups, -1).sort(dim=-1, descending=True).values[..., :1 if flags & GMAX else 2].sum(-1)
        order = two.sort(dim=-1, descending=True, stable=True).indices[:, :kept]
        keep = torch.zeros(T, groups, dtype=torch.bool, device=l.device).scatter_(1, order, True)
        free = free & keep.repeat_interleave(E // groups, 1)
    key = torch.where(free, l if bias is None else key, -math.inf)
    chosen = key.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    real = free.gather(1, chosen)
    at = torch.where(real, l.gather(1, chosen), -math.inf)
    if flags & RENORM:
        # Ratios of the scores by their logarithms, which never underflow.
        log = torch.nn.functional.logsigmoid(at) if flags & SIG else at
        log = torch.where(real, log, -math.inf)
        top = log.amax(-1, keepdim=True)
        w = torch.exp(log - torch.where(top > -math.inf, top, 0)) * real
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
    else:
        w = torch.where(real, s.gather(1, chosen), 0.0)
    return torch.where(real, chosen, -1).int(), w * scale


def check_route(logits, k, flags, what="", **kw):
    e, w = mxq.moe_route(logits, k, flags, **kw)
    we, ww = route64(logits, k, flags, **kw)
    bad = (e != we).any(1).nonzero().flatten()
    assert len(bad) == 0, f"{what}: {len(bad)} tokens differ, first {int(bad[0])}: {e[bad[0]].tolist()} for {we[bad[0]].tolist()}"
    off = (w.double() - ww).abs()
    assert (off <= 100 * U * ww + 1e-37).all(), f"{what}: weights off by {float((off / ww.clamp(min=1e-30)).max())}"
    return e, w


def draw(T, E, seed, dtype=torch.float32, spread=1.0, ld=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(T, ld or E, generator=gen, device="cuda") * spread).to(dtype)[:, :E], gen


MODES = [0, SIG, RENORM, SIG | RENORM]
SHAPES = [(1, 1, 1), (1, 8, 2), (5, 31, 4), (6, 32, 32), (9, 33, 3), (130, 64, 4), (3, 100, 8), (257, 128, 6), (64, 129, 1),
          (1000, 256, 8), (2, 257, 16), (33, 512, 32), (70, 160, 6), (41, 192, 8), (9, 260, 5), (300, 384, 8)]


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("flags", MODES)
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_route(T, E, k, flags, dtype):
    l, gen = draw(T, E, T * E + k, dtype, 1.5, E + T % 3)
    bias = torch.randn(E, generator=gen, device="cuda") * 0.1
    check_route(l, k, flags, scale=2.5)
    check_route(l, k, flags, bias=bias)
    check_route(l, k, flags, bias=torch.zeros_like(bias))


@gpu
@pytest.mark.parametrize("gmax", [0, GMAX], ids=["two", "best"])
@pytest.mark.parametrize("flags", MODES)
@pytest.mark.parametrize("T,E,groups,kept,k", [(7, 8, 8, 3, 3), (300, 64, 8, 3, 8), (100, 120, 8, 4, 6), (65, 36, 3, 2, 20),
                                               (400, 256, 8, 4, 8), (50, 512, 32, 5, 16), (20, 42, 21, 20, 5), (9, 16, 4, 4, 4),
                                               (3, 32, 32, 1, 1), (4, 12, 2, 1, 6), (60, 160, 8, 3, 6), (60, 160, 5, 2, 6),
                                               (90, 192, 8, 4, 8), (90, 384, 8, 4, 8), (33, 312, 8, 6, 6)])
def test_groups(T, E, groups, kept, k, flags, gmax):
    for dtype in (torch.bfloat16, torch.float32):
        l, gen = draw(T, E, E + k, dtype)
        bias = torch.randn(E, generator=gen, device="cuda") * 0.1
        check_route(l, k, flags | gmax, groups=groups, kept=kept)
        check_route(l, k, flags | gmax, groups=groups, kept=kept, bias=bias, scale=0.5)


@gpu
@pytest.mark.parametrize("flags", MODES)
@pytest.mark.parametrize("E,groups,kept", [(36, 3, 2), (120, 8, 4), (160, 5, 2), (500, 20, 7)])
def test_groups_that_lanes_share(E, groups, kept, flags):
    """Groups that begin or end inside a lane's experts: a chosen key's expert is looked
    up among keys that another lane has masked.  Many tokens, many times."""
    l, gen = draw(6000, E, E)
    bias = torch.randn(E, generator=gen, device="cuda") * 0.1
    for kw in ({}, {"bias": bias}):
        first = check_route(l, 6, flags, groups=groups, kept=kept, **kw)
        for _ in range(10):
            again = mxq.moe_route(l, 6, flags, groups=groups, kept=kept, **kw)
            assert all(torch.equal(a, b) for a, b in zip(again, first))


@gpu
@pytest.mark.parametrize("flags", MODES)
def test_masked_experts(flags):
    l, gen = draw(400, 48, 3)
    l[torch.rand(400, 48, generator=gen, device="cuda") < torch.linspace(0, 1, 400, device="cuda")[:, None]] = -math.inf
    l[17] = -math.inf                                       # nothing left
    l[18] = -math.inf
    l[18, 47] = 1.0                                         # one left
    low = torch.finfo(torch.float32).min
    l[19] = low                                             # the lowest value is not a mask
    l[20, 5:] = low
    l[21, :40] = -math.inf
    l[21, 40:] = low
    bias = torch.randn(48, generator=gen, device="cuda") * 0.1
    for kw in ({}, {"bias": bias}, {"groups": 6, "kept": 2}, {"groups": 6, "kept": 2, "bias": bias}):
        e, w = check_route(l, 6, flags, str(kw.keys()), **kw)
        assert (e[17] == -1).all() and (w[17] == 0).all()
        # With groups expert 47's has no second expert, so that others are kept.
        assert e[18].tolist() == ([-1] if "groups" in kw else [47]) + [-1] * 5
        assert (w[e < 0] == 0).all()
    shut = bias.clone()
    shut[::2] = -math.inf
    e, _ = check_route(l, 6, flags, bias=shut)
    assert ((e < 0) | (e % 2 == 1)).all()
    b = l.bfloat16()
    b[19] = torch.finfo(torch.bfloat16).min
    check_route(b, 6, flags)


@gpu
@pytest.mark.parametrize("flags", MODES)
def test_ties_and_near_ties(flags):
    """Equal scores go to the lower expert; scores that fp32 cannot tell apart are
    told apart all the same."""
    T, E = 64, 96
    for l in (torch.zeros(T, E, device="cuda"), torch.full((T, E), -0.0, device="cuda"),
              draw(T, E, 1)[0].round(), draw(T, E, 2)[0].round().bfloat16()):
        l[::3, ::2] = -0.0
        for kw in ({}, {"bias": torch.zeros(E, device="cuda")}, {"groups": 8, "kept": 3},
                   {"groups": 8, "kept": 3, "bias": torch.full((E,), 0.25, device="cuda")}):
            check_route(l, 8, flags, "ties", **kw)
    l, gen = draw(T, E, 5)
    if flags & SIG:
        # Keys that differ by their rounding alone, and sigmoids that fp32 rounds to one.
        near = (0.5 - torch.sigmoid(l[:1].double())).float().flatten()
        check_route(l[:1].repeat(T, 1), 8, flags, "near", bias=near)
        check_route(l[:1].repeat(T, 1), 8, flags, "near groups", bias=near, groups=8, kept=4)
        check_route(l + 19, 8, flags, "saturated", bias=torch.randn(E, generator=gen, device="cuda") * 1e-9)
    else:
        near = (0.5 - torch.softmax(l[:1].double(), 1)).float().flatten()
        check_route(l[:1].repeat(T, 1), 8, flags, "near", bias=near)
        check_route(l[:1].repeat(T, 1), 8, flags, "near groups", bias=near, groups=8, kept=4)
    # Logits one step apart.
    step = torch.nextafter(torch.ones(1), torch.full((1,), 2.0)).item() - 1
    check_route(1 + step * torch.randint(0, 50, (T, E), generator=gen, device="cuda").float(), 8, flags, "steps",
                bias=torch.zeros(E, device="cuda"))


# The fp32 keys of a last slot and the next expert tie by the same logit and bias, and a
# third one stands within their error behind them.
@gpu
@pytest.mark.parametrize("flags,k,logits,bias,want", [
    (SIG, 1, (20, 20, 20.5), (0, 0, 0), [2]),
    (SIG, 1, (17.5, 17.5, 18), (0, 0, 0), [2]),
    (SIG, 2, (25, 17.5, 17.5, 18, 17.5), (0, 0, 0, 0, 0), [0, 3]),
    (SIG, 1, (17.5, 17.5, 17.5, 3), (0, 0, 0, 0.03), [0]),
    (0, 1, (0, 0, 1e-8), (0, 0, 0), [2]),
    (0, 2, (10, -8, -8, -7.96875), (0, 0.25, 0.25, 0.25), [0, 3]),
    (0, 2, (10, -8, -8, -8.03125), (0, 0.25, 0.25, 0.25), [0, 1]),
])
def test_near_behind_a_tie(flags, k, logits, bias, want):
    bias = torch.tensor(bias, dtype=torch.float32, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        if dtype == torch.bfloat16 and 1e-8 in logits:
            continue
        l = torch.tensor([logits] * 5, dtype=dtype, device="cuda")
        for renorm in (0, RENORM):
            e, _ = check_route(l, k, flags | renorm, bias=bias)
            assert e.tolist() == [want] * 5


@gpu
@pytest.mark.parametrize("flags", MODES)
@pytest.mark.parametrize("E,groups,kept", [(24, 1, 1), (64, 1, 1), (256, 1, 1), (500, 1, 1), (64, 8, 5), (256, 8, 6), (120, 8, 6), (384, 6, 5)])
@pytest.mark.parametrize("k", [1, 2, 5, 8, 31, 32])
def test_near_behind_many_ties(E, groups, kept, k, flags):
    """Experts of the same logit and bias, and some that are better by less than fp32
    shows, few or many, among them anywhere."""
    T = 300
    gen = torch.Generator(device="cuda").manual_seed(E + k)
    if k > E // groups * kept:
        k = E // groups * kept
    rate = torch.tensor([0.0, 1 / E, 4 / E, 0.2, 0.9], device="cuda")[torch.arange(T, device="cuda") % 5, None]
    better = torch.rand(T, E, generator=gen, device="cuda") < rate
    if flags & SIG:
        l = torch.where(better, 18.0, 17.5)
    else:
        l = torch.where(better, 1e-8, 0.0)
    step = torch.where(torch.rand(E, generator=gen, device="cuda") < 0.5, 0.0, 0.125)
    for bias in (torch.zeros(E, device="cuda"), torch.full((E,), -0.375, device="cuda"), step):
        check_route(l, k, flags, bias=bias, groups=groups, kept=kept)
        if flags & SIG:
            check_route(l.bfloat16(), k, flags, bias=bias, groups=groups, kept=kept)


@gpu
@pytest.mark.parametrize("renorm", [0, RENORM])
def test_logits_apart_by_more_than_fp32(renorm):
    """Softmax logits whose differences are infinite in fp32: a score of zero, whose key is
    its bias exactly, beside thirds that their rounding alone tells from it."""
    third = torch.tensor(1 / 3, dtype=torch.float32)
    below = torch.nextafter(third, torch.zeros(()))
    above = torch.nextafter(third, torch.ones(()))
    for b in (third, below, above):
        for order in ([0, 1, 2, 3], [3, 0, 1, 2], [1, 3, 0, 2]):
            l = torch.tensor([2e38, 2e38, 2e38, -2e38], device="cuda")[order].repeat(3, 1)
            bias = torch.tensor([0, -1, -1, float(b)], device="cuda")[order]
            for k in (1, 2, 3):
                check_route(l, k, renorm, bias=bias)
                check_route(l.bfloat16(), k, renorm, bias=bias)


@gpu
@pytest.mark.parametrize("flags", [0, SIG])
def test_groups_of_huge_biases(flags):
    """Sums of two keys that pass fp32's range, upwards and downwards."""
    l, _ = draw(9, 16, 3)
    for values in ([1e38, 3e38, 2e38, -3e38], [-3e38, -2e38, -3.2e38, -2.5e38], [3e38, 3e38, 3.1e38, 1.0]):
        bias = torch.tensor(values, device="cuda").repeat_interleave(4)
        for kept in (1, 2, 3):
            for gmax in (0, GMAX):
                check_route(l, 4, flags | gmax, bias=bias, groups=4, kept=kept)
        # Groups that a lane's experts do not fill.
        check_route(l[:, :12].contiguous(), 3, flags, bias=bias[:12].contiguous(), groups=3, kept=1)


@gpu
def test_many_tokens_and_large_logits():
    l, gen = draw(20000, 64, 8, spread=30.0)
    for flags in MODES:
        check_route(l, 8, flags, bias=torch.randn(64, generator=gen, device="cuda") * 0.3)
        check_route(l, 8, flags)


@gpu
@pytest.mark.parametrize("flags", MODES)
def test_nan_and_infinity(flags):
    l, gen = draw(20, 40, 9)
    clean_e, clean_w = mxq.moe_route(l, 5, flags)
    l[3, 7] = math.nan
    l[11, 39] = math.inf
    bias = torch.zeros(40, device="cuda")
    for kw in ({}, {"bias": bias}, {"groups": 4, "kept": 2}):
        e, w = mxq.moe_route(l, 5, flags, **kw)
        for t in (3, 11):
            assert (e[t] == -1).all() and w[t].isnan().all()
    e, w = mxq.moe_route(l, 5, flags)
    keep = torch.ones(20, dtype=torch.bool, device="cuda")
    keep[3] = keep[11] = False
    assert torch.equal(e[keep], clean_e[keep]) and torch.equal(w[keep], clean_w[keep])


@gpu
def test_route_outputs_in_place_and_empty():
    l, _ = draw(37, 50, 2)
    e, check_e = guarded((37, 7), torch.int32, 99)
    w, check_w = guarded((37, 7), torch.float32, 99)
    mxq.moe_route(l, 7, experts=e, weights=w)
    check_e()
    check_w()
    assert torch.equal(e, route64(l, 7, RENORM)[0])
    e, w = mxq.moe_route(l[:0], 7)
    assert e.shape == (0, 7) and w.shape == (0, 7)


# ---------------------------------------------------------------------------
# Backward
# ---------------------------------------------------------------------------

def back64(dw, logits, experts, flags, scale):
    l = logits.double().requires_grad_()
    real = (experts >= 0) & (experts < l.shape[1])
    at = experts.long().clamp(0, l.shape[1] - 1)
    s = torch.sigmoid(l) if flags & SIG else torch.softmax(l, 1)
    w = torch.where(real, s.gather(1, at), 0.0)
    if flags & RENORM:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1)
    return torch.autograd.grad((w * scale * dw.double()).sum(), l)[0]


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("flags", MODES)
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_backward(T, E, k, flags, dtype):
    l, gen = draw(T, E, T + E * k, dtype, 1.5, E + T % 5)
    e, _ = mxq.moe_route(l, k, flags)
    dw = torch.randn(T, k, generator=gen, device="cuda")
    got = mxq.moe_route_backward(dw, l, e, flags, scale=2.0)
    assert got.dtype == dtype
    want = back64(dw, l, e, flags, 2.0)
    # Every gradient is a weight (2 at most, with the scale) times differences of g.
    bound = 200 * U * 2 * dw.abs().amax(1, keepdim=True).double() * torch.ones_like(want)
    if dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * want.abs()
    assert ((got.double() - want).abs() <= bound).all()


@gpu
@pytest.mark.parametrize("flags", [RENORM, SIG | RENORM])
def test_backward_of_one_renormalised_expert_is_zero(flags):
    l, gen = draw(200, 72, 8, spread=20.0)
    e, w = mxq.moe_route(l, 1, flags, scale=2.5)
    assert (w == 2.5).all()
    dw = torch.randn(200, 1, generator=gen, device="cuda")
    assert not mxq.moe_route_backward(dw, l, e, flags, scale=2.5).any()


@gpu
@pytest.mark.parametrize("flags", MODES)
def test_backward_odd_choices(flags):
    """Slots without an expert, ids out of range, an expert twice, no expert at all,
    an expert that was masked out of the others' softmax."""
    l, gen = draw(40, 24, 6)
    e = torch.randint(0, 24, (40, 6), generator=gen, device="cuda").int()
    e[0] = -1
    e[1, 2:] = -1
    e[2] = 5
    e[3, 0] = 24
    e[4, 1] = -2 ** 31
    l[5:9, 20:] = -math.inf
    e[5:9] = e[5:9] % 20
    dw = torch.randn(40, 6, generator=gen, device="cuda")
    got = mxq.moe_route_backward(dw, l, e, flags)
    want = back64(dw, l, e, flags, 1.0)
    assert not got[0].any()
    # Up to six slots of one expert add up.
    assert ((got.double() - want).abs() <= 1200 * U * dw.abs().amax(1, keepdim=True)).all()
    out, check = guarded((40, 24), torch.float32, 3)
    assert torch.equal(mxq.moe_route_backward(dw, l, e, flags, dlogits=out), got)
    check()
    wide = torch.full((40, 31), 4.0, device="cuda")
    mxq.moe_route_backward(dw, l, e, flags, dlogits=wide[:, 3:27])
    assert torch.equal(wide[:, 3:27], got) and (wide[:, :3] == 4).all() and (wide[:, 27:] == 4).all()


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("flags", MODES)
def test_backward_where_no_gradient_reaches(flags, dtype):
    """Tokens without an expert, whatever their logits, and slots whose experts' scores
    are all zero: the gradient is zero there, and other tokens' are as without them."""
    l, gen = draw(12, 40, 6, dtype)
    e, _ = mxq.moe_route(l, 4, flags)
    dw = torch.randn(12, 4, generator=gen, device="cuda")
    want = mxq.moe_route_backward(dw, l, e, flags)
    bad = l.clone()
    bad[1, 7] = math.nan
    bad[2, 3] = math.inf
    bad[3] = math.nan
    bad[4] = -math.inf
    bad[5, 20:] = -math.inf
    chosen, w = mxq.moe_route(bad, 4, flags)
    chosen[5] = torch.tensor([20, 21, 39, -1])
    got = mxq.moe_route_backward(dw, bad, chosen, flags)
    assert (chosen[1:5] == -1).all() and not got[1:6].any()
    keep = [0, *range(6, 12)]
    assert torch.equal(got[keep], want[keep])


@gpu
@pytest.mark.parametrize("spread", [1.0, 6.0, 25.0])
@pytest.mark.parametrize("flags", MODES)
def test_backward_of_small_scores(flags, spread):
    """Gradients in proportion to their own scores, however small those are.  A weight or
    score is off by 100 2^-24 of itself (spreads of 30 and more: by |l - top| 2^-24 besides),
    g - c by that of |g| + |c|, and a chosen score's own part and the row's are added."""
    l, gen = draw(300, 64, 11, spread=spread)
    e, _ = mxq.moe_route(l, 6, flags)
    dw = torch.randn(300, 6, generator=gen, device="cuda")
    got = mxq.moe_route_backward(dw, l, e, flags, scale=2.0).double()
    # By the formulas: differences of scores near one would leave rounding in 64 bits too.
    l64, g, at = l.double(), 2 * dw.double(), e.long()
    s = scores64(l64, bool(flags & SIG))
    if flags & RENORM:
        chosen = l64.gather(1, at)
        w = (torch.nn.functional.logsigmoid(chosen) if flags & SIG else chosen).softmax(1)
        slope = scores64(-chosen, True) if flags & SIG else torch.ones_like(w)
        want = torch.zeros_like(s).scatter_(1, at, w * (g - (g * w).sum(1, keepdim=True)) * slope)
        s = torch.zeros_like(s).scatter_(1, at, w * slope)
    elif flags & SIG:
        s = s * scores64(-l64, True)
        want = torch.zeros_like(s).scatter_(1, at, g) * s
    else:
        want = s * (torch.zeros_like(s).scatter_(1, at, g) - (g * s.gather(1, at)).sum(1, keepdim=True))
    steps = 100 + (l.amax(1, keepdim=True) - l.amin(1, keepdim=True)).double()
    bound = 2 * steps * U * s * (2.0 * 2 * dw.abs().amax(1, keepdim=True).double()) + 1e-37
    assert ((got - want).abs() <= bound).all()


@gpu
@pytest.mark.parametrize("flags", MODES)
def test_backward_against_differences(flags):
    l, gen = draw(3, 10, 4)
    e, _ = mxq.moe_route(l, 3, flags)
    dw = torch.randn(3, 3, generator=gen, device="cuda")
    got = mxq.moe_route_backward(dw, l, e, flags)

    def loss(x):
        s = torch.sigmoid(x) if flags & SIG else torch.softmax(x, 1)
        w = s.gather(1, e.long())
        return float(((w / w.sum(1, keepdim=True) if flags & RENORM else w) * dw.double()).sum())

    x = l.double()
    for t in range(3):
        for i in range(10):
            d = torch.zeros_like(x)
            d[t, i] = 1e-5                  # second order: 1e-10 times a third derivative
            slope = (loss(x + d) - loss(x - d)) / 2e-5
            assert abs(float(got[t, i]) - slope) <= 200 * U * float(dw[t].abs().max()) + 1e-9


# ---------------------------------------------------------------------------
# Sorting
# ---------------------------------------------------------------------------

def sort_reference(experts, E, align, length):
    flat = experts.flatten().tolist()
    lists = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if 0 <= e < E:
            lists[e].append(i)
    rows, source, offsets = [-1] * len(flat), [-1] * length, [0]
    for pairs in lists:
        for r, i in enumerate(pairs):
            rows[i] = offsets[-1] + r
            source[offsets[-1] + r] = i
        offsets.append(offsets[-1] + -(-len(pairs) // align) * align)
    return {"rows": rows, "offsets": offsets, "sizes": [len(p) for p in lists], "source": source}


@gpu
@pytest.mark.parametrize("align", [1, 32, 100])
@pytest.mark.parametrize("n,E", [(0, 4), (1, 1), (1, 512), (31, 3), (33, 8), (1000, 64), (4096, 7), (4097, 512), (8192, 1),
                                 (20011, 100), (70000, 256)])
def test_sort(n, E, align):
    gen = torch.Generator(device="cuda").manual_seed(n + E)
    p = torch.randn(E, generator=gen, device="cuda").mul(1.5).softmax(0)
    e = torch.multinomial(p, max(n, 1), replacement=True, generator=gen)[:n].int()
    if n > 20:
        e[torch.rand(n, generator=gen, device="cuda") < 0.05] = -1
        e[3], e[9] = E, -2 ** 31
        e[5] = 2 ** 31 - 1
    length = mxq.moe_sort_rows(n, E, align)
    bufs = {"rows": guarded((n,), torch.int32, 55), "offsets": guarded((E + 1,), torch.int32, 55),
            "sizes": guarded((E,), torch.int32, 55), "source": guarded((length,), torch.int32, 55)}
    out = mxq.moe_sort(e, E, align=align, **{k: t for k, (t, _) in bufs.items()})
    for name, want in sort_reference(e, E, align, length).items():
        assert out[name].tolist() == want, name
        bufs[name][1]()


# Clusters of 1, 2, 4, 8 and 16 CTAs, and pairs in registers or not; experts and rows of
# no pair that end inside a warp, so that its lanes reach the cluster's barriers apart.
@gpu
@pytest.mark.parametrize("n", [600, 1024, 2048, 4096, 8192, 16000, 262145])
@pytest.mark.parametrize("E", [1, 17, 33, 257, 511])
def test_sort_with_lanes_apart(n, E):
    gen = torch.Generator(device="cuda").manual_seed(n + E)
    e = torch.randint(0, E, (n,), generator=gen, device="cuda").int()
    first = mxq.moe_sort(e, E, align=7)
    for name, want in sort_reference(e, E, 7, mxq.moe_sort_rows(n, E, 7)).items():
        assert first[name].tolist() == want, name
    for _ in range(20):
        again = mxq.moe_sort(e, E, align=7)
        assert all(torch.equal(again[name], first[name]) for name in first)


@gpu
def test_sort_shapes():
    e = torch.randint(0, 16, (100, 4), device="cuda").int()
    out = mxq.moe_sort(e, 16)
    assert out["rows"].shape == (100, 4)
    assert torch.equal(out["source"][out["rows"].flatten().long()], torch.arange(400, device="cuda").int())
    all_one = mxq.moe_sort(torch.full((9000,), 3, device="cuda").int(), 5)
    assert all_one["offsets"].tolist() == [0, 0, 0, 0, 9024, 9024]
    none = mxq.moe_sort(torch.full((9000,), -1, device="cuda").int(), 5)
    assert not none["offsets"].any() and (none["rows"] == -1).all() and (none["source"] == -1).all()


# ---------------------------------------------------------------------------
# Refusals
# ---------------------------------------------------------------------------

P = ctypes.c_void_p(4096)


@pytest.mark.parametrize("kw,status", [
    (dict(flags=1), 1), (dict(flags=256), 1), (dict(scale=math.nan), 1), (dict(scale=math.inf), 1), (dict(T=-1), 2),
    (dict(E=0), 2), (dict(E=513, ldl=513), 2), (dict(ldl=63), 2), (dict(k=0), 2), (dict(k=33), 2), (dict(E=4, k=5), 2),
    (dict(groups=0), 2), (dict(groups=3), 2), (dict(groups=64, kept=32), 2), (dict(groups=4, kept=5), 2),
    (dict(groups=4, kept=0), 2), (dict(groups=32, kept=1, k=3), 2), (dict(T=1 << 31), 2),
])
def test_route_refusals(kw, status):
    a = dict(logits=P, ldl=64, bias=None, T=8, E=64, k=4, groups=1, kept=1, scale=1.0, flags=0, experts=P, weights=P, stream=None)
    a.update(kw)
    assert _lib.lib().moe_route(*a.values()) == status


@pytest.mark.parametrize("kw,status", [
    (dict(flags=8192), 1), (dict(flags=1), 1), (dict(scale=math.nan), 1), (dict(T=-1), 2), (dict(E=0), 2),
    (dict(E=1000, ldl=1000, ldd=1000), 2), (dict(ldl=3), 2), (dict(ldd=3), 2), (dict(k=0), 2), (dict(k=40), 2),
])
def test_route_backward_refusals(kw, status):
    a = dict(dw=P, logits=P, ldl=64, experts=P, T=8, E=64, k=4, scale=1.0, flags=0, dlogits=P, ldd=64, stream=None)
    a.update(kw)
    assert _lib.lib().moe_route_backward(*a.values()) == status


@pytest.mark.parametrize("kw", [dict(n=-1), dict(E=0), dict(E=513), dict(align=0), dict(align=1 << 20), dict(source_rows=100),
                                dict(n=1 << 31), dict(source_rows=-1), dict(n=1 << 30, E=512, align=1 << 22)])
def test_sort_refusals(kw):
    a = dict(experts=P, n=64, E=8, align=32, rows=P, offsets=P, sizes=P, source=P, source_rows=1000, stream=None)
    a.update(kw)
    assert _lib.lib().moe_sort(*a.values()) == 2


def test_bindings_refuse_host_tensors():
    l, e = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: mxq.moe_route(l, 2), lambda: mxq.moe_route_backward(torch.zeros(4, 2), l, e), lambda: mxq.moe_sort(e, 8)):
        with pytest.raises(TypeError):
            call()


def test_sort_rows_bound():
    assert mxq.moe_sort_rows(0, 8) == 0 and mxq.moe_sort_rows(1, 8) == 32 and mxq.moe_sort_rows(100, 4, 1) == 100
    assert mxq.moe_sort_rows(100, 4, 32) == 224


@gpu
def test_device_refusals():
    l = torch.zeros(4, 8, device="cuda")
    e = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    dw = torch.zeros(4, 2, device="cuda")
    for bad in (lambda: mxq.moe_route(l.half(), 2), lambda: mxq.moe_route(l.t(), 2), lambda: mxq.moe_route(l, 9),
                lambda: mxq.moe_route(l, 2, bias=torch.zeros(7, device="cuda")), lambda: mxq.moe_route(l, 2, bias=torch.zeros(8)),
                lambda: mxq.moe_route(l, 2, experts=e[:2]), lambda: mxq.moe_route(l, 2, weights=dw.double()),
                lambda: mxq.moe_route_backward(dw, l, e.long()), lambda: mxq.moe_route_backward(dw[:3], l, e),
                lambda: mxq.moe_route_backward(dw, l[:3], e), lambda: mxq.moe_route_backward(dw, l, e, dlogits=l.bfloat16()),
                lambda: mxq.moe_sort(e.long(), 8), lambda: mxq.moe_sort(e.t(), 8), lambda: mxq.moe_sort(e, 0),
                lambda: mxq.moe_sort(e, 8, source=torch.zeros(8, dtype=torch.int32, device="cuda"))):
        with pytest.raises((TypeError, ValueError, mxq.MxqError)):
            bad()
