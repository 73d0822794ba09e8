"""How the operators are wired together in the example's blocks: against the same steps
in torch, with the same roundings at the same places and sums in 64 bits.

Both sides round the same numbers, so that they differ where a sum, off by 2^-20 of its
terms' norm (the products') or less, stands at a rounding's border: one value in 2^11
then leaves for bf16 a step further, by 2^-7 of itself, and of those one in 2^4 reaches
another E4M3 code, by 2^-3.  That is below 2^-10.5 of a norm for each of the ten
roundings on the longest way, 2^-7 with all of them.  What a step leaves
out or takes from the wrong side has to show: a test without a GPU plants such mistakes
in the torch side, and each moves a result by three bounds at least.
"""
import os
import sys

import pytest
import torch

from layer_util import e8m0_values

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

BOUND = 2.0 ** -7


def mx(t):
    """What MXFP8 keeps of t in blocks of 32 along its last axis."""
    b = t.double().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 9, -127).clamp(-127, 127)
    scale = torch.ldexp(torch.ones_like(amax), e)
    q = (b / scale).clamp(-448, 448).float().to(torch.float8_e4m3fn)
    return (q.double() * scale).flatten(-2)


def mx_cols(t):
    return mx(t.transpose(-1, -2)).transpose(-1, -2)


def bf16(t):
    return t.float().bfloat16().double()


def silu_d(x):
    s = torch.sigmoid(x)
    return x * s, s * (1 + x * (1 - s))


def feed_forward(xs, w1, w2, g, sizes, mistake):
    """Rows xs [R, H] sorted by expert, sizes rows each (multiples of 32), g their
    outputs' gradient: f, dx, dw1, dw2."""
    cols = mx if mistake == "rows for columns" else mx_cols
    f, dx = torch.zeros_like(g), torch.zeros_like(xs)
    dw1, dw2 = torch.zeros_like(w1), torch.zeros_like(w2)
    r = 0
    for e, n in enumerate(sizes):
        if n == 0:
            continue
        at = slice(r, r + n)
        r += n
        gate_up = bf16(mx(xs[at]) @ mx(w1[e]).t())
        gate, up = gate_up.chunk(2, 1)
        act = (silu_d(gate)[0] * up).float().double()
        f[at] = bf16(mx(act) @ mx(w2[e]).t())
        dh = bf16(mx(g[at]) @ mx_cols(w2[e]))
        gate, up = (gate_up if mistake == "no checkpoint" else mx(gate_up)).chunk(2, 1)
        value, slope = silu_d(gate)
        d = torch.cat((dh * up * slope, dh * value), 1).float().double()
        dx[at] = bf16(mx(d) @ mx_cols(w1[e]))
        dw1[e] = cols(d).t() @ cols(xs[at])
        dw2[e] = cols(g[at]).t() @ cols(act)
    return f, dx, dw1, dw2


def norm(x, residual, gamma):
    h = bf16(x.double() + residual.double())
    rstd = (h.square().mean(-1, keepdim=True) + 1e-6) ** -0.5
    return h, rstd, h * rstd * gamma.double()


def norm_back(dy, h, rstd, gamma, dh, mistake):
    n, g = h * rstd, dy * gamma.double()
    past = 0 if mistake == "no gradient past the norm" else dh.double()
    return past + rstd * (g - n * (g * n).mean(-1, keepdim=True)), (dy * n).sum(0)


def block_steps(x, residual, gamma, router, experts, w1, w2, dout, mistake=None):
    """The example's block_step with the choice of experts given."""
    T, k = experts.shape
    E = len(w1)
    w1, w2, router, dy = w1.double(), w2.double(), router.double(), dout.double()
    h, rstd, y = norm(x, residual, gamma)
    y = bf16(y)
    p = (y @ router.t()).gather(1, experts).softmax(1)
    flat = experts.flatten()
    counts = [int((flat == e).sum()) for e in range(E)]
    sizes = [-(-n // 32) * 32 for n in counts]
    row = torch.empty_like(flat)
    for e in range(E):
        row[flat == e] = sum(sizes[:e]) + torch.arange(counts[e], device=x.device)
    xs, g = (torch.zeros(sum(sizes), x.shape[1], dtype=torch.float64, device=x.device) for _ in range(2))
    xs[row] = y.repeat_interleave(k, 0)
    g[row] = bf16(dy.repeat_interleave(k, 0) * (1 if mistake == "gradient without weights" else p.view(-1, 1)))
    f, dx, dw1, dw2 = feed_forward(xs, w1, w2, g, sizes, mistake)
    f, dx = f[row].view(T, k, -1), dx[row].view(T, k, -1)
    dp = (f * dy.unsqueeze(1)).sum(-1)
    dlogits = torch.zeros(T, E, dtype=torch.float64, device=x.device)
    dlogits.scatter_(1, experts, p * (dp - (dp * p).sum(1, keepdim=True)))
    dn = bf16(bf16(dx.sum(1)) + (0 if mistake == "no gradient through the router" else dlogits @ router))
    dx, dgamma = norm_back(dn, h, rstd, gamma, dy, mistake)
    out = bf16(h + bf16((f * p.unsqueeze(-1)).sum(1)))
    return out, bf16(dx), dgamma, dlogits.t() @ y, dw1, dw2


def dense_steps(x, residual, gamma, w1, w2, dout, mistake=None):
    """The example's dense_step."""
    h, rstd, y = norm(x, residual, gamma)
    y = bf16(y) if mistake == "codes of the rounded norm" else y.float().double()
    f, dy, dw1, dw2 = feed_forward(y, w1.double(), w2.double(), dout.double(), [len(x)], mistake)
    dx, dgamma = norm_back(dy, h, rstd, gamma, dout, mistake)
    return bf16(h + f), bf16(dx), dgamma, dw1, dw2


def draw(T, E, H, F, device):
    """The gradient is small beside what the layer makes of it, so that dx is not all dout."""
    gen = torch.Generator().manual_seed(T + H)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen) * scale).bfloat16().to(device)

    return (normal(T, H), normal(T, H), 1 + 0.2 * normal(H).float(), normal(E, H, scale=2 * H ** -0.5).float(),
            normal(E, 2 * F, H, scale=2 * H ** -0.5), normal(E, H, F, scale=2 * F ** -0.5), normal(T, H))


def parts(results, dout):
    """With what the norm's input gets beside the gradient past it as a part of its own."""
    return [*results, results[1].double() - dout.double()]


def decode(q, s):
    return (q.view(torch.float8_e4m3fn).double().unflatten(-1, (-1, 32)) * e8m0_values(s).unsqueeze(-1)).flatten(-2)


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


BLOCKS = [(200, 2, 6, 256, 384), (64, 4, 8, 160, 96), (96, 2, 3, 512, 128)]


def choose(x, residual, gamma, router, k):
    return (bf16(norm(x, residual, gamma)[2]) @ router.double().t()).topk(k, 1).indices


@pytest.mark.parametrize("mistake", ["no gradient through the router", "no gradient past the norm", "gradient without weights",
                                     "no checkpoint", "rows for columns"])
def test_mistakes_show_in_the_block(mistake):
    T, k, E, H, F = BLOCKS[1]
    x, r, gamma, router, w1, w2, dout = draw(T, E, H, F, "cpu")
    experts = choose(x, r, gamma, router, k)
    right = parts(block_steps(x, r, gamma, router, experts, w1, w2, dout), dout)
    wrong = parts(block_steps(x, r, gamma, router, experts, w1, w2, dout, mistake), dout)
    assert max(off(b, a) for a, b in zip(right, wrong)) >= 3 * BOUND


@pytest.mark.parametrize("mistake", ["no gradient past the norm", "no checkpoint", "rows for columns"])
def test_mistakes_show_in_the_dense_block(mistake):
    x, r, gamma, _, w1, w2, dout = draw(96, 1, 256, 160, "cpu")
    right = parts(dense_steps(x, r, gamma, w1, w2, dout), dout)
    wrong = parts(dense_steps(x, r, gamma, w1, w2, dout, mistake), dout)
    assert max(off(b, a) for a, b in zip(right, wrong)) >= 3 * BOUND


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E,H,F", BLOCKS)
def test_block_step(T, k, E, H, F):
    import fp4_quantization_gb300 as mxq
    import moe_layer

    x, r, gamma, router, w1, w2, dout = draw(T, E, H, F, "cuda")
    got = moe_layer.block_step(x, r, gamma, router, k, moe_layer.MXWeights(w1), moe_layer.MXWeights(w2), dout)
    n = mxq.mx_rmsnorm(x, gamma, mxq.OUT_BF16, residual=r)
    experts = mxq.moe_route(n["y"].float() @ router.t(), k)[0].long()
    want = block_steps(x, r, gamma, router, experts, w1, w2, dout)
    for name, s, t in zip(("out", "dx", "dgamma", "drouter", "dw1", "dw2", "dx - dout"), parts(got, dout), parts(want, dout)):
        assert off(s, t) <= BOUND, name


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,F", [(32, 128, 96), (96, 256, 160), (416, 1056, 608), (1024, 512, 1024)])
def test_dense_step(T, H, F):
    import moe_layer

    x, r, gamma, _, w1, w2, dout = draw(T, 1, H, F, "cuda")
    got = moe_layer.dense_step(x, r, gamma, moe_layer.MXWeights(w1), moe_layer.MXWeights(w2), dout)
    want = dense_steps(x, r, gamma, w1, w2, dout)
    for name, s, t in zip(("out", "dx", "dgamma", "dw1", "dw2", "dx - dout"), parts(got, dout), parts(want, dout)):
        assert off(s, t) <= BOUND, name


@pytest.mark.gpu
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,H,N", [(32, 128, 96), (160, 1056, 333), (2048, 2048, 512)])
def test_products_of_the_norms_codes(T, H, N, residual):
    """Forward product and weights' gradient of the codes that mx_rmsnorm writes, against
    those of the values that the codes stand for: fp32 sums to 2^-20 of their norm."""
    import fp4_quantization_gb300 as mxq

    x, r, gamma, _, w1, _, _ = draw(T, 1, H, N, "cuda")
    out = mxq.mx_rmsnorm(x, gamma, residual=r if residual else None)
    wq = {key: t[:N] for key, t in mxq.mx_quantize_rowcol(w1[0, :(N + 31) // 32 * 32]).items() if key.endswith("row")}
    g = torch.randn(T, 160, device="cuda").bfloat16()
    gq = mxq.mx_quantize_rowcol(g)
    offsets = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    y = mxq.mx_grouped_gemm(out["q_row"], out["s_row"], wq["q_row"][None], wq["s_row"][None], offsets, out_dtype=torch.float32)
    dw = mxq.mx_grouped_wgrad(gq["q_col"], gq["s_col"], out["q_col"], out["s_col"], offsets)[0]
    values = norm(x, r if residual else torch.zeros_like(x), gamma)[2]
    rows, cols = decode(out["q_row"], out["s_row"]), decode(out["q_col"], out["s_col"])
    # (A value that an fp32 rounding takes over a border has another code.)
    assert off(rows, mx(values)) <= 2.0 ** -10 and off(cols.t(), mx_cols(values)) <= 2.0 ** -10
    for got, a, b in ((y, rows, decode(wq["q_row"], wq["s_row"]).t()), (dw, decode(gq["q_col"], gq["s_col"]), cols.t())):
        limit = 2.0 ** -20 * a.norm(dim=1, keepdim=True) * b.norm(dim=0)
        assert ((got.double() - a @ b).abs() <= limit).all()
