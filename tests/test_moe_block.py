"""The operators around the products in use: the example's block (norm, router,
sorting, products, saved activation, and back), streams, CUDA graphs, calls side by
side, and sizes past 2^31 elements."""
import os
import sys

import pytest
import torch

import fp4_quantization_gb300 as mxq

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

# E4M3 rounds a value by 2^-4 of itself at most, a random sum of such values by 2^-4 of
# its norm at most; a result's bound adds up the quantizations on its way.
E4M3, NVFP4, BF16 = 2.0 ** -4, 2.0 ** -2 + 2.0 ** -4, 2.0 ** -8


def draw(T, E, H, F, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).bfloat16()

    return (normal(T, H), normal(T, H), 1 + 0.2 * normal(H).float(), normal(E, H, scale=H ** -0.5).float(),
            normal(E, 2 * F, H, scale=H ** -0.5), normal(E, H, F, scale=F ** -0.5), normal(T, H))


def block(x, residual, gamma, router, k, w1, w2, experts):
    """The block in fp32, differentiable, with the choice of experts given."""
    h = x + residual
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * gamma
    p = torch.softmax((y @ router.t()).gather(1, experts), 1)
    out = h
    for e in range(len(w1)):
        token, slot = (experts == e).nonzero(as_tuple=True)
        gate, up = (y[token] @ w1[e].t()).chunk(2, 1)
        f = (torch.nn.functional.silu(gate) * up) @ w2[e].t()
        out = out.index_add(0, token, f * p[token, slot].unsqueeze(1))
    return out


def off(got, want):
    return float((got.float() - want).norm() / want.norm())


@pytest.mark.parametrize("T,k,E,H,F", [(200, 2, 6, 256, 384), (64, 4, 8, 160, 96), (33, 1, 5, 512, 128)])
def test_training_block(T, k, E, H, F):
    import moe_layer

    x, r, gamma, router, w1, w2, dout = draw(T, E, H, F, T)
    got = moe_layer.block_step(x, r, gamma, router, k, moe_layer.MXWeights(w1), moe_layer.MXWeights(w2), dout)
    n = mxq.mx_rmsnorm(x, gamma, mxq.OUT_BF16, residual=r)
    experts = mxq.moe_route(n["y"].float() @ router.t(), k)[0].long()
    leaves = [t.float().requires_grad_() for t in (x, gamma, router, w1, w2)]
    want = block(leaves[0], r.float(), leaves[1], leaves[2], k, leaves[3], leaves[4], experts)
    grads = torch.autograd.grad(want, leaves, dout.float())
    # out is h plus what four quantizations (y, W1, h2, W2) move; the gradients of x,
    # gamma and the router take the gate's gradient (x, W1), dy, W2, their own and W1's
    # again, and the checkpoint (twice: act and act'), those of the weights likewise.
    for t, exact, steps in zip(got, (want, *grads), (4, 8, 8, 8, 8, 4)):
        # (With one expert a token the router has no gradient, here nor there.)
        assert (t.float() - exact).norm() <= (steps * E4M3 + 4 * BF16) * exact.norm()


@pytest.mark.parametrize("T,k,E,H,F", [(1, 2, 8, 256, 384), (5, 3, 16, 512, 160)])
def test_decoding_block(T, k, E, H, F):
    import moe_layer

    x, r, gamma, router, w1, w2, _ = draw(T, E, H, F, T)
    got = moe_layer.block_decode(x, r, gamma, router, k, moe_layer.NVWeights(w1), moe_layer.NVWeights(w2))
    n = mxq.mx_rmsnorm(x, gamma, mxq.OUT_BF16, residual=r)
    experts = mxq.moe_route(n["y"].float() @ router.t(), k)[0].long()
    want = block(x.float(), r.float(), gamma, router, k, w1.float(), w2.float(), experts)
    assert off(got, want) <= 2 * NVFP4


def test_checkpoint_in_the_layer():
    import moe_layer

    x, _, _, _, w1, w2, dy = draw(128, 4, 256, 192, 3)
    experts = torch.rand(128, 4, device="cuda").topk(2, 1).indices
    a = moe_layer.train_step(x, experts, moe_layer.MXWeights(w1), moe_layer.MXWeights(w2), dy)
    b = moe_layer.train_step(x, experts, moe_layer.MXWeights(w1), moe_layer.MXWeights(w2), dy, checkpoint=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[3], b[3])       # y and dW2 do not read it
    for s, t in zip((a[1], a[2]), (b[1], b[2])):
        assert 0 < off(t, s.float()) <= 2 * E4M3


@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("T,E", [(1, 3), (40, 4), (96, 2)])
def test_slots_without_an_expert(T, E, checkpoint):
    """They add nothing, wherever they stand: not to the outputs, and not to the rows
    that pad another expert's (one pair of one expert fills 32 of them)."""
    import moe_layer

    x, _, _, _, w1, w2, dy = draw(T, E, 128, 96, T)
    w1, w2 = moe_layer.MXWeights(w1), moe_layer.MXWeights(w2)
    gen = torch.Generator(device="cuda").manual_seed(T)
    experts = torch.randint(0, E, (T, 1), generator=gen, device="cuda")
    p = torch.rand(T, 1, generator=gen, device="cuda")
    for weights in (None, p):
        want = moe_layer.train_step(x, experts, w1, w2, dy, weights, checkpoint)
        none = torch.full_like(experts, -1)
        more = None if weights is None else torch.cat((0 * p, p, 1 + p), 1)
        got = moe_layer.train_step(x, torch.cat((none, experts, none), 1), w1, w2, dy, more, checkpoint)
        if weights is not None:
            assert not got[4][:, 0].any() and not got[4][:, 2].any()
            assert torch.equal(got[4][:, 1:2], want[4])
        # (Sums of the same terms, which buffers of another length may cut otherwise.)
        for s, t in zip(got[:4], want[:4]):
            assert (s.double() - t.double()).norm() <= 2.0 ** -7 * t.double().norm()


# ---------------------------------------------------------------------------
# Streams, graphs, calls side by side
# ---------------------------------------------------------------------------

def calls(seed):
    """One call of each operator on inputs of its own: a function that makes them and
    returns the outputs as a list."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    M, K, T, E, k = 256, 1056, 700, 96, 6
    x, r, dy, dh = ((torch.randn(M, K, generator=gen, device="cuda")).bfloat16() for _ in range(4))
    w = torch.randn(K, generator=gen, device="cuda")
    g = torch.randn(M, 2 * 416, generator=gen, device="cuda").bfloat16()
    logits = torch.randn(T, E, generator=gen, device="cuda")
    bias = torch.randn(E, generator=gen, device="cuda") * 0.1
    dw = torch.randn(T, k, generator=gen, device="cuda")

    def run(stream=None):
        s = {"stream": stream}
        n = mxq.mx_rmsnorm(x, w, 3 | mxq.OUT_BF16, residual=r, **s)
        b = mxq.mx_rmsnorm_backward(dy, n["h"], n["rstd"], w, dh=dh, **s)
        a = mxq.mx_quantize_gated_save(g, 3, **s)
        d = mxq.mx_quantize_dgated_saved(dy[:, :416], a["x_q"], a["x_s"], 3, **s)
        e, p = mxq.moe_route(logits, k, mxq.ROUTE_SIGMOID | mxq.ROUTE_RENORM, bias=bias, groups=8, kept=3, **s)
        l = mxq.moe_route_backward(dw, logits, e, mxq.ROUTE_SIGMOID | mxq.ROUTE_RENORM, **s)
        t = mxq.moe_sort(e, E, **s)
        return [*n.values(), *b.values(), *a.values(), *d.values(), e, p, l, *t.values()]

    return run, (x, r, dy, dh, w, g, logits, bias, dw)


def same(a, b):
    return len(a) == len(b) and all(torch.equal(s, t) for s, t in zip(a, b))


def test_other_streams():
    run, _ = calls(1)
    want = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        inside = run()
    side.synchronize()
    assert same(inside, want)
    got = run(stream=side)
    side.synchronize()
    assert same(got, want)


def test_side_by_side():
    """Two sets of calls under way at a time, many times over."""
    runs = [calls(s)[0] for s in (1, 2)]
    wants = [run() for run in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(20):
        outs = []
        for run, stream in zip(runs, streams):
            with torch.cuda.stream(stream):
                outs.append(run())
        torch.cuda.synchronize()
        assert all(same(o, w) for o, w in zip(outs, wants))


def test_captured_and_replayed():
    run, inputs = calls(3)
    run()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        graphs.append(graph)
        outs.append(out)
    for seed in (4, 5):
        other, new = calls(seed)
        want = other()
        for t, v in zip(inputs, new):
            t.copy_(v)
        for graph, out in zip(graphs, outs):
            graph.replay()
            torch.cuda.synchronize()
            assert same(out, want)


def test_repeated_calls_give_the_same_bits():
    run, _ = calls(6)
    want = run()
    for _ in range(10):
        assert same(run(), want)


# ---------------------------------------------------------------------------
# Past 2^31 elements
# ---------------------------------------------------------------------------

def test_large_norm_and_activation():
    M, K = 262144 + 96, 8224                       # 2.16e9 elements
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(0)
    tail = torch.randn(160, K, generator=gen, device="cuda").bfloat16()
    x.zero_()
    x[-160:] = tail
    w = torch.ones(K, device="cuda")
    out = mxq.mx_rmsnorm(x, w, 3 | mxq.OUT_BF16)
    small = mxq.mx_rmsnorm(tail, w, 3 | mxq.OUT_BF16)
    for name in ("rstd", "y", "q_row", "s_row"):
        assert torch.equal(out[name][-160:], small[name]), name
    assert torch.equal(out["q_col"][:, -160:], small["q_col"]) and torch.equal(out["s_col"][:, -5:], small["s_col"])
    del out
    back = mxq.mx_rmsnorm_backward(x, x, torch.ones(M, device="cuda"), w)["dx"]
    want = mxq.mx_rmsnorm_backward(tail, tail, torch.ones(160, device="cuda"), w)["dx"]
    assert torch.equal(back[-160:], want)
    del back
    # Halves of whole blocks: 2.148e9 elements are left.
    x, tail = x[:, :8192], tail[:, :8192]
    kept = mxq.mx_quantize_gated_save(x, 3)
    want = mxq.mx_quantize_gated_save(tail, 3)
    for name in ("q_row", "s_row", "x_q", "x_s"):
        assert torch.equal(kept[name][-160:], want[name]), name
    assert torch.equal(kept["q_col"][:, -160:], want["q_col"])
    grad = x[:, :4096]
    back = mxq.mx_quantize_dgated_saved(grad, kept["x_q"], kept["x_s"], 3)
    want = mxq.mx_quantize_dgated_saved(tail[:, :4096], want["x_q"], want["x_s"], 3)
    assert torch.equal(back["q_row"][-160:], want["q_row"]) and torch.equal(back["q_col"][:, -160:], want["q_col"])


def test_large_route_and_sort():
    T, E, k = 2 ** 22 + 77, 512, 8                 # 2.15e9 logits
    logits = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    tail = torch.randn(100, E, generator=gen, device="cuda").bfloat16()
    logits[-100:] = tail
    e, w = mxq.moe_route(logits, k)
    te, tw = mxq.moe_route(tail, k)
    assert torch.equal(e[-100:], te) and torch.equal(w[-100:], tw)
    assert torch.equal(e[0], torch.arange(k, device="cuda").int())
    d = mxq.moe_route_backward(w, logits, e)
    assert torch.equal(d[-100:], mxq.moe_route_backward(tw, tail, te))
    del d, logits
    # 3.4e7 pairs: most of them of the first eight experts.
    out = mxq.moe_sort(e, E)
    flat = e.flatten().long()
    sizes = torch.bincount(flat, minlength=E)
    assert torch.equal(out["sizes"].long(), sizes)
    starts = torch.cat((torch.zeros(1, dtype=torch.long, device="cuda"), ((sizes + 31) // 32 * 32).cumsum(0)))
    assert torch.equal(out["offsets"].long(), starts)
    order = flat.argsort(stable=True)
    rank = torch.arange(len(flat), device="cuda") - (sizes.cumsum(0) - sizes)[flat[order]]
    assert torch.equal(out["rows"].flatten()[order].long(), starts[flat[order]] + rank)
    real = out["source"] >= 0
    assert int(real.sum()) == len(flat)
    assert torch.equal(out["rows"].flatten()[out["source"][real].long()].long(), real.nonzero().flatten())


@pytest.mark.parametrize("n", [262144, 262145, 300000, 1000003])
def test_sort_past_what_registers_hold(n):
    gen = torch.Generator(device="cuda").manual_seed(n)
    e = torch.randint(-1, 300, (n,), generator=gen, device="cuda").int()
    out = mxq.moe_sort(e, 299, align=128)
    flat = e.long()
    real = (flat >= 0) & (flat < 299)
    sizes = torch.bincount(flat[real], minlength=299)
    assert torch.equal(out["sizes"].long(), sizes)
    starts = torch.cat((torch.zeros(1, dtype=torch.long, device="cuda"), ((sizes + 127) // 128 * 128).cumsum(0)))
    assert torch.equal(out["offsets"].long(), starts)
    bucket = torch.where(real, flat, 299)
    order = bucket.argsort(stable=True)[:int(real.sum())]
    rank = torch.arange(len(order), device="cuda") - (sizes.cumsum(0) - sizes)[flat[order]]
    rows = torch.full((n,), -1, dtype=torch.long, device="cuda")
    rows[order] = starts[flat[order]] + rank
    assert torch.equal(out["rows"].long(), rows)
    source = torch.full((len(out["source"]),), -1, dtype=torch.long, device="cuda")
    source[rows[order]] = order
    assert torch.equal(out["source"].long(), source)
