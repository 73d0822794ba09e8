"""The mixture-of-experts example: the library's quantizations and products run
together, against the same layer in fp32.

Bounds.  E4M3 keeps 4 significant bits, so rounding moves a value by at most
2^-4 of itself and a random sum of such values by at most 2^-4 of its norm; the
bound of a result adds up the quantizations on its way (x, W1, h, W2 for y).
E2M1 keeps 2 significant bits: 2^-2 a value, and its blocks' E4M3 scales 2^-4.
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

E4M3, NVFP4 = 2.0 ** -4, 2.0 ** -2 + 2.0 ** -4


def layer(x, experts, w1, w2):
    """The layer in fp32, differentiable."""
    y = torch.zeros_like(x)
    for e in range(len(w1)):
        token, slot = (experts == e).nonzero(as_tuple=True)
        gate, up = (x[token] @ w1[e].t()).chunk(2, 1)
        y = y.index_add(0, token, (torch.nn.functional.silu(gate) * up) @ w2[e].t())
    return y


def off(got, want):
    return float((got.float() - want).norm() / want.norm())


def draw(T, k, E, H, F, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).bfloat16()

    experts = torch.rand(T, E, generator=gen, device="cuda").topk(k, 1).indices
    return (normal(T, H), experts, normal(E, 2 * F, H, scale=H ** -0.5),
            normal(E, H, F, scale=F ** -0.5), normal(T, H))


@pytest.mark.parametrize("T,k,E,H,F", [(200, 2, 6, 256, 384), (7, 1, 9, 128, 96), (64, 4, 4, 160, 64)])
def test_training_step(T, k, E, H, F):
    import moe_layer

    x, experts, w1, w2, dy = draw(T, k, E, H, F, T)
    got = moe_layer.train_step(x, experts, moe_layer.MXWeights(w1), moe_layer.MXWeights(w2), dy)
    leaves = [t.float().requires_grad_() for t in (x, w1, w2)]
    want_y = layer(leaves[0], experts, *leaves[1:])
    want_dx, want_dw1, want_dw2 = torch.autograd.grad(want_y, leaves, dy.float())
    # y: x, W1, h, W2.  dx: those of gate and up (x, W1), dy, W2, their own
    # gradient and W1.  dw1: the same without W1, and x.  dw2: dy and x, W1, h.
    for t, want, steps in zip(got, (want_y, want_dx, want_dw1, want_dw2), (4, 6, 6, 4)):
        assert off(t, want.detach()) <= steps * E4M3


@pytest.mark.parametrize("T,k,E,H,F", [(1, 2, 8, 256, 384), (5, 3, 16, 512, 160)])
def test_decoding_step(T, k, E, H, F):
    import moe_layer

    x, experts, w1, w2, _ = draw(T, k, E, H, F, T)
    got = moe_layer.decode_step(x, experts, moe_layer.NVWeights(w1), moe_layer.NVWeights(w2))
    want = layer(x.float(), experts, w1.float(), w2.float())
    assert off(got, want) <= 2 * NVFP4


def weighted_layer(x, experts, w1, w2, weights):
    """The layer in fp32 with a router's weights, differentiable."""
    y = torch.zeros_like(x)
    for e in range(len(w1)):
        token, slot = (experts == e).nonzero(as_tuple=True)
        gate, up = (x[token] @ w1[e].t()).chunk(2, 1)
        f = (torch.nn.functional.silu(gate) * up) @ w2[e].t()
        y = y.index_add(0, token, f * weights[token, slot].unsqueeze(1))
    return y


def draw_weights(experts, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    return torch.randn(experts.shape, generator=gen, device="cuda").softmax(1)


@pytest.mark.parametrize("T,k,E,H,F", [(200, 2, 6, 256, 384), (64, 4, 4, 160, 64)])
def test_training_step_with_router_weights(T, k, E, H, F):
    import moe_layer

    x, experts, w1, w2, dy = draw(T, k, E, H, F, T)
    weights = draw_weights(experts, T)
    got = moe_layer.train_step(x, experts, moe_layer.MXWeights(w1), moe_layer.MXWeights(w2), dy, weights)
    leaves = [t.float().requires_grad_() for t in (x, w1, w2, weights)]
    want_y = weighted_layer(leaves[0], experts, *leaves[1:])
    want = (want_y, *torch.autograd.grad(want_y, leaves, dy.float()))
    # As test_training_step; the weights' gradients are dy times what y sums.
    for t, exact, steps in zip(got, want, (4, 6, 6, 4, 4)):
        assert off(t, exact.detach()) <= steps * E4M3


@pytest.mark.parametrize("T,k,E,H,F", [(1, 2, 8, 256, 384), (5, 3, 16, 512, 160)])
def test_decoding_step_with_router_weights(T, k, E, H, F):
    import moe_layer

    x, experts, w1, w2, _ = draw(T, k, E, H, F, T)
    weights = draw_weights(experts, T)
    got = moe_layer.decode_step(x, experts, moe_layer.NVWeights(w1), moe_layer.NVWeights(w2), weights)
    want = weighted_layer(x.float(), experts, w1.float(), w2.float(), weights)
    assert off(got, want) <= 2 * NVFP4
