"""The gradient of the routing weights, the one output of the bf16 layer's backward pass that is a dot product with what the
products made: against f64 autograd of the whole layer."""
import pytest
import torch

import test_gpu_products as layers
from gpu_util import say
from test_gpu_experts import ep, gen, normal  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,I,E,k", [(1, 64, 8, 3, 2), (3, 128, 128, 4, 2), (100, 264, 248, 8, 3),
                                       (900, 512, 384, 4, 2)])
def test_routing_weights_gradient(ep, T, H, I, E, k):  # noqa: F811
    """gtw[t][j] = <grad_out[t], y of pick j>, y rounded once itself and made from a rounded h.  A value of y is off
    by 2^-8 of itself at most, and through h, whose values are off by 2^-8 of theirs at most with signs of
    their own, by 2^-8 of y's root mean square in the mean square over random weights.  With sigma^2 = 2^-16
    sum_c grad_out_c^2 (y_c^2 + mean y^2) that bounds the mean square; 6 sigma, and H 2^-23 of the terms'
    magnitude for sums in f32."""
    say(f"routing weights' gradient T={T} H={H} I={I} E={E} k={k}")
    g = gen(T + H + 2)
    x, logits, w13, w2 = layers.layer_inputs(g, T, H, I, E)
    r = layers.layer(ep, x, logits, k, w13, w2)
    go = normal(g, T, H)
    got = layers.layer_grad(ep, r, go, w13, w2)["gtw"]
    torch.cuda.synchronize()
    tw = r["tw"].double().requires_grad_()
    layers.layer64(x.double(), r["idx"], tw, w13.double(), w2.double()).backward(go.double())
    want = tw.grad
    # y of every pick, [T][k][H], from its formula
    y = torch.stack([layers.layer64(x.double(), r["idx"][:, j:j + 1], torch.ones_like(tw[:, :1]), w13.double(),
                                    w2.double()) for j in range(k)], 1).detach()
    assert torch.allclose((y * go.double()[:, None]).sum(2), want, rtol=1e-9, atol=1e-9)
    g2 = go.double()[:, None] ** 2
    sigma = 2.0 ** -8 * (g2 * (y ** 2 + (y ** 2).mean(2, keepdim=True))).sum(2).sqrt()
    limit = 6 * sigma + H * 2.0 ** -23 * (go.double()[:, None] * y).abs().sum(2)
    say(f"at most {((got.double() - want).abs() / limit).max().item():.3f} of the bound")
    assert got.shape == want.shape and ((got.double() - want).abs() <= limit).all()
    assert ((want.flip(1) - want).abs() > limit).double().mean() > 0.5          # the other picks' would exceed it
