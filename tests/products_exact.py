"""bf16 products of small integers: every partial sum, in whatever order, is an integer below 2^24 (|a w| <= 9, K <= 2^17),
exact in f32, so the result is the sum rounded once to bf16 -- bits, whatever the length.  Bounds of rounded sums grow
with K: at 55056 values they are wider than a whole step of k that is lost.  Weights times a power of two keep
all this."""
import math

import torch

MOST = 3


def values(g, *shape, device="cpu"):
    """Integers of [-3, 3], made piece by piece."""
    t = torch.empty(shape, dtype=torch.bfloat16, device=device)
    flat = t.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        flat[i:i + (1 << 28)].random_(-MOST, MOST + 1, generator=g)
    return t


def spread(K):
    """The power of two that brings products of K values near 1."""
    return 2.0 ** -round(math.log2(MOST * MOST * K ** 0.5 / 2))


def product(a, w):
    """Rows a [S][K], weights w [N][K] -> their products, exact in f64."""
    assert a.shape[1] * MOST ** 2 < 1 << 24
    return a.double() @ w.double().t()


def bits(y):
    """f64 integers below 2^24, times a power of two -> bf16: exact in f32, then rounded once."""
    return y.float().to(torch.bfloat16)


def check(got, want, what):
    differ = int((got != bits(want)).sum())
    assert differ == 0, f"{what}: {differ} of {got.numel()} differ"
