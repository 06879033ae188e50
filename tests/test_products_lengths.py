"""A piece of k that a product loses is seen at every length of k that the GPU tests of the bf16 and int8 products use: what
they compare with is checked here against planted losses, on the CPU."""
import pytest
import torch

import product_choice as choice
import product_turns as turns
import products_exact as exact
import products_ref as ref
import test_gpu_products as values
import test_gpu_products_kernels as kernels
import test_gpu_products_limits as limits

# Lengths of operands whose bf16 products are compared bit by bit; the others' within the bounds of products_ref.py
EXACT = sorted({s[2] for s in limits.SHAPES} | {s[2] for s in limits.LONG})


def lengths(bytes_):
    found = {choice.case(name, past, b, kind, behind)[2] for b, kind, name, past in choice.cases() if b == bytes_
             for behind in (0, kernels.BEHIND)}
    found |= {turns.case(c)[2] for c in turns.cases() if c[0] == bytes_}
    found |= {c[5] for c in kernels.SCANNED if c[0] == bytes_}
    found |= {s[4] for s in (values.SHAPES if bytes_ == 2 else values.wide(values.SHAPES))}
    if bytes_ == 1:
        found |= {min(s[2], limits.MAX - 16) for s in limits.SHAPES} | {s[2] for s in limits.LONG}
    return sorted(found)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape):
    return torch.randn(shape, generator=g).to(torch.bfloat16)


def losses(a, step):
    """(values lost, a without them): a step of k -- 128 bytes of every row -- and the least that one load brings."""
    K = a.shape[1]
    for n in (step, step // 8):
        for at in sorted({0, K // 2 // n * n, max(0, (K - 1) // n * n)}):
            v = a.clone()
            v[:, at:at + n] = 0
            yield n, at, v


@pytest.mark.parametrize("K", lengths(2))
def test_bf16(K):
    g = gen(K)
    a, w = normal(g, 8, K), normal(g, 256, K)
    y, err = ref.product_bf16(a, w)
    limit = ref.rounded(y, err)
    for n, at, v in losses(a, 64):
        assert ((ref.product_bf16(v, w)[0] - y).abs() > limit).any(), (n, at)


@pytest.mark.parametrize("K", lengths(1))
def test_int8(K):
    g = gen(K + 1)
    (a, s), (w, ws) = ref.integers(normal(g, 8, K)), ref.integers(normal(g, 64, K))
    y, err = ref.product_int8(a, s, w, ws)
    limit = ref.rounded(y, err)
    for n, at, v in losses(a, 128):
        assert ((ref.product_int8(v, s, w, ws)[0] - y).abs() > limit).any(), (n, at)


@pytest.mark.parametrize("K", EXACT)
def test_exact(K):
    g = gen(K + 2)
    a, w = exact.values(g, 8, K), exact.values(g, 64, K)
    y = exact.product(a, w)
    exact.check(exact.bits(y), y, "itself")
    # any order of sums: steps of 64 from another k on, and four waves' shares
    parts = torch.stack([a[:, k:k + 64].float() @ w[:, k:k + 64].float().t() for k in range(0, K, 64)])
    exact.check(parts.roll(3, 0).sum(0).to(torch.bfloat16), y, "another order")
    exact.check(sum(parts[i::4].sum(0) for i in range(4)).to(torch.bfloat16), y, "four shares")
    for n, at, v in losses(a, 64):
        differ = (exact.bits(exact.product(v, w)) != exact.bits(y)).double().mean()
        assert differ > (0.5 if n == 64 else 0.1), (n, at, differ)
