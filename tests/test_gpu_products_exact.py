"""bf16 products of small integers, bit by bit (products_exact.py): at the longest k, and where an operand passes 2^31
values, on both sides of that place, nothing of a sum is lost."""
import pytest
import torch

import product_choice as choice
import products_exact as exact
import products_ref as ref
import test_gpu_products_limits as limits
from gpu_util import DEV, say
from test_gpu_experts import ep, gen, offsets_of  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def check(ep, S, E, N, K, kind, off, rows_of):  # noqa: F811
    """`rows_of`: (expert, its rows to look at) of what is compared, all columns of them."""
    g = gen(S + N + K)
    a = exact.values(g, S, K, device=DEV)
    w = exact.values(g, *((E, K, N) if kind == "transposed" else (E, 2 * N if kind == "gated" else N, K)), device=DEV)
    if kind == "gated":
        w *= exact.spread(K)
        h, y = ep.ep_expert_swiglu_bf16(a, w, off, save_gate_up=True)
    else:
        y = ep.ep_expert_gemm_bf16(a, w, off, transposed=kind == "transposed")
    torch.cuda.synchronize()
    for e, r in rows_of:
        x = a[r]
        # the weights' channels piece by piece: 64 bits take four times their bytes
        for n in range(0, y.shape[1], 1 << 14):
            part = w[e][:, n:n + (1 << 14)].t() if kind == "transposed" else w[e][n:n + (1 << 14)]
            exact.check(y[r, n:n + (1 << 14)], exact.product(x, part), f"expert {e}, columns from {n}")
        if kind == "gated":
            n = torch.unique(torch.linspace(0, N - 1, min(N, 200)).long()).to(DEV)
            gu = exact.product(x, w[e][torch.cat([n, N + n])])
            want, err = ref.gated(gu, torch.zeros_like(gu))
            ref.check(h[r][:, n], want, ref.rounded(want, err), f"h of expert {e}")


@pytest.mark.parametrize("kind", ["plain", "transposed", "gated"])
@pytest.mark.parametrize("counts,N,K", limits.SHAPES, ids=limits.ids)
def test_largest_sizes(ep, counts, N, K, kind):  # noqa: F811
    E, S = len(counts), sum(counts)
    say(f"exact bf16 {kind} E={E} S={S} N={N} K={K} on {choice.product(counts, N, K, 2, kind)}")
    off = offsets_of(counts)
    seg = ref.segments(off)
    some = [seg[i] for i in sorted({0, len(seg) // 2, len(seg) - 1})]
    check(ep, S, E, N, K, kind, off, [(e, lo + limits.some(hi - lo, 6)) for e, lo, hi in some])


@pytest.mark.parametrize("kind", ["plain", "transposed", "gated"])
@pytest.mark.parametrize("S,N,K,E", limits.LONG)
def test_long(ep, S, N, K, E, kind):  # noqa: F811
    assert max(S * K, S * N, E * N * K) > 2 ** 31
    say(f"exact bf16 {kind} past 2^31: S={S} N={N} K={K} E={E}")
    if kind == "gated":
        N //= 2
    off, rows, experts = limits.long_case(S, N, K, E)
    check(ep, S, E, N, K, kind, off, [(e, rows[experts == e]) for e in torch.unique(experts).tolist()])
