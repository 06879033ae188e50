"""The same rows in different batches: the 8-bit products give the same bits whatever kernel the batch takes (their sums
are exact), the bf16 ones the same within their bounds."""
import pytest
import torch

import product_choice as choice
import products_ref as ref
from gpu_util import say
from test_gpu_experts import ep, gen, offsets_of  # noqa: F401
from test_gpu_products import int8_matrices, int8_rows, matrices, tokens

pytestmark = pytest.mark.gpu
# rows of each of four experts, the first's first ones being those that are compared
BATCHES = [[3, 0, 0, 0], [3, 5, 0, 2], [40, 60, 90, 30], [100, 0, 100, 100], [130, 200, 120, 60], [600, 500, 700, 0],
           [3000, 2900, 1, 2000], [9000, 8000, 9100, 8200]]
N, K = 1040, 2064


def batches(make):
    """(rows of each expert, operand of all rows whose first three are always the same)"""
    first = make(gen(1), 3)
    for i, counts in enumerate(BATCHES):
        x = make(gen(2 + i), sum(counts))
        x[:3] = first
        yield counts, x


def kernels(bytes_, kind):
    return {choice.product(c, N, K, bytes_, kind)[0] for c in BATCHES}


@pytest.mark.parametrize("gated", [False, True])
def test_int8(ep, gated):  # noqa: F811
    assert len(kernels(1, "gated" if gated else "plain")) >= 4
    w, w_s = int8_matrices(gen(0), 4, 2 * N if gated else N, K)
    w_s *= K ** -0.5
    seen = None
    for counts, x in batches(lambda g, S: tokens(g, S, K)):
        say(f"int8 gated={gated} in a batch of {counts}")
        a, a_s = int8_rows(x)
        if gated:
            h, s = ep.ep_expert_swiglu_int8(a, a_s, w, w_s, offsets_of(counts))
            got = [h[:3].clone(), s[:3].clone()]
        else:
            got = [ep.ep_expert_gemm_int8(a, a_s, w, w_s, offsets_of(counts))[:3].clone()]
        torch.cuda.synchronize()
        seen = seen or got
        assert all(torch.equal(a, b) for a, b in zip(got, seen)), counts


@pytest.mark.parametrize("kind", ["plain", "transposed", "gated"])
def test_bf16(ep, kind):  # noqa: F811
    assert len(kernels(2, kind)) >= 4
    w = matrices(gen(0), 4, *((K, N) if kind == "transposed" else (2 * N if kind == "gated" else N, K)))
    if kind == "gated":
        w *= K ** -0.5
    for counts, a in batches(lambda g, S: tokens(g, S, K)):
        say(f"bf16 {kind} in a batch of {counts}")
        if kind == "gated":
            y = ep.ep_expert_swiglu_bf16(a, w, offsets_of(counts))[0]
        else:
            y = ep.ep_expert_gemm_bf16(a, w, offsets_of(counts), transposed=kind == "transposed")
        torch.cuda.synchronize()
        want, err = ref.product_bf16(a[:3], w[0].t() if kind == "transposed" else w[0])
        if kind == "gated":
            want, err = ref.gated(want, err)
        ref.check(y[:3], want, ref.rounded(want, err), f"{counts}")
