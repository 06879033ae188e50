"""The expert operators against their definitions in 64 bits, within bounds that a lost piece of a sum
exceeds at every length (experts_bounds.py; test_experts_bounds.py plants such mistakes), on every kernel
that the library chooses from."""
import pytest
import torch

import expert_choice as choice
import experts_bounds as bounds
import experts_ref as ref
import test_gpu_experts as gpu
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
NAN = float("nan")
ep = gpu.ep

# (rows of each expert, rows before and behind, N, K) beside the older shapes: the persistent kernel at
# one block of k, an odd number and more than 64 of them, and several row counts of its tiles; few rows
# over many experts
PRODUCTS = [
    ([2500, 0, 700], 3, 1, 4096, 16), ([1800, 0, 2000, 300], 0, 2, 3600, 144),
    ([257, 256, 255, 1, 900], 1, 0, 7168, 2064), ([1100, 3, 800], 0, 5, 4112, 8336),
    ([300] * 70, 0, 0, 272, 400), ([0] * 30 + [1, 0, 2, 5] + [0] * 30, 0, 0, 2048, 7168),
    ([1, 0, 0, 0, 0, 0, 0, 1], 0, 0, 4096, 7168), ([1] * 8 + [0] * 8, 0, 1, 4096, 1040),
]
GATED = [
    # rows of each expert, before, behind, I, K
    ([1], 0, 0, 128, 16), ([0, 3, 20, 0], 1, 2, 256, 208), ([40, 0, 65], 0, 3, 384, 336),
    ([1500], 0, 0, 1408, 512), ([20, 3], 0, 1, 128, 8336), ([90] * 10, 0, 0, 1792, 8208),
    ([45] * 18, 3, 0, 1792, 208), ([45] * 18, 0, 1, 1792, 2000),
    ([2000, 0, 1500, 700], 0, 5, 2816, 400), ([2000, 0, 1500, 700], 2, 1, 2816, 8208),
    ([300] * 70, 1, 0, 256, 144), ([1700, 1, 0, 2050], 0, 0, 2048, 1040), ([1500, 2600], 3, 4, 3584, 16),
    ([0] * 30 + [1, 0, 2, 5] + [0] * 30, 0, 0, 1024, 2064),
]
WGRAD = [
    ([1], 0, 0, 8, 8), ([0, 3, 0], 1, 2, 72, 136), ([31, 32, 33, 0, 64], 0, 3, 264, 40),
    ([5000], 0, 0, 64, 136), ([1, 4000, 0, 333], 3, 2, 136, 264), ([1000, 1], 0, 0, 1040, 776),
    ([16384], 1, 2, 256, 512), ([100, 64, 1, 0, 700], 0, 4, 4104, 776),
    ([0, 3000, 130, 63], 5, 0, 2056, 2312), ([200, 0, 250, 1000], 2, 3, 2056, 4104),
    ([5000, 65, 0, 7000], 0, 1, 2312, 4104),
]


def test_every_kernel_is_reached():
    sizes = lambda c: sum(c[0]) + c[1] + c[2]  # noqa: E731
    assert {choice.gemm(sizes(c), c[3], len(c[0])) for c in gpu.SHAPES + PRODUCTS} == set(choice.GEMM)
    large = [c for c in PRODUCTS if choice.gemm(sizes(c), c[3], len(c[0])) == "large"]
    assert {c[4] for c in large} == {16, 144, 2064, 8336, 400}
    assert {choice.gemm(sizes(c), 2 * c[3], len(c[0]), True) for c in GATED} == {
        "large", "128x256", "64x256", "32x256"}
    large = [c for c in GATED if choice.gemm(sizes(c), 2 * c[3], len(c[0]), True) == "large"]
    assert {c[4] for c in large} == {400, 8208, 144, 1040, 16}
    kinds = [choice.wgrad(sizes(c), c[3], c[4], len(c[0])) for c in WGRAD]
    assert "large" in kinds and 1 in kinds and max(k for k in kinds if k != "large") > 30


def check(got, want, limit, what):
    assert torch.isfinite(got.double()).all(), f"{what}: not finite"
    over = ((got.double() - want).abs() - limit).max().item()
    assert over <= 0, f"{what}: {over:.3g} over the bound"


@pytest.mark.parametrize("shape", gpu.SHAPES + PRODUCTS,
                         ids=lambda s: f"E{len(s[0])}S{sum(s[0])}N{s[3]}K{s[4]}")
def test_product(ep, shape):
    counts, before, behind, N, K = shape
    E, S = len(counts), sum(counts) + before + behind
    say(f"product E={E} S={S} N={N} K={K} on {choice.gemm(S, N, E)}")
    g = gpu.gen(N * 5 + K + S)
    a, a_s = gpu.rows_of(ep, g, S, K)
    w, w_s = gpu.weights_of(ep, g, E, N, K)
    off = gpu.offsets_of(counts, before)
    y = torch.full((S, N), NAN, dtype=torch.bfloat16, device=DEV)
    ep.ep_expert_gemm_fp8(a, a_s, w, w_s, off, y=y)
    torch.cuda.synchronize()
    assert torch.isnan(y[:before]).all() and torch.isnan(y[S - behind:]).all(), "rows outside"
    av = ref.values(a, a_s)
    for e, lo, hi in ref.segments(off):
        if hi > lo:
            wv = ref.weight_values(w[e:e + 1], w_s[e:e + 1])[0]
            want, err = bounds.product(av[lo:hi], a_s[lo:hi], wv, w_s[e])
            check(y[lo:hi], want, bounds.product_bound(want, err), f"expert {e}")


@pytest.mark.parametrize("save", [False, True])
@pytest.mark.parametrize("case", GATED, ids=lambda c: f"E{len(c[0])}S{sum(c[0])}I{c[3]}K{c[4]}")
def test_gated(ep, case, save):
    counts, before, behind, I, K = case
    E, S = len(counts), sum(counts) + before + behind
    say(f"gated E={E} S={S} I={I} K={K} save={save} on {choice.gemm(S, 2 * I, E, True)}")
    g = gpu.gen(I * 5 + K + S)
    a, a_s = gpu.rows_of(ep, g, S, K)
    w, w_s = gpu.weights_of(ep, g, E, 2 * I, K)
    off = gpu.offsets_of(counts, before)
    h = torch.full((S, I), 0x33, dtype=torch.uint8, device=DEV)
    h_s = torch.full((S, I // 128), 0x33, dtype=torch.uint8, device=DEV)
    gu = torch.full((S, 2 * I), NAN, dtype=torch.bfloat16, device=DEV) if save else None
    ep.ep_expert_swiglu_fp8(a, a_s, w, w_s, off, h=h, h_scale=h_s, gate_up=gu)
    torch.cuda.synchronize()
    outside = torch.ones(S, dtype=torch.bool, device=DEV)
    outside[before:S - behind] = False
    assert (h[outside] == 0x33).all() and (h_s[outside] == 0x33).all()
    if save:
        assert torch.isnan(gu[outside]).all()
    av = ref.values(a, a_s)
    for e, lo, hi in ref.segments(off):
        if hi == lo:
            continue
        wv = ref.weight_values(w[e:e + 1], w_s[e:e + 1])[0]
        want, err = bounds.product(av[lo:hi], a_s[lo:hi], wv, w_s[e])
        if save:
            check(gu[lo:hi], want, bounds.product_bound(want, err), f"gate_up of expert {e}")
        hv, herr = bounds.gated(want, err)
        top, slack = (v.view(hi - lo, -1, 128).amax(-1) for v in (hv.abs(), herr))
        byte = h_s[lo:hi].int()
        least = ref.scale_exponent((top - slack).clamp(min=0)) + 127
        assert ((byte >= least) | (top <= slack)).all(), f"scale of expert {e}"
        assert (byte <= ref.scale_exponent(top + slack) + 127).all(), f"scale of expert {e}"
        got = ref.values(h[lo:hi].view(torch.float8_e4m3fn), h_s[lo:hi])
        check(got, hv, bounds.quantised_bound(hv, herr, bounds.row_scales(h_s[lo:hi], I)),
              f"h of expert {e}")


@pytest.mark.parametrize("case", WGRAD, ids=lambda c: f"E{len(c[0])}S{sum(c[0])}N{c[3]}K{c[4]}")
def test_weight_gradient(ep, case):
    """The 2-norm of each expert's error; values of a matrix that lose their rows are seen as such by
    the norm over pieces of it too."""
    counts, before, behind, N, K = case
    E, S = len(counts), sum(counts) + before + behind
    say(f"weight gradient E={E} S={S} N={N} K={K}: {choice.wgrad(S, N, K, E)}")
    g = gpu.gen(N * 5 + K + S)
    dy, x = gpu.normal(g, S, N), gpu.normal(g, S, K)
    dy[:before], x[:before], dy[S - behind:], x[S - behind:] = NAN, NAN, NAN, NAN
    off = gpu.offsets_of(counts, before)
    dw = torch.full((E, N, K), NAN, device=DEV)
    ep.ep_expert_wgrad(dy, x, off, grad_w=dw)
    old = gpu.normal(g, E, N, K).float()
    acc = ep.ep_expert_wgrad(dy, x, off, grad_w=old.clone(), accumulate=True)
    torch.cuda.synchronize()
    for e, lo, hi in ref.segments(off):
        want = dy[lo:hi].double().t() @ x[lo:hi].double()
        limit = bounds.wgrad_norm(hi - lo)
        assert bounds.norm_excess(dw[e].view(1, -1), want.view(1, -1), limit, N * K) <= 0, f"expert {e}"
        if hi == lo:
            assert (dw[e] == 0).all()
    assert torch.equal(acc, old + dw)


@pytest.mark.parametrize("T,H,I,E,k,fp8", gpu.MOE + [(64, 2048, 256, 8, 8, True), (64, 2048, 256, 8, 8, False)])
def test_few_tokens(ep, T, H, I, E, k, fp8):
    say(f"moe tokens T={T} H={H} I={I} E={E} k={k} fp8={fp8}")
    c = gpu.moe_case(ep, T, H, I, E, k, fp8, seed=5)
    out = torch.full((T, H), NAN, dtype=torch.bfloat16, device=DEV)
    ep.ep_moe_tokens(**c, out=out)
    torch.cuda.synchronize()
    want, _ = gpu.moe_ref(c)
    assert torch.isfinite(out).all()
    over = bounds.norm_excess(out, want, bounds.MOE_NORM)
    assert over <= 0, f"{over:.3g} over the bound"
