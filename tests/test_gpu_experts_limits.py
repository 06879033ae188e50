"""The expert operators at the largest sizes that their documentation allows (2^17 values on an axis, 1024
experts, 64 picks of 64 tokens, rows of 2^20 values to quantise), against their definitions in 64 bits."""
import pytest
import torch

import expert_choice as choice
import experts_bounds as bounds
import experts_ref as ref
import test_gpu_experts as gpu
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
ep = gpu.ep
MAX = 1 << 17


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def product(a, a_byte, w, w_scale):
    """bounds.product for some rows of both and long k (w_scale: the scale at each place of w): the
    additions' errors by the partial sums that occur.  The sum may start at any block of k and go round,
    so a partial sum is a difference of two of these."""
    p = (a[:, None, :] * w[None, :, :]).view(a.shape[0], w.shape[0], -1, 8)
    top = p.sum(-1).cumsum(-1).abs().amax(-1)
    size = p.abs().sum(-1).amax(-1)                       # of one group's own sum
    cut = bounds._tops(a, bounds.row_scales(a_byte, a.shape[1])) @ bounds._tops(w, w_scale).t()
    adds = bounds.additions(a.shape[1]) * 2.0 ** -23 * (2 * top + size)
    return a @ w.t(), bounds.GROUP * 2.0 ** -13 * cut + adds


def expert(w, w_s, e, n):
    """Rows n of expert e's weights as values, and the scale at each place."""
    scale = torch.exp2(w_s[e].double() - 127)[n // 128].repeat_interleave(128, 1)[:, :w.shape[2]]
    return pick(w[e], n).double() * scale, scale


def some(n, k):
    return torch.unique(torch.linspace(0, n - 1, min(n, k)).long()).to(DEV)


def check(got, want, limit, what, share=0.5):
    assert (want.abs() > limit).double().mean() > share, f"{what}: the bound takes zeros"
    assert torch.isfinite(got.double()).all(), f"{what}: not finite"
    over = ((got.double() - want).abs() - limit).max().item()
    assert over <= 0, f"{what}: {over:.3g} over the bound"


def pick(t, rows):
    return t.view(torch.uint8)[rows].view(t.dtype)


PLAIN = [([5], 16, MAX), ([3, 0, 300], MAX, 16), ([2000], 4096, MAX), ([700], MAX, 144),
         ([1] * 1024, 128, 1040), ([300], 4096, MAX), ([1] * 1000 + [200] * 24, 16, 16)]


@pytest.mark.parametrize("counts,N,K", PLAIN, ids=lambda v: f"E{len(v)}" if isinstance(v, list) else v)
def test_product(ep, counts, N, K):
    E, S = len(counts), sum(counts)
    say(f"product E={E} S={S} N={N} K={K} on {choice.gemm(S, N, E)}")
    g = gpu.gen(N + K)
    a, a_s = gpu.rows_of(ep, g, S, K)
    w, w_s = gpu.weights_of(ep, g, E, N, K)
    off = gpu.offsets_of(counts)
    y = ep.ep_expert_gemm_fp8(a, a_s, w, w_s, off)
    torch.cuda.synchronize()
    seg = ref.segments(off)
    for e, lo, hi in [seg[i] for i in sorted({0, E // 2, E - 2, E - 1}) if i >= 0 and counts[i]]:
        r, n = lo + some(hi - lo, 6), some(N, 40)
        av = ref.values(pick(a, r), a_s[r])
        want, err = product(av, a_s[r], *expert(w, w_s, e, n))
        check(y[r][:, n], want, bounds.product_bound(want, err), f"expert {e}")


GATED = [([5], 128, MAX), ([3, 0, 300], 1 << 13, MAX - 16), ([40], MAX, 16), ([3000], MAX, 144),
         ([2500], 1024, MAX), ([1] * 1024, 128, 272)]


@pytest.mark.parametrize("counts,I,K", GATED, ids=lambda v: f"E{len(v)}" if isinstance(v, list) else v)
def test_gated(ep, counts, I, K):
    E, S = len(counts), sum(counts)
    say(f"gated E={E} S={S} I={I} K={K} on {choice.gemm(S, 2 * I, E, True)}")
    g = gpu.gen(I + K)
    a, a_s = gpu.rows_of(ep, g, S, K)
    # the quantiser takes 2^17 rows at most: gate and up on their own, in whole blocks
    w, w_s = (torch.cat(p, 1) for p in zip(*((q.view(torch.uint8), s) for q, s in (
        gpu.weights_of(ep, g, E, I, K) for _ in range(2)))))
    w = w.view(torch.float8_e4m3fn)
    w_s -= 5                                    # gates within silu's bend, not all far out
    off = gpu.offsets_of(counts)
    h, h_s, gu = ep.ep_expert_swiglu_fp8(a, a_s, w, w_s, off, save_gate_up=True)
    torch.cuda.synchronize()
    seg = ref.segments(off)
    for e, lo, hi in [seg[i] for i in sorted({0, E // 2, E - 1}) if counts[i]]:
        r, n = lo + some(hi - lo, 6), some(I, 30)
        av = ref.values(pick(a, r), a_s[r])
        want, err = product(av, a_s[r], *expert(w, w_s, e, torch.cat([n, n + I])))
        check(gu[r][:, torch.cat([n, n + I])], want, bounds.product_bound(want, err), f"gate_up of expert {e}")
        hv, herr = bounds.gated(want, err)
        unit = torch.exp2(h_s[r].double() - 127)[:, n // 128]
        check(pick(h, r).double()[:, n] * unit, hv, bounds.quantised_bound(hv, herr, unit),
              f"h of expert {e}", 0.1)


@pytest.mark.parametrize("counts,N,K", [([5, 0, 40], MAX, 8), ([5, 0, 40], 8, MAX), ([700], MAX, 264),
                                        ([700], 264, MAX), ([5000], 8, MAX), ([2] * 1024, 72, 136)],
                         ids=lambda v: f"E{len(v)}" if isinstance(v, list) else v)
def test_weight_gradient(ep, counts, N, K):
    E, S = len(counts), sum(counts)
    say(f"weight gradient E={E} S={S} N={N} K={K}: {choice.wgrad(S, N, K, E)}")
    g = gpu.gen(N + K)
    dy, x, off = gpu.normal(g, S, N), gpu.normal(g, S, K), gpu.offsets_of(counts)
    dw = ep.ep_expert_wgrad(dy, x, off)
    torch.cuda.synchronize()
    for e, lo, hi in ref.segments(off):
        want = dy[lo:hi].double().t() @ x[lo:hi].double()
        limit = bounds.wgrad_norm(hi - lo)
        assert bounds.norm_excess(dw[e].view(1, -1), want.view(1, -1), limit, N * K) <= 0, f"expert {e}"


@pytest.mark.parametrize("T,H,I,E,k,fp8", [
    (1, MAX, 128, 2, 1, True), (3, MAX, 128, 2, 2, True), (64, MAX, 16, 2, 1, False),
    (1, 16, MAX, 2, 1, True), (5, 16, MAX, 2, 2, False), (64, 16, MAX, 64, 64, True),
    (64, 128, 128, 1024, 8, True), (64, 144, 16, 1024, 64, False)])
def test_few_tokens(ep, T, H, I, E, k, fp8):
    """The limit on the 2-norm as in experts_bounds.py, with the additions of these lengths."""
    say(f"moe tokens T={T} H={H} I={I} E={E} k={k} fp8={fp8}")
    c = gpu.moe_case(ep, T, H, I, E, k, fp8 and I < MAX)
    if fp8 and I == MAX:             # as above; the second weights are within the quantiser's limit
        d = [ep.ep_quantize_weight_fp8(v.contiguous()) for v in (*c["w13"].chunk(2, 1), c["w2"])]
        c["w13"] = torch.cat([d[0]["q"].view(torch.uint8), d[1]["q"].view(torch.uint8)], 1).view(
            torch.float8_e4m3fn)
        c |= dict(w13_scale=torch.cat([d[0]["scale"], d[1]["scale"]], 1), w2=d[2]["q"], w2_scale=d[2]["scale"])
    out = ep.ep_moe_tokens(**c)
    torch.cuda.synchronize()
    want, _ = gpu.moe_ref(c)
    limit = 2.0 ** -8 + max(2.0 ** -10, (H / 2 + I) / 4 * 2.0 ** -23) + 2.0 ** -14
    assert torch.isfinite(out).all() and bounds.norm_excess(out, want, limit) <= 0


def test_quantise(ep):
    g = gpu.gen(1)
    for S, H in ((3, 1 << 20), (4099, 16)):
        say(f"quantise rows {S} x {H}")
        x = gpu.normal(g, S, H)
        q, s = ep.ep_quantize_fp8(x)
        pos = torch.randperm(S * 64, generator=g, device=DEV).to(torch.int32).view(S, 64)
        send, scale = ep.ep_dispatch_fp8(x, pos) if H < 1 << 20 else (None, None)
        torch.cuda.synchronize()
        want, byte = ref.quantize_rows(x)
        assert torch.equal(s, byte)
        gpu.same_e4m3(q, want, "q")
        if send is not None:
            for j in (0, 31, 63):
                assert torch.equal(pick(send, pos[:, j].long()).view(torch.uint8), q.view(torch.uint8))
                assert torch.equal(scale[pos[:, j].long()], s)
    for E, N, K in ((2, MAX, 16), (1, 16, MAX), (1024, 16, 144)):
        say(f"quantise weights {E} x {N} x {K}")
        w = gpu.normal(g, E, N, K)
        d = ep.ep_quantize_weight_fp8(w, transposed=True)
        torch.cuda.synchronize()
        want, byte = ref.quantize_weight(w)
        assert torch.equal(d["scale"], byte) and torch.equal(d["scale_t"], byte.transpose(1, 2))
        gpu.same_e4m3(d["q"], want, "q")
        assert torch.equal(d["q_t"].view(torch.uint8), d["q"].view(torch.uint8).transpose(1, 2))


def test_activation_gradient(ep):
    g = gpu.gen(2)
    S, I = 5, MAX
    say("activation gradient of 2^17 values a row")
    dh, gu = gpu.normal(g, S, I), gpu.normal(g, S, 2 * I)
    dgu, h = ep.ep_swiglu_grad(dh, gu)
    cols = some(I, 4096)
    # I % 8 == 0 pieces of the same values, at a small size that other tests check
    few, hf = ep.ep_swiglu_grad(dh[:, cols].contiguous(), torch.cat([gu[:, cols], gu[:, cols + I]], 1))
    torch.cuda.synchronize()
    n = len(cols)
    assert n % 8 == 0
    assert torch.equal(h[:, cols], hf) and torch.equal(dgu[:, cols], few[:, :n])
    assert torch.equal(dgu[:, cols + I], few[:, n:])
