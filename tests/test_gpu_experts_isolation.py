"""NaN stays with its rows, and offsets that make no sense stay inside the buffers, on every kernel that
the library chooses from: the sizes are checked to reach the kernel that a case is named for."""
import pytest
import torch

import expert_choice as choice
import test_gpu_experts as gpu
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
NAN = float("nan")
ep = gpu.ep

# kernel -> (rows of three or more experts, N of the plain product, K)
PLAIN = {
    "large": ([3000, 0, 4000, 1, 2999], 2064, 400),
    "128x256": ([70] * 40, 1040, 272),
    "64x256": ([45] * 18, 2816, 336),
    "32x256": ([11] * 15 + [100], 2816, 400),
    "128x128": ([16, 33, 0, 40, 7], 4096, 336),
    "64x128": ([4] * 64, 1040, 336),
    "32x64": ([5, 9, 3], 144, 336),
}
GATED = {
    "large": ([3000, 0, 4000, 1, 2999], 1024, 400),
    "128x256": ([70] * 40, 1024, 272),
    "64x256": ([45] * 18, 1792, 336),
    "32x256": ([5, 9, 3], 256, 336),
}


def names(which):
    table = GATED if which == "gated" else PLAIN
    return sorted(table)


def case(kernel, gated, behind):
    counts, n, K = (GATED if gated else PLAIN)[kernel]
    S, N = sum(counts) + behind, 2 * n if gated else n
    assert choice.gemm(S, N, len(counts), gated) == kernel
    return counts, S, N, K


def test_sizes_reach_their_kernels():
    for kernel in PLAIN:
        case(kernel, False, 7)
    for kernel in GATED:
        case(kernel, True, 7)


def spoil(a, a_s, w, w_s, off):
    """NaN in one row of the first expert with rows, behind the segments (values and scales), in all
    weights of the last expert with rows, in one weight row of another, and as a scale byte of a row.
    Returns (rows that are NaN throughout, the expert and weight row that are NaN)."""
    b = off.tolist()
    used = [e for e in range(len(b) - 1) if b[e + 1] > b[e]]
    S = a.shape[0]
    bad = torch.zeros(S, dtype=torch.bool, device=DEV)
    first, other, last = used[0], used[1], used[-1]
    a.view(torch.uint8)[b[first]] = 0x7F
    bad[b[first]] = True
    a_s[b[other + 1] - 1, 0] = 255
    bad[b[other + 1] - 1] = True
    a.view(torch.uint8)[b[-1]:] = 0x7F
    a_s[b[-1]:] = 255
    w.view(torch.uint8)[last] = 0x7F
    w_s[last] = 255
    bad[b[last]:b[last + 1]] = True
    w.view(torch.uint8)[other, 5] = 0xFF
    return bad, other


@pytest.mark.parametrize("kernel", names("plain"))
def test_product_keeps_nan_to_its_rows(ep, kernel):
    counts, S, N, K = case(kernel, False, 7)
    g = gpu.gen(S)
    a, a_s = gpu.rows_of(ep, g, S, K)
    w, w_s = gpu.weights_of(ep, g, len(counts), N, K)
    off = gpu.offsets_of(counts)
    n = sum(counts)
    clean = ep.ep_expert_gemm_fp8(a, a_s, w, w_s, off)[:n].clone()
    rows, e = spoil(a, a_s, w, w_s, off)
    say(f"product with NaN on {kernel}")
    y = torch.full((S, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ep.ep_expert_gemm_fp8(a, a_s, w, w_s, off, y=y)
    torch.cuda.synchronize()
    assert (y[n:] == 7.0).all()
    bad = rows[:n, None].expand(n, N).clone()
    bad[off[e]:off[e + 1], 5] = True
    assert torch.isnan(y[:n][bad]).all()
    assert torch.equal(y[:n][~bad], clean[~bad])


@pytest.mark.parametrize("save", [False, True])
@pytest.mark.parametrize("kernel", names("gated"))
def test_gated_keeps_nan_to_its_rows(ep, kernel, save):
    counts, S, N, K = case(kernel, True, 7)
    I = N // 2
    g = gpu.gen(S + 1)
    a, a_s = gpu.rows_of(ep, g, S, K)
    w, w_s = gpu.weights_of(ep, g, len(counts), N, K)
    off = gpu.offsets_of(counts)
    n = sum(counts)
    ch, cs, cgu = (None if t is None else t[:n].clone() for t in ep.ep_expert_swiglu_fp8(
        a, a_s, w, w_s, off, save_gate_up=save))
    rows, e = spoil(a, a_s, w, w_s, off)
    say(f"gated product with NaN on {kernel} save={save}")
    h = torch.full((S, I), 0x33, dtype=torch.uint8, device=DEV)
    hs = torch.full((S, I // 128), 0x33, dtype=torch.uint8, device=DEV)
    gu = torch.full((S, N), 7.0, dtype=torch.bfloat16, device=DEV) if save else None
    ep.ep_expert_swiglu_fp8(a, a_s, w, w_s, off, h=h, h_scale=hs, gate_up=gu)
    torch.cuda.synchronize()
    assert (h[n:] == 0x33).all() and (hs[n:] == 0x33).all()
    bad = rows[:n, None].expand(n, I).clone()
    bad[off[e]:off[e + 1], 5] = True
    assert torch.isnan(h[:n].view(torch.float8_e4m3fn).float()[bad]).all()
    # the spoilt value leaves its block's scale to the others: rows that lost their largest value may
    # take a smaller scale there, all other blocks and rows are as before
    block = rows[:n, None].expand(n, I // 128).clone()
    block[off[e]:off[e + 1], 0] = True
    same = ~block.repeat_interleave(128, 1)
    assert torch.equal(hs[:n][~block], cs[~block])
    assert torch.equal(h[:n][same], ch.view(torch.uint8)[same])
    if save:
        assert (gu[n:] == 7.0).all()
        bad = rows[:n, None].expand(n, N).clone()
        bad[off[e]:off[e + 1], 5] = True
        assert torch.isnan(gu[:n][bad]).all() and torch.equal(gu[:n][~bad], cgu[~bad])


def nonsense(S, E):
    """Offsets that decrease, overlap or leave the buffer, E + 1 of them."""
    up = torch.linspace(0, S, E + 1).long()
    out = [up.flip(0), up * 3 - S, torch.where(torch.arange(E + 1) % 2 == 0, 0, S),
           torch.where(torch.arange(E + 1) % 2 == 0, 2 ** 30, -2 ** 30)]
    swapped = up.clone()
    swapped[1:-1] = up[1:-1].flip(0)
    return [o.to(torch.int32).to(DEV) for o in out + [swapped]]


@pytest.mark.parametrize("kernel", names("plain"))
def test_product_stays_inside(ep, kernel):
    """Unspecified rows, never an access outside: a buffer with guards on both sides."""
    counts, S, N, K = case(kernel, False, 0)
    E, pad = len(counts), 64
    g = gpu.gen(S + 2)
    a, a_s = gpu.rows_of(ep, g, S, K)
    w, w_s = gpu.weights_of(ep, g, E, N, K)
    y = torch.full((S + 2 * pad, N), 7.0, dtype=torch.bfloat16, device=DEV)
    for i, off in enumerate(nonsense(S, E)):
        say(f"product on {kernel} with offsets {i}")
        ep.ep_expert_gemm_fp8(a, a_s, w, w_s, off, y=y[pad:pad + S])
        torch.cuda.synchronize()
        assert (y[:pad] == 7.0).all() and (y[pad + S:] == 7.0).all()


@pytest.mark.parametrize("kernel", names("gated"))
def test_gated_stays_inside(ep, kernel):
    counts, S, N, K = case(kernel, True, 0)
    E, pad, I = len(counts), 64, N // 2
    g = gpu.gen(S + 3)
    a, a_s = gpu.rows_of(ep, g, S, K)
    w, w_s = gpu.weights_of(ep, g, E, N, K)
    h = torch.full((S + 2 * pad, I), 0x11, dtype=torch.uint8, device=DEV)
    hs = torch.full((S + 2 * pad, I // 128), 0x11, dtype=torch.uint8, device=DEV)
    gu = torch.full((S + 2 * pad, N), 7.0, dtype=torch.bfloat16, device=DEV)
    for i, off in enumerate(nonsense(S, E)):
        say(f"gated product on {kernel} with offsets {i}")
        ep.ep_expert_swiglu_fp8(a, a_s, w, w_s, off, h=h[pad:pad + S], h_scale=hs[pad:pad + S],
                                gate_up=gu[pad:pad + S])
        torch.cuda.synchronize()
        for t, v in ((h, 0x11), (hs, 0x11), (gu, 7.0)):
            assert (t[:pad] == v).all() and (t[pad + S:] == v).all()


# weight gradients: (rows, N, K) of the large tiles, the small ones and split rows
WGRAD = {"large": ([300, 0, 400, 65], 2056, 2312), "small": ([100, 64, 1, 0, 700], 1032, 776),
         "parts": ([1, 4000, 0, 333], 136, 264)}


def wgrad_case(kind):
    counts, N, K = WGRAD[kind]
    got = choice.wgrad(sum(counts) + 5, N, K, len(counts))
    assert kind == (got if got == "large" else "small" if got == 1 else "parts"), got
    return counts, N, K


def test_wgrad_sizes_reach_their_kernels():
    for kind in WGRAD:
        wgrad_case(kind)


@pytest.mark.parametrize("kind", sorted(WGRAD))
def test_weight_gradient_keeps_nan_to_its_expert(ep, kind):
    """NaN rows of one expert, and behind the segments, reach that expert's matrix only; one NaN value
    of dy only its row of it."""
    counts, N, K = wgrad_case(kind)
    S, g = sum(counts) + 5, gpu.gen(N)
    dy, x = gpu.normal(g, S, N), gpu.normal(g, S, K)
    off = gpu.offsets_of(counts)
    clean = ep.ep_expert_wgrad(dy, x, off)
    b = off.tolist()
    used = [e for e in range(len(counts)) if counts[e]]
    dy[b[used[0]], 3] = NAN
    x[b[used[-1]]] = NAN
    dy[sum(counts):], x[sum(counts):] = NAN, NAN
    say(f"weight gradient with NaN: {kind}")
    dw = ep.ep_expert_wgrad(dy, x, off)
    torch.cuda.synchronize()
    assert torch.isnan(dw[used[0], 3]).all() and torch.isnan(dw[used[-1]]).all()
    keep = torch.ones_like(dw, dtype=torch.bool)
    keep[used[0], 3] = False
    keep[used[-1]] = False
    assert torch.equal(dw[keep], clean[keep])


@pytest.mark.parametrize("kind", sorted(WGRAD))
def test_weight_gradient_stays_inside(ep, kind):
    counts, N, K = wgrad_case(kind)
    S, E, g = sum(counts) + 5, len(counts), gpu.gen(K)
    dy, x = gpu.normal(g, S, N), gpu.normal(g, S, K)
    for accumulate in (False, True):
        for i, off in enumerate(nonsense(S, E)):
            say(f"weight gradient {kind} with offsets {i} accumulate={accumulate}")
            buf = torch.full((E + 2, N, K), 7.0, device=DEV)
            ep.ep_expert_wgrad(dy, x, off, grad_w=buf[1:-1], accumulate=accumulate)
            torch.cuda.synchronize()
            assert (buf[0] == 7.0).all() and (buf[-1] == 7.0).all()
            assert torch.isfinite(buf).all()
