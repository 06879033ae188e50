"""The expert operators where an operand passes 2^31 values, each operand in turn, on the kernels that
large buffers reach: rows and experts on both sides of 2^31 values and bytes, at the segments' cuts and
at the ends, against the definitions in 64 bits (bounds: experts_bounds.py)."""
import pytest
import torch

import expert_choice as choice
import experts_bounds as bounds
import experts_ref as ref
import test_gpu_experts as gpu
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
ep = gpu.ep


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def around(places, S, width=20):
    """Rows around the places, within [0, S)."""
    r = torch.cat([torch.arange(p - width, p + width) for p in places])
    return torch.unique(r[(r >= 0) & (r < S)]).to(DEV)


def check(got, want, limit, what, share=0.5):
    """Within the limit, which zeros would exceed at more than `share` of the places."""
    assert (want.abs() > limit).double().mean() > share, f"{what}: the bound takes zeros"
    assert torch.isfinite(got.double()).all(), f"{what}: not finite"
    over = ((got.double() - want).abs() - limit).max().item()
    assert over <= 0, f"{what}: {over:.3g} over the bound"


def random_rows(g, S, K):
    """Any e4m3 values but NaN, scales from 2^-3 to 2^4."""
    a = torch.randint(0, 256, (S, K), generator=g, device=DEV, dtype=torch.uint8)
    a[(a & 0x7F) == 0x7F] = 0x30
    s = torch.randint(124, 132, (S, ref.blocks(K)), generator=g, device=DEV, dtype=torch.uint8)
    return a.view(torch.float8_e4m3fn), s


def take(t, rows):
    return t.view(torch.uint8)[rows].view(t.dtype)


# (kernel, S, N, K, E): rows of a, rows of y, and weights past 2^31
PLAIN = [("large", 1_060_000, 512, 2064, 3), ("large", 530_000, 4112, 272, 3),
         ("64x128", 40_000, 16, 55_056, 1024), ("64x128", 40_000, 55_056, 16, 1024),
         ("128x256", 100_000, 22_032, 16, 1024), ("64x128", 300, 4096, 4112, 150),
         ("32x64", 5, 2064, 7168, 160)]


def product_case(ep, S, N, K, E):
    g = gpu.gen(S + N)
    a, a_s = random_rows(g, S, K)
    w = torch.randint(0, 0x70, (E, N, K), generator=g, device=DEV, dtype=torch.uint8)
    w ^= (w & 1) << 7
    w_s = torch.randint(124, 132, (E, ref.blocks(N), ref.blocks(K)), generator=g, device=DEV,
                        dtype=torch.uint8)
    off = torch.linspace(0, S, E + 1).long()
    for p in (2 ** 31 // K - 3, 2 ** 31 // N + 5):       # a segment that starts at a place of its own
        e = int((off - p).abs()[1:-1].argmin()) + 1
        if off[e - 1] < p < off[e + 1]:
            off[e] = p
    return a, a_s, w.view(torch.float8_e4m3fn), w_s, off


def seen(off, S, E, N, K):
    """Rows and their experts: at 0, the ends, a few cuts, 2^31 of a and of y, and of the weights."""
    at = [0, S, 2 ** 31 // K, 2 ** 31 // N, 2 ** 32 // N, *off[1:-1][:: max(1, E // 4)].tolist()]
    at += [int(off[min(E - 1, 2 ** 31 // (N * K) + d)]) for d in (0, 1)] + [int(off[E - 1])]
    rows = around(at, S, 8)
    return rows, torch.searchsorted(off.to(DEV), rows, right=True) - 1


@pytest.mark.parametrize("kernel,S,N,K,E", PLAIN)
def test_product(ep, kernel, S, N, K, E):
    assert choice.gemm(S, N, E) == kernel and max(S * K, S * N, E * N * K) > 2 ** 31
    say(f"product past 2^31 on {kernel}: S={S} N={N} K={K} E={E}")
    a, a_s, w, w_s, off = product_case(ep, S, N, K, E)
    y = ep.ep_expert_gemm_fp8(a, a_s, w, w_s, off.to(torch.int32).to(DEV))
    torch.cuda.synchronize()
    rows, experts = seen(off, S, E, N, K)
    for e in torch.unique(experts).tolist():
        r = rows[experts == e]
        av = ref.values(take(a, r), a_s[r])
        wv = ref.weight_values(take(w, torch.tensor([e], device=DEV)), w_s[e:e + 1])[0]
        want, err = bounds.product(av, a_s[r], wv, w_s[e])
        check(y[r], want, bounds.product_bound(want, err), f"expert {e}")


# rows of a and of gate_up; of h and of gate_up; weights
@pytest.mark.parametrize("kernel,S,I,K,E", [
    ("large", 1_060_000, 1024, 2064, 3), ("large", 530_000, 4096, 144, 3),
    ("64x256", 300, 2048, 4112, 150), ("64x256", 40_000, 128, 55_056, 1024)])
def test_gated(ep, kernel, S, I, K, E):
    N = 2 * I
    assert choice.gemm(S, N, E, True) == kernel and max(S * K, S * I, E * N * K) > 2 ** 31
    say(f"gated product past 2^31 on {kernel}: S={S} I={I} K={K} E={E}")
    a, a_s, w, w_s, off = product_case(ep, S, N, K, E)
    w_s -= 20                                           # gates within silu's bend, not all far out
    h, h_s, gu = ep.ep_expert_swiglu_fp8(a, a_s, w, w_s, off.to(torch.int32).to(DEV), save_gate_up=True)
    torch.cuda.synchronize()
    rows, experts = seen(off, S, E, N, K)
    rows = torch.unique(torch.cat([rows, around([2 ** 31 // I], S)]))
    experts = torch.searchsorted(off.to(DEV), rows, right=True) - 1
    for e in torch.unique(experts).tolist():
        r = rows[experts == e]
        av = ref.values(take(a, r), a_s[r])
        wv = ref.weight_values(take(w, torch.tensor([e], device=DEV)), w_s[e:e + 1])[0]
        want, err = bounds.product(av, a_s[r], wv, w_s[e])
        check(gu[r], want, bounds.product_bound(want, err), f"gate_up of expert {e}")
        hv, herr = bounds.gated(want, err)
        check(ref.values(take(h, r), h_s[r]), hv,
              bounds.quantised_bound(hv, herr, bounds.row_scales(h_s[r], I)), f"h of expert {e}", 0.2)


@pytest.mark.parametrize("kind,S,N,K", [("large", 530_000, 4096, 4112), ("parts", 1_130_000, 128, 2048),
                                        ("parts", 1_130_000, 2048, 128), ("small", 530_000, 4096, 904)])
def test_weight_gradient_rows(ep, kind, S, N, K):
    """Rows past 2^31 values: only a few hundred rows of dy differ from zero, around 0, the segments'
    cut, 2^31 values and bytes of either operand and the end, so that a row from a wrong address
    changes the sums by far more than the bound."""
    E = 2 if kind != "small" else 1
    got = choice.wgrad(S, N, K, E)
    assert kind == ("small" if got == 1 else got if got == "large" else "parts")
    assert S * max(N, K) > 2 ** 31
    say(f"weight gradient past 2^31 rows: {kind} S={S} N={N} K={K}")
    g = gpu.gen(S + N + K)
    x = torch.empty((S, K), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    cut = 2 ** 31 // max(N, K) - 5
    off = [0, cut, S] if E == 2 else [0, S]
    rows = around([0, cut, S] + [2 ** b // n for b in (30, 31, 32) for n in (N, K)], S)
    dy = torch.zeros((S, N), dtype=torch.bfloat16, device=DEV)
    dy[rows] = gpu.normal(g, len(rows), N)
    dw = ep.ep_expert_wgrad(dy, x, torch.tensor(off, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    for e in range(E):
        r = rows[(rows >= off[e]) & (rows < off[e + 1])]
        assert len(r) >= 20
        v, u = dy[r].double(), x[r].double()
        want = v.t() @ u
        # zeros add nothing: two additions for each row at most, and parts that are joined
        limit = bounds.additions(len(r) * 8) * 2.0 ** -23 * (v.abs().t() @ u.abs()) + 2.0 ** -24 * want.abs()
        check(dw[e], want, limit, f"expert {e}", 0.9)


@pytest.mark.parametrize("kind,rows,N,K", [("large", 200, 4096, 4112), ("small", 7, 4096, 4112)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradient_matrices(ep, kind, rows, N, K, accumulate):
    """The output past 2^31 values."""
    E = 130
    S = E * rows
    got = choice.wgrad(S, N, K, E)
    assert kind == (got if got == "large" else "small") and E * N * K > 2 ** 31
    say(f"weight gradient of 2^31 weights: {kind} accumulate={accumulate}")
    g = gpu.gen(rows)
    dy, x = gpu.normal(g, S, N), gpu.normal(g, S, K)
    dw = torch.full((E, N, K), 0.5 if accumulate else float("nan"), device=DEV)
    ep.ep_expert_wgrad(dy, x, gpu.offsets_of([rows] * E), grad_w=dw, accumulate=accumulate)
    torch.cuda.synchronize()
    for e in (0, 1, 2 ** 29 // (N * K), 2 ** 30 // (N * K), 2 ** 31 // (N * K), 128, 129):
        v, u = dy[e * rows:(e + 1) * rows].double(), x[e * rows:(e + 1) * rows].double()
        want = v.t() @ u
        limit = bounds.additions(rows * 4) * 2.0 ** -23 * (v.abs().t() @ u.abs())
        if accumulate:
            want += 0.5
        check(dw[e], want, limit + 2.0 ** -23 * want.abs(), f"expert {e}")
    del dy, x
    assert torch.isfinite(dw.view(-1)[:: 4099]).all()


def test_dispatch(ep):
    """Quantised rows past 2^31 bytes: every row where it belongs."""
    T, k, H = 33_000, 8, 8208
    say("fp8 dispatch past 2^31")
    g = gpu.gen(9)
    x = gpu.normal(g, T, H)
    pos = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32).view(T, k)
    send, scale = ep.ep_dispatch_fp8(x, pos)
    q, s = ep.ep_quantize_fp8(x)
    torch.cuda.synchronize()
    assert send.numel() > 2 ** 31
    for j in range(k):
        assert torch.equal(take(send, pos[:, j].long()).view(torch.uint8), q.view(torch.uint8))
        assert torch.equal(scale[pos[:, j].long()], s)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("T", [1, 3, 40])
def test_few_tokens(ep, T, fp8):
    """Both weights past 2^31 values, quantised by the library: picks of experts on both sides."""
    E, H, I, k = 260, 4096, 2048, 4
    say(f"few tokens, weights past 2^31: T={T} fp8={fp8}")
    g = gpu.gen(T)
    w13 = torch.empty((E, 2 * I, H), dtype=torch.bfloat16, device=DEV).normal_(0, H ** -0.5, generator=g)
    w2 = torch.empty((E, H, I), dtype=torch.bfloat16, device=DEV).normal_(0, I ** -0.5, generator=g)
    assert w2.numel() > 2 ** 31
    places = torch.tensor([0, 63, 64, 127, 128, 129, 255, 256, 259], device=DEV, dtype=torch.int32)
    c = dict(x=gpu.normal(g, T, H), topk_w=torch.rand((T, k), generator=g, device=DEV), w13=w13, w2=w2,
             w13_scale=None, w2_scale=None)
    pick = torch.rand((T, len(places)), generator=g, device=DEV).argsort(1)[:, :k]
    c["topk_idx"] = places[pick].contiguous()
    if fp8:
        d13, d2 = ep.ep_quantize_weight_fp8(w13, transposed=True), ep.ep_quantize_weight_fp8(w2)
        torch.cuda.synchronize()
        for d, w in ((d13, w13), (d2, w2)):
            for e in (0, 127, 128, 255, 256, 259):
                want, byte = ref.quantize_weight(w[e:e + 1])
                gpu.same_e4m3(d["q"][e:e + 1], want, f"expert {e}")
                assert torch.equal(d["scale"][e:e + 1], byte)
                if "q_t" in d:
                    assert torch.equal(d["q_t"][e].view(torch.uint8), d["q"][e].view(torch.uint8).t())
        c |= dict(w13=d13["q"], w13_scale=d13["scale"], w2=d2["q"], w2_scale=d2["scale"])
    out = ep.ep_moe_tokens(**c)
    torch.cuda.synchronize()
    want, _ = gpu.moe_ref(c)
    assert bounds.norm_excess(out, want, bounds.MOE_NORM) <= 0
