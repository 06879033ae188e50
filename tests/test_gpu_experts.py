"""The expert operators against their definitions in 64 bits (experts_ref.py, where the bounds are
derived): quantisation, the grouped products, their gradients and the few-token layer, each at the
sizes, segments and values where it can go wrong, and together as a model's layer uses them."""
import pytest
import torch

import experts_ref as ref
from experts_ref import BF16, E4M3, F32
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module")
def ep():
    from combine_ep_route_topk_amd import ep as mod
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    return mod


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def offsets_of(counts, start=0):
    c = torch.tensor([start] + list(counts))
    return torch.cumsum(c, 0).to(torch.int32).to(DEV)


def rows_of(ep, g, S, K):
    x = normal(g, S, K) * torch.exp(normal(g, S, 1, dtype=torch.float32)).to(torch.bfloat16)
    return ep.ep_quantize_fp8(x)


def weights_of(ep, g, E, N, K):
    d = ep.ep_quantize_weight_fp8(normal(g, E, N, K))
    return d["q"], d["scale"]


def close(got, want, bound, what):
    got, want = got.double(), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = ((got - want).abs() - bound).max().item() if got.numel() else -1.0
    assert over <= 0, f"{what}: {over:.3g} over the bound"


def same_e4m3(got, want, what):
    got = got.double()
    bad = (got != want) & ~(torch.isnan(got) & torch.isnan(want))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} values differ"


# ----------------------------------------------------------------- quantisation
@pytest.mark.parametrize("S,H", [(1, 16), (5, 128), (7, 208), (300, 1040), (33, 7168), (5000, 7168)])
def test_quantize_rows(ep, S, H):
    say(f"quantize rows S={S} H={H}")
    g = gen(S * 7 + H)
    x = normal(g, S, H) * torch.exp(4 * normal(g, S, 1, dtype=torch.float32)).to(torch.bfloat16)
    q, scale = ep.ep_quantize_fp8(x)
    torch.cuda.synchronize()
    want, byte = ref.quantize_rows(x)
    assert torch.equal(scale, byte)
    same_e4m3(q, want, "q")


def test_quantize_special_values(ep):
    rows = []
    for v in (0.0, 1.75, 1.7578125, 448.0, 450.0, 3.3895313892515355e38, 2.0 ** -126, 2.0 ** -133,
              2.0 ** -120, float("inf"), -float("inf"), NAN):
        r = torch.linspace(-1, 1, 256).to(torch.bfloat16) * (0 if v == 0 else 1e-3)
        r[3] = v
        rows.append(r)
    rows.append(torch.full((256,), NAN, dtype=torch.bfloat16))
    rows.append(torch.full((256,), 2.0 ** -133, dtype=torch.bfloat16))
    # every tie between two neighbouring e4m3 values, and its neighbours in bf16
    ties = torch.tensor([(8 + i + 0.5) * 2.0 ** e for i in range(8) for e in range(-9, 3)])
    t = torch.cat([ties, ties * (1 + 2 ** -7), ties * (1 - 2 ** -7)]).to(torch.bfloat16)
    rows.append(torch.cat([t[:255], torch.tensor([448.0], dtype=torch.bfloat16)]))
    rows.append(torch.cat([-t[-255:], torch.tensor([448.0], dtype=torch.bfloat16)]))
    x = torch.stack(rows).to(DEV)
    say("quantize special values")
    q, scale = ep.ep_quantize_fp8(x)
    torch.cuda.synchronize()
    want, byte = ref.quantize_rows(x)
    assert torch.equal(scale, byte)
    same_e4m3(q, want, "q")


@pytest.mark.parametrize("T,H,k", [(1, 16, 1), (5, 272, 3), (128, 7168, 8), (4096, 2064, 8)])
def test_dispatch_fp8(ep, T, H, k):
    say(f"dispatch fp8 T={T} H={H} k={k}")
    g = gen(T + H)
    x = normal(g, T, H)
    pos = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32).view(T, k)
    skip = {0: -1, T * k - 1: T * k, T * k // 2: 2 ** 30} if T > 1 else {}
    rows = pos.view(-1).clone()
    for i, v in skip.items():
        pos.view(-1)[i] = v
    send = torch.full((T * k, H), 0x55, dtype=torch.uint8, device=DEV)
    scale = torch.full((T * k, ref.blocks(H)), 0x55, dtype=torch.uint8, device=DEV)
    ep.ep_dispatch_fp8(x, pos, send, scale)
    q, s = ep.ep_quantize_fp8(x)
    torch.cuda.synchronize()
    want = torch.full_like(send, 0x55)
    want_s = torch.full_like(scale, 0x55)
    keep = torch.ones(T * k, dtype=torch.bool, device=DEV)
    keep[list(skip)] = False
    token = torch.arange(T, device=DEV).repeat_interleave(k)
    want[rows[keep].long()] = q.view(torch.uint8)[token[keep]]
    want_s[rows[keep].long()] = s[token[keep]]
    assert torch.equal(send, want) and torch.equal(scale, want_s)


@pytest.mark.parametrize("E,N,K", [(1, 16, 16), (3, 144, 272), (2, 256, 1408), (2, 4096, 720)])
def test_quantize_weight(ep, E, N, K):
    say(f"quantize weight E={E} N={N} K={K}")
    w = normal(gen(N + K), E, N, K)
    w[0, :min(N, 128), :min(K, 128)] = 0
    d = ep.ep_quantize_weight_fp8(w, transposed=True)
    torch.cuda.synchronize()
    want, byte = ref.quantize_weight(w)
    assert torch.equal(d["scale"], byte)
    same_e4m3(d["q"], want, "q")
    assert torch.equal(d["scale_t"], byte.transpose(1, 2))
    assert torch.equal(d["q_t"].view(torch.uint8), d["q"].view(torch.uint8).transpose(1, 2))


# ----------------------------------------------------------------- grouped products
# (rows of each expert, rows before the first and behind the last segment, N, K)
SHAPES = [
    ([1], 0, 0, 16, 16),
    ([0, 1, 0], 0, 0, 208, 144),
    ([3, 0, 17, 1], 2, 5, 128, 128),
    ([0, 0], 4, 0, 64, 64),
    ([16, 33, 0, 40, 7], 0, 1, 4096, 336),
    ([200, 1, 0, 310], 3, 9, 272, 400),
    ([256, 257, 511], 0, 0, 512, 1024),
    ([700, 0, 65, 900, 300], 0, 40, 1040, 2064),
    ([1] * 130, 0, 0, 256, 256),
    ([5] * 70 + [0] * 900 + [90] * 3, 0, 0, 144, 128),
    ([2500], 0, 0, 7168, 256),
    ([3000, 0, 4000, 1, 2999], 0, 7, 2064, 400),
    ([70] * 69 + [0], 0, 3, 1040, 272),
    ([11] * 15 + [100], 0, 0, 2816, 400),
    ([40, 0, 9], 0, 2, 272, 8464),
    ([11] * 15 + [100], 0, 0, 2816, 1664), ([9] * 8, 2, 0, 4096, 2064),     # weights over 64 MB
    ([45] * 18, 0, 1, 2816, 144), ([45] * 18, 0, 0, 2816, 1440), ([4] * 64, 0, 1, 1040, 1040), ([20], 0, 0, 4096, 16640),
    ([70, 20, 60, 0, 50, 90, 49, 61, 60], 1, 0, 4112, 8320),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"E{len(s[0])}S{sum(s[0])}N{s[3]}K{s[4]}")
def test_expert_gemm(ep, shape):
    counts, before, behind, N, K = shape
    E, S = len(counts), sum(counts) + before + behind
    say(f"expert gemm E={E} S={S} N={N} K={K}")
    g = gen(N * 3 + K + S)
    a, a_s = rows_of(ep, g, S, K)
    w, w_s = weights_of(ep, g, E, N, K)
    off = offsets_of(counts, before)
    y = torch.full((S, N), NAN, dtype=torch.bfloat16, device=DEV)
    ep.ep_expert_gemm_fp8(a, a_s, w, w_s, off, y=y)
    torch.cuda.synchronize()
    want, mag = ref.grouped(ref.values(a, a_s), ref.weight_values(w, w_s), off)
    lo, hi = before, S - behind
    assert torch.isnan(y[:lo]).all() and torch.isnan(y[hi:]).all(), "rows outside were written"
    close(y[lo:hi], want[lo:hi], BF16 * want[lo:hi].abs() + ref.sum_bound(K, mag[lo:hi]), "y")
    y2 = ep.ep_expert_gemm_fp8(a, a_s, w, w_s, off)
    assert torch.equal(y2[lo:hi], y[lo:hi]), "a second call gives other bits"


@pytest.mark.parametrize("many", [False, True])
def test_expert_gemm_keeps_nan_to_its_rows(ep, many):
    """NaN rows, NaN weights of another expert and NaN behind the segments reach no other row."""
    g = gen(3)
    counts = [300, 301, 20] if many else [5, 9, 3]
    S, N, K = sum(counts) + 7, 144, 336
    a, a_s = rows_of(ep, g, S, K)
    w, w_s = weights_of(ep, g, 3, N, K)
    off = offsets_of(counts)
    clean = ep.ep_expert_gemm_fp8(a, a_s, w, w_s, off)
    a.view(torch.uint8)[2] = 0x7F
    a.view(torch.uint8)[sum(counts):] = 0x7F
    a_s[sum(counts):] = 255
    w.view(torch.uint8)[2] = 0x7F
    w.view(torch.uint8)[1, 5] = 0xFF
    say(f"expert gemm with NaN many={many}")
    y = ep.ep_expert_gemm_fp8(a, a_s, w, w_s, off)
    torch.cuda.synchronize()
    bad = torch.zeros(S, N, dtype=torch.bool, device=DEV)
    bad[2] = True
    bad[counts[0] + counts[1]:] = True
    bad[counts[0]:counts[0] + counts[1], 5] = True
    n = sum(counts)
    assert torch.isnan(y[:n][bad[:n]]).all()
    assert torch.equal(y[:n][~bad[:n]], clean[:n][~bad[:n]])


def test_expert_gemm_scale_range(ep):
    """Scales far from 1: rows of 1e-30 against weights of 1e+30, block by block."""
    g = gen(11)
    S, N, K = 70, 128, 512
    x = normal(g, S, K)
    x[:, :128] *= 1e-30
    x[:, 128:256] *= 1e30
    w = normal(g, 1, N, K)
    w[:, :, :128] *= 1e30
    w[:, :, 128:256] *= 1e-30
    a, a_s = ep.ep_quantize_fp8(x)
    d = ep.ep_quantize_weight_fp8(w)
    off = offsets_of([S])
    say("expert gemm scale range")
    y = ep.ep_expert_gemm_fp8(a, a_s, d["q"], d["scale"], off)
    torch.cuda.synchronize()
    want, mag = ref.grouped(ref.values(a, a_s), ref.weight_values(d["q"], d["scale"]), off)
    close(y, want, BF16 * want.abs() + ref.sum_bound(K, mag), "y")


@pytest.mark.parametrize("bad", [[0, 50, 20, 60], [-5, 10, 30, 200], [70, 60, 50, 40],
                                 [2 ** 30, -2 ** 30, 2 ** 30, 7]])
def test_expert_offsets_out_of_order(ep, bad):
    """Offsets that decrease or leave the buffer: unspecified rows, nothing written outside."""
    g = gen(13)
    S, N, K, pad = 60, 128, 128, 64
    a, a_s = rows_of(ep, g, S, K)
    w, w_s = weights_of(ep, g, 3, 2 * N, K)
    off = torch.tensor(bad, dtype=torch.int32, device=DEV)
    y = torch.full((S + 2 * pad, 2 * N), 7.0, dtype=torch.bfloat16, device=DEV)
    h = torch.full((S + 2 * pad, N), 0x11, dtype=torch.uint8, device=DEV)
    say(f"expert products with offsets {bad}")
    ep.ep_expert_gemm_fp8(a, a_s, w, w_s, off, y=y[pad:pad + S])
    ep.ep_expert_swiglu_fp8(a, a_s, w, w_s, off, h=h[pad:pad + S])
    dw = ep.ep_expert_wgrad(y[pad:pad + S].clone(), normal(g, S, K), off)
    torch.cuda.synchronize()
    assert dw.shape == (3, 2 * N, K)
    for t, v in ((y, 7.0), (h, 0x11)):
        assert (t[:pad] == v).all() and (t[pad + S:] == v).all()


@pytest.mark.parametrize("save", [False, True])
@pytest.mark.parametrize("counts,before,behind,I,K", [
    ([1], 0, 0, 128, 16), ([0, 3, 20, 0], 1, 2, 256, 208), ([40, 0, 65], 0, 3, 384, 336),
    ([300, 5, 0, 600], 2, 1, 256, 1040), ([1500], 0, 0, 1408, 512),
    ([2000, 0, 1500, 700], 0, 5, 2816, 400), ([70] * 66, 0, 0, 512, 144),
    ([20, 3], 0, 1, 128, 8336), ([90] * 10, 0, 0, 1792, 8208), ([30] * 10, 0, 0, 1792, 2000),
    ([45] * 18, 3, 0, 1792, 208), ([45] * 18, 0, 1, 1792, 2000)])
def test_expert_swiglu(ep, counts, before, behind, I, K, save):
    E, S = len(counts), sum(counts) + before + behind
    say(f"expert swiglu E={E} S={S} I={I} K={K} save={save}")
    g = gen(I + K + S)
    a, a_s = rows_of(ep, g, S, K)
    w, w_s = weights_of(ep, g, E, 2 * I, K)
    off = offsets_of(counts, before)
    h = torch.full((S, I), 0x33, dtype=torch.uint8, device=DEV)
    h_s = torch.full((S, I // 128), 0x33, dtype=torch.uint8, device=DEV)
    _, _, gu = ep.ep_expert_swiglu_fp8(a, a_s, w, w_s, off, h=h, h_scale=h_s, save_gate_up=save)
    torch.cuda.synchronize()
    assert (gu is not None) == save
    lo, hi = before, S - behind
    for t in (h, h_s):
        assert (t[:lo] == 0x33).all() and (t[hi:] == 0x33).all(), "rows outside were written"
    want, mag = ref.grouped(ref.values(a, a_s), ref.weight_values(w, w_s), off)
    want, mag = want[lo:hi], mag[lo:hi]
    if save:
        close(gu[lo:hi], want, BF16 * want.abs() + ref.sum_bound(K, mag), "gate_up")
    hv, err = ref.gated(want, mag, K)
    top = hv.abs().view(hi - lo, -1, 128).amax(-1)
    slack = err.view(hi - lo, -1, 128).amax(-1)
    byte = h_s[lo:hi].int()
    assert (byte >= ref.scale_exponent((top - slack).clamp(min=0)) + 127).logical_or(
        top <= slack).all()
    assert (byte <= ref.scale_exponent(top + slack) + 127).all(), "scale"
    got = ref.values(h.view(torch.float8_e4m3fn), h_s)[lo:hi]
    unit = torch.exp2(h_s[lo:hi].double() - 127).repeat_interleave(128, -1)
    close(got, hv, E4M3 * (hv.abs() + err) + 2.0 ** -10 * unit + err, "h")


# ----------------------------------------------------------------- gradients
@pytest.mark.parametrize("S,I", [(1, 8), (3, 72), (257, 1408), (3000, 2048)])
def test_swiglu_grad(ep, S, I):
    say(f"swiglu grad S={S} I={I}")
    g = gen(S + I)
    dh, gu = normal(g, S, I), normal(g, S, 2 * I) * 3
    gu.view(-1)[:8] = torch.tensor([0.0, -0.0, 80, -80, 1e4, -1e4, 1e-30, -1.28], device=DEV)
    dgu, h = ep.ep_swiglu_grad(dh, gu)
    torch.cuda.synchronize()
    d, gate, up = dh.double(), gu[:, :I].double(), gu[:, I:].double()
    sig = torch.sigmoid(gate)
    silu = gate * sig
    part = sig + silu.abs() * (1 - sig)
    steps = (gate.abs().clamp(max=128) + 16) * 2.0 ** -23      # exp and the operations after it
    tiny = 2.0 ** -126 * (1 + gate.abs())                      # sigmoid below f32's normal range
    want = torch.cat([d * up * (sig + silu * (1 - sig)), d * silu], 1)
    mag = torch.cat([(d * up).abs() * part, (d * silu).abs()], 1)
    low = torch.cat([(d * up).abs() * tiny * (1 + gate.abs()), d.abs() * tiny], 1)
    close(dgu, want, BF16 * want.abs() + 2 * steps.repeat(1, 2) * mag + low + 2.0 ** -133, "grad")
    close(h, silu * up, BF16 * (silu * up).abs() + steps * (silu * up).abs() +
          up.abs() * tiny + 2.0 ** -133, "h")
    # against central differences of silu(g) u in f64: their error is below e^2 |f'''| / 6 plus the
    # f64 rounding 2^-52 |f| / e, |f'''| <= |dh u|, with e = 2^-13 both below 2^-28 (|dh h| + |dh u|)
    e = 2.0 ** -13
    f = lambda a, b: a * torch.sigmoid(a) * b                   # noqa: E731
    num = torch.cat([d * (f(gate + e, up) - f(gate - e, up)) / (2 * e),
                     d * (f(gate, up + e) - f(gate, up - e)) / (2 * e)], 1)
    fd = 2.0 ** -28 * ((d * silu * up).abs() + (d * up).abs() + (d * silu).abs()).repeat(1, 2)
    fd = fd + 2.0 ** -38 * (gate.abs() * up.abs() * d.abs()).repeat(1, 2) + 2.0 ** -38 * (
        d * silu).abs().repeat(1, 2)
    close(dgu, num, BF16 * want.abs() + 2 * steps.repeat(1, 2) * mag + low + fd + 2.0 ** -100, "differences")


@pytest.mark.parametrize("counts,before,behind,N,K", [
    ([1], 0, 0, 8, 8), ([0, 3, 0], 1, 2, 72, 136), ([31, 32, 33, 0, 64], 0, 3, 264, 40),
    ([300, 5, 0, 600], 2, 1, 256, 512), ([1000, 1], 0, 0, 1040, 776), ([2] * 70, 0, 0, 24, 16),
    ([5000], 0, 0, 64, 136), ([1, 4000, 0, 333], 3, 2, 136, 264),
    ([100, 64, 1, 0, 700], 0, 4, 4104, 776), ([0, 3000, 130, 63], 5, 0, 2056, 2312),
    ([300, 64, 1, 0, 900], 0, 4, 4104, 776), ([200, 0, 250, 1000], 2, 3, 2056, 4104)])
def test_expert_wgrad(ep, counts, before, behind, N, K):
    E, S = len(counts), sum(counts) + before + behind
    say(f"expert wgrad E={E} S={S} N={N} K={K}")
    g = gen(N + K + S)
    dy, x = normal(g, S, N), normal(g, S, K)
    dy[:before], x[:before], dy[S - behind:], x[S - behind:] = NAN, NAN, NAN, NAN
    off = offsets_of(counts, before)
    dw = torch.full((E, N, K), NAN, device=DEV)
    ep.ep_expert_wgrad(dy, x, off, grad_w=dw)
    torch.cuda.synchronize()
    want = torch.zeros(E, N, K, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(want)
    for e, lo, hi in ref.segments(off):
        want[e] = dy[lo:hi].double().t() @ x[lo:hi].double()
        mag[e] = dy[lo:hi].double().abs().t() @ x[lo:hi].double().abs()
    bound = torch.stack([ref.sum_bound(n, mag[e]) for e, n in enumerate(counts)])
    close(dw, want, bound + F32 * want.abs(), "dw")
    old = normal(g, E, N, K, dtype=torch.float32)
    acc = old.clone()
    ep.ep_expert_wgrad(dy, x, off, grad_w=acc, accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(acc, old + dw), "accumulate adds the same sums"
    assert torch.equal(ep.ep_expert_wgrad(dy, x, off), dw), "a second call gives other bits"


def test_expert_wgrad_against_differences(ep):
    """d(sum r * (x W^T)) / dW by central differences of the f64 loss at a few places: the loss is
    linear in W, so the quotient is exact up to f64 rounding."""
    g = gen(5)
    counts, N, K = [20, 0, 13], 24, 40
    S = sum(counts)
    dy, x = normal(g, S, N), normal(g, S, K)
    off = offsets_of(counts)
    dw = ep.ep_expert_wgrad(dy, x, off)
    w = normal(g, 3, N, K).double()

    def loss(w):
        return (ref.grouped(x.double(), w, off)[0] * dy.double()).sum()

    for e, n, k in [(0, 0, 0), (0, 23, 39), (1, 5, 7), (2, 11, 20)]:
        d = torch.zeros_like(w)
        d[e, n, k] = 0.5
        diff = loss(w + d) - loss(w - d)
        lo, hi = int(off[e]), int(off[e + 1])
        mag = (dy[lo:hi, n].double() * x[lo:hi, k].double()).abs().sum()
        assert (dw[e, n, k].double() - diff).abs() <= ref.sum_bound(counts[e] + 1, mag) + 1e-9


def test_no_rows(ep):
    """S = 0: empty outputs, and zero weight gradients."""
    e8 = torch.empty((0, 128), dtype=torch.float8_e4m3fn, device=DEV)
    sc = torch.empty((0, 1), dtype=torch.uint8, device=DEV)
    w, w_s = weights_of(ep, gen(1), 2, 256, 128)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    b = torch.empty((0, 128), dtype=torch.bfloat16, device=DEV)
    say("no rows")
    assert ep.ep_quantize_fp8(b)[0].shape == (0, 128)
    assert ep.ep_expert_gemm_fp8(e8, sc, w, w_s, off).shape == (0, 256)
    assert ep.ep_expert_swiglu_fp8(e8, sc, w, w_s, off)[0].shape == (0, 128)
    gu = torch.empty((0, 256), dtype=torch.bfloat16, device=DEV)
    assert ep.ep_swiglu_grad(b, gu)[0].shape == (0, 256)
    dw = torch.full((2, 256, 128), NAN, device=DEV)
    ep.ep_expert_wgrad(gu, b, off, grad_w=dw)
    torch.cuda.synchronize()
    assert (dw == 0).all()


def test_offsets_past_32_bits(ep):
    """2.3e9 values in a buffer: rows on both sides of 2^31 values and bytes, and sums over all."""
    g = gen(21)
    S, K, N = 1_130_000, 2048, 128
    say(f"offsets past 32 bits S={S} K={K}")
    x = torch.empty((S, K), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    q, sc = ep.ep_quantize_fp8(x)
    w, w_s = weights_of(ep, g, 2, N, K)
    cut = 2 ** 31 // K - 5                             # the second segment straddles 2^31 bytes
    off = torch.tensor([0, cut, S], dtype=torch.int32, device=DEV)
    y = ep.ep_expert_gemm_fp8(q, sc, w, w_s, off)
    torch.cuda.synchronize()
    rows = torch.cat([torch.arange(lo, lo + 20) for lo in (0, cut - 10, 2 ** 31 // K - 10, S - 20)])
    rows = rows.to(DEV)
    wantq, byte = ref.quantize_rows(x[rows])
    assert torch.equal(sc[rows], byte)
    same_e4m3(q.view(torch.uint8)[rows].view(torch.float8_e4m3fn), wantq, "q")
    a = ref.values(q.view(torch.uint8)[rows].view(torch.float8_e4m3fn), sc[rows])
    wv = ref.weight_values(w, w_s)[(rows >= cut).long()]
    want, mag = (wv @ a[:, :, None])[..., 0], (wv.abs() @ a.abs()[:, :, None])[..., 0]
    close(y[rows], want, BF16 * want.abs() + ref.sum_bound(K, mag), "y")
    del q, sc

    dw = ep.ep_expert_wgrad(y, x, off)
    torch.cuda.synchronize()
    want = torch.zeros(2, N, K, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(want)
    for e, lo, hi in ref.segments(off):
        for b in range(lo, hi, 1 << 17):
            yy, xx = y[b:min(b + (1 << 17), hi)].double(), x[b:min(b + (1 << 17), hi)].double()
            want[e] += yy.t() @ xx
            mag[e] += yy.abs().t() @ xx.abs()
    close(dw, want, ref.sum_bound(S, mag) + F32 * want.abs(), "dw")

    dh = torch.empty((S, K // 2), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    dgu, h = ep.ep_swiglu_grad(dh, x)                  # x as the saved gate and up values
    some = ep.ep_swiglu_grad(dh[rows].contiguous(), x[rows].contiguous())
    torch.cuda.synchronize()
    assert torch.equal(dgu[rows], some[0]) and torch.equal(h[rows], some[1])


# ----------------------------------------------------------------- few tokens
def moe_case(ep, T, H, I, E, k, fp8, seed=0):
    g = gen(T * 1000 + H + I + seed)
    x = normal(g, T, H)
    idx = torch.rand((T, E), generator=g, device=DEV).argsort(1)[:, :k].to(torch.int32).contiguous()
    w = torch.rand((T, k), generator=g, device=DEV)
    w13 = (normal(g, E, 2 * I, H).float() / H ** 0.5).to(torch.bfloat16)
    w2 = (normal(g, E, H, I).float() / I ** 0.5).to(torch.bfloat16)
    s13 = s2 = None
    if fp8:
        d13, d2 = ep.ep_quantize_weight_fp8(w13), ep.ep_quantize_weight_fp8(w2)
        w13, s13, w2, s2 = d13["q"], d13["scale"], d2["q"], d2["scale"]
    return dict(x=x, topk_idx=idx, topk_w=w, w13=w13, w2=w2, w13_scale=s13, w2_scale=s2)


def moe_ref(c):
    """(out, bound) in f64; see experts_ref for the sums' bound.  h is kept to 2^-16."""
    x, idx, tw = c["x"].double(), c["topk_idx"], c["topk_w"].double()
    T, H = x.shape
    E, k = c["w13"].shape[0], idx.shape[1]
    I = c["w13"].shape[1] // 2
    out, mag, err = (torch.zeros_like(x) for _ in range(3))
    for e in range(E):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if not len(t):
            continue
        w13 = ref.weight_values(c["w13"][e:e + 1],
                                None if c["w13_scale"] is None else c["w13_scale"][e:e + 1])[0]
        w2 = ref.weight_values(c["w2"][e:e + 1],
                               None if c["w2_scale"] is None else c["w2_scale"][e:e + 1])[0]
        h, dh = ref.gated(x[t] @ w13.t(), x[t].abs() @ w13.abs().t(), H)
        s = tw[t, j][:, None]
        h, dh = h * s, (dh + 2.0 ** -15 * h.abs()) * s.abs() + 2.0 ** -120
        out.index_add_(0, t, h @ w2.t())
        mag.index_add_(0, t, h.abs() @ w2.abs().t())
        err.index_add_(0, t, dh @ w2.abs().t())
    return out, BF16 * out.abs() + ref.sum_bound(2 * k * I + 16, mag + err) + err


MOE = [(1, 16, 128, 1, 1, True), (1, 7168, 256, 16, 8, True), (3, 208, 128, 8, 2, True),
       (16, 256, 384, 4, 4, True), (17, 272, 256, 5, 3, True), (33, 1040, 128, 12, 6, True),
       (64, 512, 256, 3, 2, True), (64, 256, 128, 70, 8, True),
       (1, 16, 16, 1, 1, False), (2, 4096, 1408, 9, 8, False), (5, 144, 80, 6, 2, False),
       (2, 8336, 128, 3, 2, True), (2, 256, 8320, 3, 2, True), (1, 8336, 8320, 2, 2, True),
       (48, 144, 128, 1, 1, True), (9, 528, 128, 20, 12, True), (5, 1040, 256, 3, 3, True),
       (8, 4096, 512, 12, 4, True), (40, 4096, 256, 12, 2, False),          # weights over 64 MB
       (64, 4096, 256, 24, 2, True), (40, 144, 80, 1, 1, False), (1, 272, 80, 20, 16, False), (3, 8336, 48, 2, 2, False),
       (31, 336, 48, 4, 3, False), (64, 256, 112, 2, 1, False), (64, 128, 64, 64, 64, False)]


@pytest.mark.parametrize("T,H,I,E,k,fp8", MOE)
def test_moe_tokens(ep, T, H, I, E, k, fp8):
    say(f"moe tokens T={T} H={H} I={I} E={E} k={k} fp8={fp8}")
    c = moe_case(ep, T, H, I, E, k, fp8)
    ws = torch.full((ep.ep_moe_tokens_workspace_bytes(T, k, I),), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full((T, H), NAN, dtype=torch.bfloat16, device=DEV)
    ep.ep_moe_tokens(**c, out=out, workspace=ws)
    torch.cuda.synchronize()
    want, bound = moe_ref(c)
    close(out, want, bound, "out")
    assert torch.equal(ep.ep_moe_tokens(**c), out), "a second call gives other bits"


@pytest.mark.parametrize("fp8", [True, False])
def test_moe_tokens_picks(ep, fp8):
    """Picks outside [0, E), tokens without any, one expert picked twice by a token."""
    c = moe_case(ep, 20, 256, 128, 6, 4, fp8)
    idx = c["topk_idx"]
    idx[0] = -1                                     # a padded token
    idx[1, 0], idx[1, 3] = 6, 2 ** 31 - 1
    idx[2] = 3                                      # the same expert in all four picks
    idx[3, 2] = idx[3, 0]
    idx[19, :3] = -5
    say(f"moe tokens picks fp8={fp8}")
    out = ep.ep_moe_tokens(**c)
    torch.cuda.synchronize()
    want, bound = moe_ref(c)
    close(out, want, bound, "out")
    assert (out[0] == 0).all()
    idx[:] = -1
    out = ep.ep_moe_tokens(**c)
    torch.cuda.synchronize()
    assert (out == 0).all()


@pytest.mark.parametrize("T", [1, 12])
@pytest.mark.parametrize("byte,weight", [(10, 1e34), (246, 1e-30)])
def test_moe_tokens_scale_range(ep, T, byte, weight):
    """The smallest and the largest scale that 8-bit weights are exact for."""
    c = moe_case(ep, T, 256, 128, 3, 2, True)
    c["w2_scale"].fill_(byte)
    c["topk_w"] *= weight
    say(f"moe tokens T={T} scale byte {byte}")
    out = ep.ep_moe_tokens(**c)
    torch.cuda.synchronize()
    want, bound = moe_ref(c)
    close(out, want, bound, "out")


@pytest.mark.parametrize("fp8", [True, False])
def test_moe_one_token_picks(ep, fp8):
    """One token: picks outside [0, E), an expert picked three times, no pick at all."""
    c = moe_case(ep, 1, 272, 128, 6, 6, fp8)
    say(f"moe one token picks fp8={fp8}")
    for picks in ([3, 3, 0, 3, 5, 0], [-1, 6, 2, 2 ** 31 - 1, -2 ** 31, 2], [-1] * 6):
        c["topk_idx"][0] = torch.tensor(picks, dtype=torch.int32, device=DEV)
        out = ep.ep_moe_tokens(**c)
        torch.cuda.synchronize()
        want, bound = moe_ref(c)
        close(out, want, bound, "out")
    assert (out == 0).all()


@pytest.mark.parametrize("fp8", [True, False])
def test_moe_tokens_keeps_nan_to_its_tokens(ep, fp8):
    c = moe_case(ep, 18, 256, 128, 5, 2, fp8)
    clean = ep.ep_moe_tokens(**c)
    bytes_ = c["w2"].view(torch.uint8)
    bytes_[4] = 0xFF if not fp8 else 0x7F           # NaN in every weight of expert 4
    c["x"][7, 3] = float("inf")
    say(f"moe tokens with NaN fp8={fp8}")
    out = ep.ep_moe_tokens(**c)
    torch.cuda.synchronize()
    hit = (c["topk_idx"] == 4).any(1)
    hit[7] = True
    assert torch.isnan(out[hit]).any(1).all()
    assert torch.equal(out[~hit], clean[~hit])


# ----------------------------------------------------------------- together
def layer(ep, x, logits, k, W):
    """One layer as a serving program runs it: route, layout, FP8 dispatch, experts, combine."""
    idx, tw = ep.ep_route_topk(logits, k)
    E = W["w13"].shape[0]
    lay = ep.ep_dispatch_layout(idx, E, 1)
    a, a_s = ep.ep_dispatch_fp8(x, lay["pos"])
    h, h_s, gu = ep.ep_expert_swiglu_fp8(a, a_s, W["w13"], W["w13_scale"], lay["expert_offsets"],
                                         save_gate_up=True)
    y = ep.ep_expert_gemm_fp8(h, h_s, W["w2"], W["w2_scale"], lay["expert_offsets"])
    out = ep.ep_combine(y, lay["pos"], tw)
    return dict(idx=idx, tw=tw, lay=lay, a=a, a_s=a_s, h=h, h_s=h_s, gu=gu, y=y, out=out)


def layer_grad(ep, r, x, grad_out, W):
    """Its backward pass, from saved tensors only."""
    lay = r["lay"]
    off = lay["expert_offsets"]
    gy, gtw = ep.ep_combine_grad(grad_out, r["y"], lay["pos"], r["tw"])
    gyq, gys = ep.ep_quantize_fp8(gy)
    gh = ep.ep_expert_gemm_fp8(gyq, gys, W["w2_t"], W["w2_t_scale"], off)
    ggu, hb = ep.ep_swiglu_grad(gh, r["gu"])
    dw2 = ep.ep_expert_wgrad(gy, hb, off)
    dw13 = ep.ep_expert_wgrad(ggu, ep.ep_dispatch(x, lay["pos"]), off)
    gq, gs = ep.ep_quantize_fp8(ggu)
    gx = ep.ep_dispatch_grad(ep.ep_expert_gemm_fp8(gq, gs, W["w13_t"], W["w13_t_scale"], off),
                             lay["pos"])
    return dict(gy=gy, gh=gh, ggu=ggu, hb=hb, dw2=dw2, dw13=dw13, gx=gx, gtw=gtw)


def layer_weights(ep, g, E, H, I):
    w13 = (normal(g, E, 2 * I, H).float() / H ** 0.5).to(torch.bfloat16)
    w2 = (normal(g, E, H, I).float() / I ** 0.5).to(torch.bfloat16)
    d13 = ep.ep_quantize_weight_fp8(w13, transposed=True)
    d2 = ep.ep_quantize_weight_fp8(w2, transposed=True)
    return dict(w13=d13["q"], w13_scale=d13["scale"], w13_t=d13["q_t"], w13_t_scale=d13["scale_t"],
                w2=d2["q"], w2_scale=d2["scale"], w2_t=d2["q_t"], w2_t_scale=d2["scale_t"])


@pytest.mark.parametrize("T,H,I,E,k", [(3, 128, 128, 4, 2), (100, 272, 256, 8, 3), (900, 512, 384, 4, 2)])
def test_layer_and_its_gradients(ep, T, H, I, E, k):
    """The whole layer, forward and backward: every stage against its definition on the inputs that
    it got, and the result against the layer in f64 on the unquantised input.

    The last bound: quantising puts each a and h off by 2^-4 of its value or 2^-10 of its scale; the
    values' signs are independent, so errors of a sum add as squares.  The bound used is on the 2-norm:
    weights are the same on both sides, a's relative error is at most 2^-4 in the 2-norm (plus the
    2^-10 scale part, < 2^-10 * sqrt(128) / 1.75), hence [g; u] off by at most 0.07 of ||W|| ||a||, and
    a random W passes the 2-norm of a fixed error and of a on alike (up to sampling); silu(g) u then
    doubles it, h adds its own 2^-4: 0.07 * 2.2 + 0.07 = 0.22 of the result's norm, with 0.3 asked."""
    say(f"layer T={T} H={H} I={I} E={E} k={k}")
    g = gen(T + H)
    x, logits = normal(g, T, H), normal(g, T, E, dtype=torch.float32)
    W = layer_weights(ep, g, E, H, I)
    r = layer(ep, x, logits, k, W)
    go = normal(g, T, H)
    b = layer_grad(ep, r, x, go, W)
    torch.cuda.synchronize()
    off, pos = r["lay"]["expert_offsets"], r["lay"]["pos"].long()
    w13, w2 = (ref.weight_values(W[n], W[n + "_scale"]) for n in ("w13", "w2"))
    # stages
    q, s = ref.quantize_rows(x)
    token = torch.empty(T * k, dtype=torch.long, device=DEV)
    token[pos.view(-1)] = torch.arange(T, device=DEV).repeat_interleave(k)
    same_e4m3(r["a"], q[token], "a")
    assert torch.equal(r["a_s"], s[token])
    gu, mag = ref.grouped(ref.values(r["a"], r["a_s"]), w13, off)
    close(r["gu"], gu, BF16 * gu.abs() + ref.sum_bound(H, mag), "gate_up")
    y, mag = ref.grouped(ref.values(r["h"], r["h_s"]), w2, off)
    close(r["y"], y, BF16 * y.abs() + ref.sum_bound(I, mag), "y")
    gyq, gys = ref.quantize_rows(b["gy"])
    gh, mag = ref.grouped(ref.values(gyq, gys), w2.transpose(1, 2), off)
    close(b["gh"], gh, BF16 * gh.abs() + ref.sum_bound(H, mag), "grad h")
    for name, d, v in (("dw2", b["gy"], b["hb"]), ("dw13", b["ggu"], x[token])):
        for e, lo, hi in ref.segments(off):
            want = d[lo:hi].double().t() @ v[lo:hi].double()
            mag = d[lo:hi].double().abs().t() @ v[lo:hi].double().abs()
            close(b[name][e], want, ref.sum_bound(hi - lo, mag) + F32 * want.abs(), name)
    # the whole, against f64 autograd of the unquantised layer
    xd = x.double().requires_grad_()
    w13d, w2d = w13.clone().requires_grad_(), w2.clone().requires_grad_()
    tw = r["tw"].double()
    out = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    for e in range(E):
        t, j = torch.nonzero(r["idx"] == e, as_tuple=True)
        u = xd[t] @ w13d[e].t()
        h = u[:, :I] * torch.sigmoid(u[:, :I]) * u[:, I:]
        out = out.index_add(0, t, (h @ w2d[e].t()) * tw[t, j][:, None])
    out.backward(go.double())
    for name, got, want in (("out", r["out"], out.detach()), ("grad x", b["gx"], xd.grad),
                            ("dw2", b["dw2"], w2d.grad), ("dw13", b["dw13"], w13d.grad)):
        rel = ((got.double() - want).norm() / want.norm()).item()
        say(f"{name}: relative to the unquantised layer {rel:.4f}")
        assert rel < 0.3, (name, rel)


def test_few_token_layer_agrees_with_the_grouped_one(ep):
    """The same tokens through ep_moe_tokens and through dispatch and the grouped products: the first
    keeps activations in bf16, so they differ by the quantisation only (bound as above)."""
    g = gen(21)
    T, H, I, E, k = 40, 512, 256, 8, 3
    x, logits = normal(g, T, H), normal(g, T, E, dtype=torch.float32)
    W = layer_weights(ep, g, E, H, I)
    r = layer(ep, x, logits, k, W)
    out = ep.ep_moe_tokens(x, r["idx"], r["tw"], W["w13"], W["w2"], W["w13_scale"], W["w2_scale"])
    torch.cuda.synchronize()
    rel = ((out.double() - r["out"].double()).norm() / out.double().norm()).item()
    assert rel < 0.3, rel


def test_captured_layer(ep):
    """Forward, backward and the few-token layer in one graph, replayed on new inputs between eager
    work: every replay equals the eager run."""
    g = gen(31)
    T, H, I, E, k = 48, 256, 128, 6, 2
    W = layer_weights(ep, g, E, H, I)
    x, logits, go = normal(g, T, H), normal(g, T, E, dtype=torch.float32), normal(g, T, H)

    def step(x, logits, go):
        r = layer(ep, x, logits, k, W)
        b = layer_grad(ep, r, x, go, W)
        few = ep.ep_moe_tokens(x, r["idx"], r["tw"], W["w13"], W["w2"], W["w13_scale"],
                               W["w2_scale"])
        return [r["out"], b["gx"], b["dw2"], b["dw13"], b["gtw"], few]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(x, logits, go)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    say("capture of the layer")
    with torch.cuda.graph(graph, stream=s):
        got = step(x, logits, go)
    for rep in range(4):
        for t in (x, logits, go):
            t.copy_(torch.randn(t.shape, generator=g, device=DEV))
        say(f"replay {rep}")
        graph.replay()
        torch.cuda.synchronize()
        want = step(x, logits, go)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), rep


def test_two_streams(ep):
    """Calls that overlap on two streams, each with its own workspace: the same bits as alone."""
    c = [moe_case(ep, 24, 512, 256, 8, 4, True, seed=s) for s in (1, 2)]
    want = [ep.ep_moe_tokens(**v) for v in c]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    say("two streams")
    for _ in range(10):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                outs[i].append(ep.ep_moe_tokens(**c[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for o in outs[i]:
            assert torch.equal(o, want[i])


@pytest.mark.parametrize("handle", ["stream", "integer", "null"])
def test_own_workspace_belongs_to_the_calls_stream(ep, handle, monkeypatch):
    """A workspace made inside a call on another stream is not handed out on the current one while
    the call may still run."""
    s = torch.cuda.Stream()
    stream = {"stream": s, "integer": s.cuda_stream, "null": 0}[handle]
    c = moe_case(ep, 24, 512, 256, 8, 4, True)
    want = ep.ep_moe_tokens(**c)
    g = gen(2)
    dy, x, off = normal(g, 4096, 256), normal(g, 4096, 256), offsets_of([4096])
    dw = ep.ep_expert_wgrad(dy, x, off)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    used = []

    def spy(name, at):
        real = getattr(ep.library(), name)

        def call(*args):
            used.append(args[at])
            return real(*args)
        monkeypatch.setattr(ep.library(), name, call)

    spy("ep_moe_tokens", 13)
    spy("ep_expert_wgrad", 9)
    say(f"own workspace on {handle}")
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda.current_stream().synchronize()
        out = ep.ep_moe_tokens(**c, stream=stream)
        n = ep.ep_moe_tokens_workspace_bytes(24, 4, 256)
        mine = torch.empty(n, dtype=torch.uint8, device=DEV)
        dw2 = ep.ep_expert_wgrad(dy, x, off, stream=stream)
        m = ep.ep_expert_wgrad_workspace_bytes(4096, 256, 256, 1)
        mine2 = torch.empty(m, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    assert m > 0 and all(used)
    assert used[0] != mine.data_ptr() and used[1] != mine2.data_ptr()
    assert torch.equal(out, want) and torch.equal(dw2, dw)


def test_timing_events(ep):
    """The one-shot measurement hook brackets an expert operator's kernels."""
    ev = ep.HipEvents()
    a, b = ev.create(), ev.create()
    c = moe_case(ep, 4, 512, 256, 8, 4, True)
    ep.ep_moe_tokens(**c)
    ep.ep_set_timing_events(a, b)
    ep.ep_moe_tokens(**c)
    torch.cuda.synchronize()
    assert 0 < ev.elapsed_ms(a, b) < 1000
    ev.destroy(a)
    ev.destroy(b)
