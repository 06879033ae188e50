"""The bf16 and int8 expert operators at the largest sizes that their documentation allows (2^17 values on an axis,
1024 experts, rows of 2^20 values to quantise), and where an operand passes 2^31 values: on both sides of
that place, against the definitions in 64 bits."""
import pytest
import torch

import experts_bounds as bounds
import product_choice as choice
import products_ref as ref
import test_gpu_products as gpu
from experts_ref import BF16
from gpu_util import DEV, say
from test_gpu_experts import ep, gen, normal, offsets_of  # noqa: F401
from test_gpu_experts_long import around

pytestmark = pytest.mark.gpu
MAX = 1 << 17


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def some(n, k):
    return torch.unique(torch.linspace(0, n - 1, min(n, k)).long()).to(DEV)


def near(got, want, n, what):
    """Within the 2-norm that n bf16 products with independent signs, summed in f32, and one rounding allow:
    a partial sum is in the 2-norm no larger than the whole, so n / 4 + 2 additions are off by that many
    times 2^-23 of it."""
    assert torch.isfinite(got.double()).all(), what
    rel = ((got.double() - want).norm() / want.norm()).item()
    assert rel <= bounds.additions(n) * 2.0 ** -23 + BF16, (what, rel)


def int8_any(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8)


def scales(g, *shape):
    return torch.rand(shape, generator=g, device=DEV) * 0.1 + 0.01


def bf16_any(g, *shape):
    """Normal values, made piece by piece."""
    t = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    flat = t.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        flat[i:i + (1 << 28)].normal_(generator=g)
    return t


# (rows of each expert, columns, K)
SHAPES = [([5], 16, MAX), ([3, 0, 300], MAX, 16), ([2000], 4096, MAX), ([700], MAX, 144), ([1] * 1024, 128, 1040),
          ([1] * 1000 + [200] * 24, 16, 16)]


def ids(v):
    return f"E{len(v)}" if isinstance(v, list) else str(v)


@pytest.mark.parametrize("kind", ["plain", "transposed", "gated"])
@pytest.mark.parametrize("counts,N,K", SHAPES, ids=ids)
def test_bf16(ep, counts, N, K, kind):  # noqa: F811
    E, S = len(counts), sum(counts)
    say(f"bf16 {kind} E={E} S={S} N={N} K={K} on {choice.product(counts, N, K, 2, kind)}")
    g = gen(N + K)
    a = bf16_any(g, S, K)
    w = bf16_any(g, *((E, K, N) if kind == "transposed" else (E, 2 * N if kind == "gated" else N, K)))
    if kind == "gated":
        w *= K ** -0.5
    off = offsets_of(counts)
    if kind == "gated":
        y, gate_up = ep.ep_expert_swiglu_bf16(a, w, off, save_gate_up=True)
    else:
        y = ep.ep_expert_gemm_bf16(a, w, off, transposed=kind == "transposed")
    torch.cuda.synchronize()
    seg = ref.segments(off)
    for e, lo, hi in [seg[i] for i in sorted({0, len(seg) // 2, len(seg) - 1})]:
        r, n = lo + some(hi - lo, 6), some(N, 40)
        if kind == "gated":
            both = torch.cat([n, N + n])
            gu = a[r].double() @ w[e][both].double().t()
            near(gate_up[r][:, both], gu, K, f"gate_up of expert {e}")
            # h from what was saved: silu's slope and the product pass 2^-8 of each on, at most 2.2 times
            h = gu[:, :len(n)] * torch.sigmoid(gu[:, :len(n)]) * gu[:, len(n):]
            rel = ((y[r][:, n].double() - h).norm() / h.norm()).item()
            assert rel <= 2.2 * bounds.additions(K) * 2.0 ** -23 + BF16, (e, rel)
        else:
            wn = w[e][:, n].t() if kind == "transposed" else w[e][n]
            near(y[r][:, n], a[r].double() @ wn.double().t(), K, f"expert {e}")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts,N,K", SHAPES, ids=ids)
def test_int8(ep, counts, N, K, gated):  # noqa: F811
    K = min(K, MAX - 16)
    E, S = len(counts), sum(counts)
    say(f"int8 gated={gated} E={E} S={S} N={N} K={K} on {choice.product(counts, N, K, 1, 'gated' if gated else 'plain')}")
    g = gen(N + K + 1)
    rows = 2 * N if gated else N
    a, w = int8_any(g, S, K), int8_any(g, E, rows, K)
    a_s, w_s = scales(g, S), scales(g, E, rows) * (K ** -0.5 / 50)
    off = offsets_of(counts)
    if gated:
        h, h_s = ep.ep_expert_swiglu_int8(a, a_s, w, w_s, off)
    else:
        y = ep.ep_expert_gemm_int8(a, a_s, w, w_s, off)
    torch.cuda.synchronize()
    seg = ref.segments(off)
    for e, lo, hi in [seg[i] for i in sorted({0, len(seg) // 2, len(seg) - 1})]:
        r = lo + some(hi - lo, 6)
        if gated:
            gu, err = ref.product_int8(a[r], a_s[r], w[e], w_s[e])
            ref.check_quantised(h[r], h_s[r], *ref.gated(gu, err), f"expert {e}")
        else:
            n = some(N, 40)
            want, err = ref.product_int8(a[r], a_s[r], w[e][n], w_s[e][n])
            ref.check(y[r][:, n], want, ref.rounded(want, err), f"expert {e}")


@pytest.mark.parametrize("S,H", [(2100, 1 << 20), (300_000, 7168), (1_100_000, 2000)])
def test_quantise(ep, S, H):  # noqa: F811
    say(f"quantise int8 past 2^31: S={S} H={H}")
    x = bf16_any(gen(S), S, H)
    q, s = ep.ep_quantize_int8(x)
    torch.cuda.synchronize()
    r = around([0, 2 ** 31 // H, 2 ** 30 // H, S], S, 20)
    ref.check_rows(q[r], s[r], x[r])


def test_dispatch(ep):  # noqa: F811
    T, H, k = 40_000, 7168, 8
    say("dispatch int8 past 2^31")
    g = gen(4)
    x = bf16_any(g, T, H)
    pos = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32).view(T, k)
    send, s = ep.ep_dispatch_int8(x, pos)
    torch.cuda.synchronize()
    r = around([0, 2 ** 31 // H, T * k], T * k, 50)
    token = torch.empty(T * k, dtype=torch.long, device=DEV)
    token[pos.view(-1).long()] = torch.arange(T, device=DEV).repeat_interleave(k)
    ref.check_rows(send[r], s[r], x[token[r]])


# (S, columns, K, E): rows of a, rows of y and weights past 2^31 values, on tiles large and small
LONG = [(1_060_000, 512, 2064, 3), (530_000, 4112, 272, 3), (40_000, 16, 55_056, 1024), (100_000, 22_032, 16, 1024),
        (300, 4096, 4112, 150), (5, 2064, 7168, 160)]


def long_case(S, N, K, E):
    off = torch.linspace(0, S, E + 1).long()
    for p in (2 ** 31 // K - 3, 2 ** 31 // N + 5):       # a segment that starts at a place of its own
        e = int((off - p).abs()[1:-1].argmin()) + 1
        if off[e - 1] < p < off[e + 1]:
            off[e] = p
    at = [0, S, 2 ** 31 // K, 2 ** 31 // N, 2 ** 32 // N, *off[1:-1][:: max(1, E // 4)].tolist()]
    at += [int(off[min(E - 1, 2 ** 31 // (N * K) + d)]) for d in (0, 1)] + [int(off[E - 1])]
    rows = around(at, S, 6)
    return off.to(torch.int32).to(DEV), rows, torch.searchsorted(off.to(DEV), rows, right=True) - 1


@pytest.mark.parametrize("kind", ["plain", "transposed", "gated"])
@pytest.mark.parametrize("S,N,K,E", LONG)
def test_bf16_long(ep, S, N, K, E, kind):  # noqa: F811
    assert max(S * K, S * N, E * N * K) > 2 ** 31
    say(f"bf16 {kind} past 2^31: S={S} N={N} K={K} E={E}")
    g = gen(S + N)
    if kind == "gated":
        N //= 2
    a = bf16_any(g, S, K)
    w = bf16_any(g, *((E, K, N) if kind == "transposed" else (E, 2 * N if kind == "gated" else N, K)))
    off, rows, experts = long_case(S, N, K, E)
    if kind == "gated":
        w *= K ** -0.5
        h, y = ep.ep_expert_swiglu_bf16(a, w, off, save_gate_up=True)
    else:
        y = ep.ep_expert_gemm_bf16(a, w, off, transposed=kind == "transposed")
    torch.cuda.synchronize()
    for e in torch.unique(experts).tolist():
        r = rows[experts == e]
        want, err = ref.product_bf16(a[r], w[e].t() if kind == "transposed" else w[e])
        ref.check(y[r], want, ref.rounded(want, err), f"expert {e}")
        if kind == "gated":
            want, err = ref.gated(want, err)
            ref.check(h[r], want, ref.rounded(want, err), f"h of expert {e}")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("S,N,K,E", LONG)
def test_int8_long(ep, S, N, K, E, gated):  # noqa: F811
    say(f"int8 past 2^31: S={S} N={N} K={K} E={E} gated={gated}")
    g = gen(S + N + 1)
    if gated:
        N = max(16, N // 32 * 16)
    channels = 2 * N if gated else N
    a, w = int8_any(g, S, K), int8_any(g, E, channels, K)
    a_s, w_s = scales(g, S), scales(g, E, channels) * (K ** -0.5 / 50)
    off, rows, experts = long_case(S, N, K, E)
    if gated:
        h, h_s = ep.ep_expert_swiglu_int8(a, a_s, w, w_s, off)
    else:
        y = ep.ep_expert_gemm_int8(a, a_s, w, w_s, off)
    torch.cuda.synchronize()
    for e in torch.unique(experts).tolist():
        r = rows[experts == e]
        want, err = ref.product_int8(a[r], a_s[r], w[e], w_s[e])
        if gated:
            ref.check_quantised(h[r], h_s[r], *ref.gated(want, err), f"h of expert {e}")
        else:
            ref.check(y[r], want, ref.rounded(want, err), f"expert {e}")
