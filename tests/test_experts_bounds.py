"""The expert operators' error bounds can fail: planted mistakes -- a result of zeros, a lost piece of a
sum, a doubled scale, a lost row -- exceed them at every shape that the GPU tests use them for."""
import pytest
import torch

import experts_bounds as bounds
import experts_ref as ref
import test_gpu_experts as gpu
import test_gpu_experts_bounds as sharp


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape):
    return torch.randn(shape, generator=g).to(torch.bfloat16)


def operands(N, K, rows=8):
    """Quantised rows and one expert's weights, as f64 values and scale bytes."""
    g = gen(N + K)
    q, a_byte = ref.quantize_rows(normal(g, rows, K))
    w, w_byte = ref.quantize_weight(normal(g, 1, N, K))
    return (ref.values(q, a_byte), a_byte, ref.weight_values(w, w_byte)[0], w_byte[0])


def mistakes(a, w):
    """(name, a, w) of every planted mistake: 16 values of k lost at three places, a doubled scale of a
    row's or a weight's block, the rows moved by one."""
    K = a.shape[1]
    for at in sorted({0, K // 32 * 16, K - 16}):
        lost = a.clone()
        lost[:, at:at + 16] = 0
        yield f"lost k {at}", lost, w
    b = (ref.blocks(K) - 1) * 128
    twice = a.clone()
    twice[:, b:b + 128] *= 2
    yield "row scale", twice, w
    twice = w.clone()
    twice[:128, b:b + 128] *= 2
    yield "weight scale", a, twice
    yield "rows moved", a.roll(1, 0), w


PRODUCTS = sorted({(min(s[3], 512), s[4]) for s in gpu.SHAPES + sharp.PRODUCTS})


@pytest.mark.parametrize("N,K", PRODUCTS)
def test_product(N, K):
    a, a_byte, w, w_byte = operands(N, K)
    y, err = bounds.product(a, a_byte, w, w_byte)
    limit = bounds.product_bound(y, err)
    # the unit's own arithmetic stays within: eight at a time, cut to 2^-13 of the largest
    assert ((unit_product(a, w).to(torch.bfloat16).double() - y).abs() <= limit).all()
    assert (y.abs() > limit).double().mean() > 0.9          # zeros
    for name, am, wm in mistakes(a, w):
        assert ((am @ wm.t() - y).abs() > limit).any(), name


def unit_product(a, w):
    """Eight products at a time cut to multiples of 2^(E - 13), E at most the largest product's."""
    K = a.shape[1]
    y = a.new_zeros(a.shape[0], w.shape[0])
    for k in range(0, K, 8):
        p = a[:, None, k:k + 8] * w[None, :, k:k + 8]
        step = torch.exp2(torch.frexp(p.abs().amax(-1, keepdim=True))[1].double() - 1 - 13)
        y = (y + (torch.trunc(p / step) * step).sum(-1)).float().double()
    return y.float()


GATED = sorted({(c[3], c[4]) for c in sharp.GATED})


@pytest.mark.parametrize("I,K", GATED)
def test_gated(I, K):
    I = min(I, 256)
    a, a_byte, w, w_byte = operands(2 * I, K)
    gu, err = bounds.product(a, a_byte, w, w_byte)
    h, herr = bounds.gated(gu, err)
    byte = ref.quantize_rows(h)[1]
    limit = bounds.quantised_bound(h, herr, bounds.row_scales(byte, I))
    # zeros: half of the gates are negative, and far out silu is next to nothing there
    assert (h.abs() > limit).double().mean() > 0.25
    for name, am, wm in mistakes(a, w):
        bad = am @ wm.t()
        hb = bad[:, :I] * torch.sigmoid(bad[:, :I]) * bad[:, I:]
        assert ((hb - h).abs() > limit).any(), name


@pytest.mark.parametrize("n,N,K", sorted({(max(c[0]), c[3], c[4]) for c in sharp.WGRAD if max(c[0])}))
def test_weight_gradient(n, N, K):
    g = gen(n + N + K)
    N, K = min(N, 136), min(K, 136)
    dy, x = normal(g, n, N).double(), normal(g, n, K).double()
    want = dy.t() @ x
    limit = bounds.wgrad_norm(n)
    assert bounds.norm_excess((want.float()).view(1, -1), want.view(1, -1), limit, N * K) <= 0
    for name, s in (("zeros", slice(0, n)), ("a row", slice(n // 2, n // 2 + 1)),
                    ("the last rows", slice(n - (n % 32 or min(n, 32)), n))):
        lost = dy.clone()
        lost[s] = 0
        assert bounds.norm_excess((lost.t() @ x).view(1, -1), want.view(1, -1), limit, N * K) > 0, name


@pytest.mark.parametrize("T,H,I,E,k,fp8", gpu.MOE)
def test_few_tokens(T, H, I, E, k, fp8):
    """A few of the tokens, each with its own k experts; scaled like the weights of moe_case."""
    T = min(T, 3)
    g = gen(T + H + I)
    x, tw = normal(g, T, H).double(), torch.rand((T, k), generator=g).double()
    kinds = (["lost gate k", "lost up k", "lost down k"] + (["gate scale", "up scale", "down scale"] if fp8
                                                            else []) + ["lost pick"])
    want = torch.zeros(T, H, dtype=torch.float64)
    bad = {n: torch.zeros(T, H, dtype=torch.float64) for n in kinds}
    kH, kI = (ref.blocks(H) - 1) * 128, (ref.blocks(I) - 1) * 128
    for t in range(T):
        for j in range(k):
            # f32 rows of weights, the products in f64 (one expert of the largest shape has 2e8 weights)
            w13 = torch.randn((2 * I, H), generator=g).mul_(H ** -0.5)
            w2 = torch.randn((H, I), generator=g).mul_(I ** -0.5)
            xt = x[t].float()
            gu = (w13 @ xt).double()
            part = (w13[:, kH:kH + 128] @ xt[kH:kH + 128]).double()

            def down(v):
                s = v[:I] * torch.sigmoid(v[:I]) * v[I:] * tw[t, j]
                return (w2 @ s.float()).double(), s
            y, h = down(gu)
            want[t] += y
            last = (w2[:, kI:kI + 128] @ h[kI:kI + 128].float()).double()
            for n in kinds:
                # every pick's last block of k is lost; one block's scale of one pick is doubled
                if n == "lost gate k" or n == "lost up k":
                    v = gu.clone()
                    half = slice(0, I) if "gate" in n else slice(I, 2 * I)
                    v[half] -= part[half]
                    bad[n][t] += down(v)[0]
                elif n == "lost down k":
                    bad[n][t] += y - last
                elif n == "lost pick":
                    bad[n][t] += y if j else 0
                elif j:
                    bad[n][t] += y
                elif n == "down scale":
                    b = y.clone()
                    b[:128] += last[:128]
                    bad[n][t] += b
                else:
                    v = gu.clone()
                    half = slice(0, 128) if "gate" in n else slice(I, I + 128)
                    v[half] += part[half]
                    bad[n][t] += down(v)[0]
    assert bounds.norm_excess(want.to(torch.bfloat16), want, bounds.MOE_NORM) <= 0
    assert bounds.norm_excess(torch.zeros_like(want), want, bounds.MOE_NORM) > 0
    for n in kinds:
        assert bounds.norm_excess(bad[n], want, bounds.MOE_NORM) > 0, n
