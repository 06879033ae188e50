"""The expert operators in bf16 and in 8-bit integers against their definitions in 64 bits (products_ref.py,
where the bounds are derived), each at the sizes, segments and values where it can go wrong, and together
as a model's layer uses them."""
import pytest
import torch

import products_ref as ref
from gpu_util import DEV, say
from test_gpu_experts import ep, gen, normal, offsets_of  # noqa: F401

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def tokens(g, S, K):
    return normal(g, S, K) * torch.exp(normal(g, S, 1, dtype=torch.float32)).to(torch.bfloat16)


def matrices(g, E, N, K):
    w = torch.empty(E, N, K, dtype=torch.bfloat16, device=DEV)
    for e in range(E):
        w[e] = normal(g, N, K)
    return w


def int8_rows(x):
    q, s = ref.integers(x)
    return q.to(torch.int8), s.float()


def int8_matrices(g, E, N, K):
    q = torch.empty(E, N, K, dtype=torch.int8, device=DEV)
    s = torch.empty(E, N, dtype=torch.float32, device=DEV)
    for e in range(E):
        q[e], s[e] = int8_rows(normal(g, N, K))
    return q, s


# ----------------------------------------------------------------- rows to integers
@pytest.mark.parametrize("S,H", [(1, 16), (5, 128), (7, 208), (300, 1040), (33, 2048), (33, 2064), (33, 7168),
                                 (9, 8192), (9, 8208), (5000, 7168), (2, 1 << 20)])
def test_quantize_rows(ep, S, H):  # noqa: F811
    say(f"quantize int8 rows S={S} H={H}")
    g = gen(S * 7 + H)
    x = normal(g, S, H) * torch.exp(4 * normal(g, S, 1, dtype=torch.float32)).to(torch.bfloat16)
    q, scale = ep.ep_quantize_int8(x)
    torch.cuda.synchronize()
    ref.check_rows(q, scale, x)


def test_quantize_weights(ep):  # noqa: F811
    g = gen(2)
    w = matrices(g, 3, 80, 272)
    say("quantize int8 weights")
    q, scale = ep.ep_quantize_int8(w)
    torch.cuda.synchronize()
    assert q.shape == w.shape and scale.shape == w.shape[:2]
    ref.check_rows(q, scale, w)


@pytest.mark.parametrize("H", [256, 4096, 8208])
def test_quantize_special_values(ep, H):  # noqa: F811
    """Zeros, the least and the largest magnitudes, infinities and NaN at every place of a row, and
    every quotient of two bf16 mantissas: each tie among them."""
    rows = []
    for v in (0.0, 1.0, -1.0, 254.0, 3.3895313892515355e38, 2.0 ** -126, 2.0 ** -133, 1.9921875 * 2.0 ** -120,
              2.0 ** -119, INF, -INF, NAN):
        for at in (0, 5, H // 2 + 3, H - 1):
            r = torch.linspace(-1, 1, H).to(torch.bfloat16) * (0 if v == 0 else min(abs(v), 1e-3))
            r[at] = v
            rows.append(r)
    rows.append(torch.full((H,), NAN, dtype=torch.bfloat16))
    rows.append(torch.full((H,), 2.0 ** -133, dtype=torch.bfloat16))
    rows.append(torch.zeros(H, dtype=torch.bfloat16))
    mant = torch.arange(128, 256).float()
    for top in range(128, 256):
        v = torch.cat([mant * 2.0 ** -e for e in range(1, 9)])[:H - 1]
        v = torch.where(v <= top, v, v / 2)
        rows.append(torch.cat([v * (1 if top % 2 else -1), torch.zeros(H - 1 - v.numel()),
                               torch.tensor([float(top)])]).to(torch.bfloat16))
    x = torch.stack(rows).to(DEV)
    say(f"quantize int8 special values H={H}")
    q, scale = ep.ep_quantize_int8(x)
    torch.cuda.synchronize()
    ref.check_rows(q, scale, x)


@pytest.mark.parametrize("T,H,k", [(1, 16, 1), (5, 272, 3), (128, 7168, 8), (4096, 2064, 8), (3, 8208, 64)])
def test_dispatch(ep, T, H, k):  # noqa: F811
    say(f"dispatch int8 T={T} H={H} k={k}")
    g = gen(T + H)
    x = tokens(g, T, H)
    pos = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32).view(T, k)
    skip = {0: -1, T * k - 1: T * k, T * k // 2: 2 ** 30} if T > 1 else {}
    rows = pos.view(-1).clone()
    for i, v in skip.items():
        pos.view(-1)[i] = v
    send = torch.full((T * k, H), 0x55, dtype=torch.int8, device=DEV)
    scale = torch.full((T * k,), 7.0, device=DEV)
    ep.ep_dispatch_int8(x, pos, send, scale)
    q, s = ep.ep_quantize_int8(x)
    torch.cuda.synchronize()
    ref.check_rows(q, s, x)
    want, want_s = torch.full_like(send, 0x55), torch.full_like(scale, 7.0)
    keep = torch.ones(T * k, dtype=torch.bool, device=DEV)
    keep[list(skip)] = False
    token = torch.arange(T, device=DEV).repeat_interleave(k)
    want[rows[keep].long()] = q[token[keep]]
    want_s[rows[keep].long()] = s[token[keep]]
    assert torch.equal(send, want) and torch.equal(scale, want_s)


# ----------------------------------------------------------------- products
# (rows of each expert, rows before the first and behind the last segment, N, K): multiples of 8; the int8
# forms take those of 16
SHAPES = [
    ([1], 0, 0, 8, 8), ([1], 0, 0, 16, 16), ([0, 1, 0], 0, 0, 208, 144), ([3, 0, 17, 1], 2, 5, 128, 128),
    ([0, 0], 4, 0, 64, 64), ([5, 9, 3], 0, 0, 72, 1000), ([63, 64, 65, 1], 1, 0, 264, 200),
    ([40, 7, 0, 90], 3, 2, 1040, 400), ([129, 31, 257], 0, 3, 520, 712), ([1] * 8 + [0] * 8, 0, 1, 4096, 1040),
    ([0] * 30 + [1, 0, 2, 5] + [0] * 30, 0, 0, 2048, 2064), ([4] * 64, 7, 0, 1040, 336),
    ([2] * 100, 0, 0, 144, 80), ([11] * 15 + [100], 0, 2, 2816, 400), ([300] * 70, 0, 0, 272, 400),
    ([70] * 40, 0, 0, 1040, 272), ([500, 0, 300], 2, 2, 2048, 7168), ([257, 256, 255, 1, 900], 1, 0, 7168, 2064),
    ([3000, 0, 4000, 1, 2999], 0, 7, 2064, 400), ([1100, 3, 800], 0, 5, 4112, 8336),
    ([2500, 0, 700], 3, 1, 4096, 16),
]


def ids(s):
    return f"E{len(s[0])}S{sum(s[0])}N{s[3]}K{s[4]}"


def wide(shapes):
    return [s for s in shapes if s[3] % 16 == 0 and s[4] % 16 == 0]


def untouched(t, before, behind, value):
    n = t.shape[0]
    assert (t[:before] == value).all() and (t[n - behind:] == value).all()


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_gemm_bf16(ep, shape, transposed):  # noqa: F811
    counts, before, behind, N, K = shape
    E, S = len(counts), sum(counts) + before + behind
    say(f"bf16 product E={E} S={S} N={N} K={K} transposed={transposed}")
    g = gen(N * 5 + K + S)
    a = tokens(g, S, K)
    w = matrices(g, E, K, N) if transposed else matrices(g, E, N, K)
    off = offsets_of(counts, before)
    y = torch.full((S, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ep.ep_expert_gemm_bf16(a, w, off, transposed=transposed, y=y)
    torch.cuda.synchronize()
    untouched(y, before, behind, 7.0)
    for e, lo, hi in ref.segments(off):
        want, err = ref.product_bf16(a[lo:hi], w[e].t() if transposed else w[e])
        ref.check(y[lo:hi], want, ref.rounded(want, err), f"expert {e}")


@pytest.mark.parametrize("save", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_swiglu_bf16(ep, shape, save):  # noqa: F811
    counts, before, behind, I, K = shape
    E, S = len(counts), sum(counts) + before + behind
    say(f"bf16 gated E={E} S={S} I={I} K={K} save={save}")
    g = gen(I * 3 + K + S)
    a, w = tokens(g, S, K), matrices(g, E, 2 * I, K) * K ** -0.5
    off = offsets_of(counts, before)
    h = torch.full((S, I), 7.0, dtype=torch.bfloat16, device=DEV)
    gate_up = torch.full((S, 2 * I), 7.0, dtype=torch.bfloat16, device=DEV) if save else None
    ep.ep_expert_swiglu_bf16(a, w, off, h=h, gate_up=gate_up)
    torch.cuda.synchronize()
    untouched(h, before, behind, 7.0)
    if save:
        untouched(gate_up, before, behind, 7.0)
    for e, lo, hi in ref.segments(off):
        gu, err = ref.product_bf16(a[lo:hi], w[e])
        want, herr = ref.gated(gu, err)
        ref.check(h[lo:hi], want, ref.rounded(want, herr), f"h of expert {e}")
        if save:
            ref.check(gate_up[lo:hi], gu, ref.rounded(gu, err), f"gate_up of expert {e}")


@pytest.mark.parametrize("shape", wide(SHAPES), ids=ids)
def test_gemm_int8(ep, shape):  # noqa: F811
    counts, before, behind, N, K = shape
    E, S = len(counts), sum(counts) + before + behind
    say(f"int8 product E={E} S={S} N={N} K={K}")
    g = gen(N * 5 + K + S)
    a, a_s = int8_rows(tokens(g, S, K))
    w, w_s = int8_matrices(g, E, N, K)
    off = offsets_of(counts, before)
    y = torch.full((S, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ep.ep_expert_gemm_int8(a, a_s, w, w_s, off, y=y)
    torch.cuda.synchronize()
    untouched(y, before, behind, 7.0)
    for e, lo, hi in ref.segments(off):
        want, err = ref.product_int8(a[lo:hi], a_s[lo:hi], w[e], w_s[e])
        ref.check(y[lo:hi], want, ref.rounded(want, err), f"expert {e}")


@pytest.mark.parametrize("shape", wide(SHAPES), ids=ids)
def test_swiglu_int8(ep, shape):  # noqa: F811
    counts, before, behind, I, K = shape
    E, S = len(counts), sum(counts) + before + behind
    say(f"int8 gated E={E} S={S} I={I} K={K}")
    g = gen(I * 3 + K + S)
    a, a_s = int8_rows(tokens(g, S, K))
    w, w_s = int8_matrices(g, E, 2 * I, K)
    w_s *= K ** -0.5
    off = offsets_of(counts, before)
    h = torch.full((S, I), 0x55, dtype=torch.int8, device=DEV)
    h_s = torch.full((S,), 7.0, device=DEV)
    ep.ep_expert_swiglu_int8(a, a_s, w, w_s, off, h=h, h_scale=h_s)
    torch.cuda.synchronize()
    untouched(h, before, behind, 0x55)
    untouched(h_s, before, behind, 7.0)
    for e, lo, hi in ref.segments(off):
        gu, err = ref.product_int8(a[lo:hi], a_s[lo:hi], w[e], w_s[e])
        ref.check_quantised(h[lo:hi], h_s[lo:hi], *ref.gated(gu, err), f"expert {e}")


def test_int8_extremes(ep):  # noqa: F811
    """Every product 127 * 127 or 128 * 128 of one sign at the longest K: the integer sum does not wrap; and
    scales whose product with each other is subnormal while the results are not."""
    K = (1 << 17) - 16
    a_s = torch.tensor([2.0 ** -126, 1.0, 2.0 ** 60], device=DEV)
    w_s = torch.full((1, 32), 2.0 ** -4, device=DEV)
    w_s[0, :2] = torch.tensor([2.0 ** 20, 2.0 ** -20])
    off = offsets_of([3])
    for v, x in ((127, 127), (-127, 127), (-128, -128), (127, -128)):
        say(f"int8 extremes {v} {x}")
        a = torch.full((3, K), v, dtype=torch.int8, device=DEV)
        w = torch.full((1, 32, K), x, dtype=torch.int8, device=DEV)
        y = ep.ep_expert_gemm_int8(a, a_s, w, w_s, off)
        torch.cuda.synchronize()
        want = float(v * x * K) * torch.outer(a_s.double(), w_s[0].double())
        ref.check(y, want, ref.rounded(want, 4 * 2.0 ** -24 * want.abs()), f"{v} {x}")


def test_no_rows(ep):  # noqa: F811
    off = offsets_of([0, 0])
    e = lambda *s, d=torch.bfloat16: torch.empty(s, dtype=d, device=DEV)  # noqa: E731
    say("no rows")
    assert ep.ep_expert_gemm_bf16(e(0, 64), e(2, 32, 64), off).shape == (0, 32)
    assert ep.ep_expert_gemm_bf16(e(0, 64), e(2, 64, 32), off, transposed=True).shape == (0, 32)
    h, gu = ep.ep_expert_swiglu_bf16(e(0, 64), e(2, 32, 64), off, save_gate_up=True)
    assert h.shape == (0, 16) and gu.shape == (0, 32)
    q, s = ep.ep_quantize_int8(e(0, 64))
    assert q.shape == (0, 64) and s.shape == (0,)
    i8, f = torch.int8, torch.float32
    w, ws = e(2, 32, 64, d=i8), e(2, 32, d=f)
    assert ep.ep_expert_gemm_int8(q, s, w, ws, off).shape == (0, 32)
    h, hs = ep.ep_expert_swiglu_int8(q, s, w, ws, off)
    assert h.shape == (0, 16) and hs.shape == (0,)
    torch.cuda.synchronize()


# ----------------------------------------------------------------- together
def layer(ep, x, logits, k, w13, w2):  # noqa: F811
    """One layer as a training program runs it: route, layout, dispatch, experts, combine."""
    idx, tw = ep.ep_route_topk(logits, k)
    lay = ep.ep_dispatch_layout(idx, w13.shape[0], 1)
    off = lay["expert_offsets"]
    a = ep.ep_dispatch(x, lay["pos"])
    h, gu = ep.ep_expert_swiglu_bf16(a, w13, off, save_gate_up=True)
    y = ep.ep_expert_gemm_bf16(h, w2, off)
    return dict(idx=idx, tw=tw, lay=lay, a=a, h=h, gu=gu, y=y, out=ep.ep_combine(y, lay["pos"], tw))


def layer_grad(ep, r, grad_out, w13, w2):  # noqa: F811
    """Its backward pass, from saved tensors and the forward weights."""
    pos, off = r["lay"]["pos"], r["lay"]["expert_offsets"]
    gy, gtw = ep.ep_combine_grad(grad_out, r["y"], pos, r["tw"])
    gh = ep.ep_expert_gemm_bf16(gy, w2, off, transposed=True)
    ggu, h = ep.ep_swiglu_grad(gh, r["gu"])
    ga = ep.ep_expert_gemm_bf16(ggu, w13, off, transposed=True)
    return dict(gtw=gtw, gh=gh, ga=ga, dw2=ep.ep_expert_wgrad(gy, h, off),
                dw13=ep.ep_expert_wgrad(ggu, r["a"], off), gx=ep.ep_dispatch_grad(ga, pos))


def layer_int8(ep, x, logits, k, W13, W2):  # noqa: F811
    """One layer as a serving program runs it in 8 bits."""
    idx, tw = ep.ep_route_topk(logits, k)
    lay = ep.ep_dispatch_layout(idx, W13[0].shape[0], 1)
    off = lay["expert_offsets"]
    a, a_s = ep.ep_dispatch_int8(x, lay["pos"])
    h, h_s = ep.ep_expert_swiglu_int8(a, a_s, *W13, off)
    y = ep.ep_expert_gemm_int8(h, h_s, *W2, off)
    return ep.ep_combine(y, lay["pos"], tw)


def layer64(x, idx, tw, w13, w2):
    out = torch.zeros_like(x)
    I = w2.shape[2]
    for e in range(w13.shape[0]):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        gu = x[t] @ w13[e].t()
        h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        out = out.index_add(0, t, (h @ w2[e].t()) * tw[t, j][:, None])
    return out


def layer_inputs(g, T, H, I, E):
    return (normal(g, T, H), normal(g, T, E, dtype=torch.float32),
            (matrices(g, E, 2 * I, H).float() / H ** 0.5).to(torch.bfloat16),
            (matrices(g, E, H, I).float() / I ** 0.5).to(torch.bfloat16))


@pytest.mark.parametrize("T,H,I,E,k", [(1, 64, 8, 3, 2), (3, 128, 128, 4, 2), (100, 264, 248, 8, 3),
                                       (900, 512, 384, 4, 2)])
def test_layer_and_its_gradients(ep, T, H, I, E, k):  # noqa: F811
    """The layer, forward and backward, against f64 autograd.  The bound: bf16 roundings of relative size
    2^-8 at most, each of independent sign, on the way to an output at most six of them in a row (y, gy,
    gate_up and its gradient, h, the result), each passed on by random weights in the 2-norm as the value
    itself, silu(g) u and its gradients at most doubling what g and u are off by: 12 * 2^-8 of the
    2-norm."""
    say(f"bf16 layer T={T} H={H} I={I} E={E} k={k}")
    g = gen(T + H)
    x, logits, w13, w2 = layer_inputs(g, T, H, I, E)
    r = layer(ep, x, logits, k, w13, w2)
    go = normal(g, T, H)
    b = layer_grad(ep, r, go, w13, w2)
    torch.cuda.synchronize()
    v = [t.double().requires_grad_() for t in (x, w13, w2)]
    out = layer64(v[0], r["idx"], r["tw"].double(), v[1], v[2])
    out.backward(go.double())
    for name, got, want in (("out", r["out"], out.detach()), ("grad x", b["gx"], v[0].grad),
                            ("dw13", b["dw13"], v[1].grad), ("dw2", b["dw2"], v[2].grad)):
        rel = ((got.double() - want).norm() / want.norm()).item()
        say(f"{name}: {rel:.5f}")
        assert rel < 12 * 2.0 ** -8, (name, rel)


def test_input_gradient_against_differences(ep):  # noqa: F811
    """y moves along a direction d of its input as the transposed product says: the two sides of
    <W a, gy> = <a, W^T gy> for every row, and a difference of two products.  Both in f64 from bf16 results,
    2^-8 of the sum of magnitudes off at most each."""
    g = gen(9)
    counts, N, K = [33, 0, 70, 1], 264, 136
    S, off = sum(counts), offsets_of(counts)
    a, d, gy = normal(g, S, K), normal(g, S, K), normal(g, S, N)
    w = matrices(g, 4, N, K)
    say("input gradient against differences")
    step = (a.float() + d.float()).to(torch.bfloat16)        # a + d, rounded: the direction is what it got
    y0, y1 = ep.ep_expert_gemm_bf16(a, w, off), ep.ep_expert_gemm_bf16(step, w, off)
    ga = ep.ep_expert_gemm_bf16(gy, w, off, transposed=True)
    torch.cuda.synchronize()
    moved = ((y1.double() - y0.double()) * gy.double()).sum(1)
    said = (ga.double() * (step.double() - a.double())).sum(1)
    mag = ((y1.double().abs() + y0.double().abs()) * gy.double().abs()).sum(1)
    mag += (ga.double() * (step.double() - a.double())).abs().sum(1)
    assert ((moved - said).abs() <= 1.05 * 2.0 ** -8 * mag).all()
    assert ((moved - said.roll(1)).abs() > 1.05 * 2.0 ** -8 * mag).double().mean() > 0.5


@pytest.mark.parametrize("T,H,I,E,k", [(1, 64, 16, 3, 2), (5, 128, 128, 4, 2), (200, 528, 400, 8, 3)])
def test_int8_layer(ep, T, H, I, E, k):  # noqa: F811
    """The 8-bit layer against the layer in f64 on the same quantised weights.  A row's integers are half a
    step off at most: 1 / 254 of the row's largest magnitude, which is at most 5 times the root mean
    square of normal values (and of a product of two, 12 times): independent signs, so relative
    2-norms of 5 / 254 / sqrt(3) = 0.012 for a, passed on to [g; u] and doubled by silu(g) u, and 0.028
    of h's own: 0.052, and bf16's roundings below 0.01."""
    say(f"int8 layer T={T} H={H} I={I} E={E} k={k}")
    g = gen(T + H + 1)
    x, logits, w13, w2 = layer_inputs(g, T, H, I, E)
    W13, W2 = ep.ep_quantize_int8(w13), ep.ep_quantize_int8(w2)
    out = layer_int8(ep, x, logits, k, W13, W2)
    idx, tw = ep.ep_route_topk(logits, k)
    torch.cuda.synchronize()
    values = [q.double() * s.double()[..., None] for q, s in (W13, W2)]
    want = layer64(x.double(), idx, tw.double(), *values)
    rel = ((out.double() - want).norm() / want.norm()).item()
    say(f"relative {rel:.5f}")
    assert rel < 0.07, rel


def test_captured_layers(ep):  # noqa: F811
    """Forward and backward in bf16 and the 8-bit layer in one graph, replayed on new inputs between eager
    work: every replay equals the eager run."""
    g = gen(31)
    T, H, I, E, k = 48, 256, 128, 6, 2
    x, logits, w13, w2 = layer_inputs(g, T, H, I, E)
    W13, W2 = ep.ep_quantize_int8(w13), ep.ep_quantize_int8(w2)
    go = normal(g, T, H)

    def step():
        r = layer(ep, x, logits, k, w13, w2)
        b = layer_grad(ep, r, go, w13, w2)
        return [r["out"], b["gx"], b["dw2"], b["dw13"], b["gtw"], layer_int8(ep, x, logits, k, W13, W2)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    say("capture of the layers")
    with torch.cuda.graph(graph, stream=s):
        got = step()
    for rep in range(4):
        for t in (x, logits, go):
            t.copy_(torch.randn(t.shape, generator=g, device=DEV))
        say(f"replay {rep}")
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), rep
