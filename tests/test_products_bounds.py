"""The error bounds of the bf16 and int8 products can fail: planted mistakes -- zeros, a lost piece of a sum, a
row's or a channel's scale that is lost, rows moved by one -- exceed them, on the CPU, at every length that
the GPU tests use; and the quantiser's definition at the values where it can go wrong."""
import pytest
import torch

import products_ref as ref

LENGTHS = [8, 16, 72, 144, 400, 1040, 2064, 4096, 7168, 8336]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape):
    return torch.randn(shape, generator=g).to(torch.bfloat16)


def lost(a):
    """(name, a) with eight values of k lost, and moved rows."""
    K = a.shape[1]
    for at in sorted({0, K // 16 * 8, K - 8}):
        v = a.clone()
        v[:, at:at + 8] = 0
        yield f"lost k {at}", v
    yield "rows moved", a.roll(1, 0)


@pytest.mark.parametrize("K", LENGTHS)
def test_bf16(K):
    g = gen(K)
    a, w = normal(g, 8, K), normal(g, 256, K)
    y, err = ref.product_bf16(a, w)
    limit = ref.rounded(y, err)
    assert (y.abs() > limit).double().mean() > 0.9                  # zeros
    got = torch.zeros_like(y, dtype=torch.float32)                  # eight at a time in f32
    for k in range(0, K, 8):
        got += (a[:, k:k + 8].double() @ w[:, k:k + 8].double().t()).float()
    assert ((got.to(torch.bfloat16).double() - y).abs() <= limit).all()
    for name, v in lost(a):
        assert ((ref.product_bf16(v, w)[0] - y).abs() > limit).any(), name


@pytest.mark.parametrize("K", [k for k in LENGTHS if k % 16 == 0])
def test_int8(K):
    g = gen(K + 1)
    (a, s), (w, ws) = ref.integers(normal(g, 8, K)), ref.integers(normal(g, 256, K))
    y, err = ref.product_int8(a, s, w, ws)
    limit = ref.rounded(y, err)
    assert (y.abs() > limit).double().mean() > 0.9
    f = torch.float32
    got = (a @ w.t()).to(f) * torch.outer(s.to(f), ws.to(f))
    assert ((got.to(torch.bfloat16).double() - y).abs() <= limit).all()
    for name, v in lost(a):
        assert ((ref.product_int8(v, s, w, ws)[0] - y).abs() > limit).any(), name
    for name, got in (("row scale", ref.product_int8(a, s.roll(1), w, ws)[0]),
                      ("channel scale", ref.product_int8(a, s, w, ws.roll(1))[0])):
        assert ((got - y).abs() > limit).any(), name


def test_gated():
    g = gen(3)
    a, w = normal(g, 8, 512), normal(g, 256, 512) * 0.05
    h, err = ref.gated(*ref.product_bf16(a, w))
    limit = ref.rounded(h, err)
    assert (h.abs() > limit).double().mean() > 0.9
    gu = (a.float() @ w.float().t())
    got = gu[:, :128] * torch.sigmoid(gu[:, :128]) * gu[:, 128:]
    assert ((got.to(torch.bfloat16).double() - h).abs() <= limit).all()
    swapped = gu[:, 128:] * torch.sigmoid(gu[:, 128:]) * gu[:, :128]
    assert ((swapped.double() - h).abs() > limit).any()
    q, s = ref.integers(got.to(torch.bfloat16))
    ref.check_quantised(q, s.float(), h, err, "h")
    for bad_q, bad_s in ((q.roll(1, 1), s), (q, s * 1.01), (q + 1, s)):
        with pytest.raises(AssertionError):
            ref.check_quantised(bad_q, bad_s.float(), h, err, "h")


def test_integers():
    """The definition itself: ties to even, the row of zeros, the least scale, infinities and NaN."""
    x = torch.tensor([[127.0, 63.5, 62.5, -0.5, 1.5, -127.0, 0.0, 126.5],
                      [1.0, 0.5, -0.5, 0.25, 0.75, -1.0, 2.0 ** -8, 0.0],
                      [0.0] * 8,
                      [2.0 ** -133] + [0.0] * 7,
                      [float("inf"), 1.0] + [0.0] * 6, [NAN := float("nan"), 1.0] + [0.0] * 6])
    q, s = ref.integers(x.to(torch.bfloat16))
    assert q[0].tolist()[:7] == [127, 64, 62, 0, 2, -127, 0]
    assert q[1].tolist() == [127, 64, -64, 32, 95, -127, 0, 0]      # 63.5 to even, 31.75, 95.25
    assert not q[2:].any()
    assert s[0] == 1.0 and s[2] == s[3] == 2.0 ** -126 and torch.isnan(s[4:]).all() and NAN != NAN
