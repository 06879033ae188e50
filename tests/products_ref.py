"""The bf16 and int8 expert operators' definitions in 64 bits (plain torch, any device) and their error
bounds.

bf16 products.  The matrix unit adds eight products at a time to f32 accuracy, and one f32 addition is off by
at most 2^-23 of its result (cut, or rounded with half that): n / 4 + 2 additions of partial sums that are no
larger than sum|terms| (experts_bounds.additions).  int8 products: the sum is an integer, exact; its
conversion to f32, the product of the scales and the last product are off by at most 2^-24 each: 4 * 2^-24 of
the value covers the three, as long as nothing is subnormal.  Results round to bf16: 2^-8 of the value.

Quantised rows: q is the integer nearest to 127 x / m exactly (ties to even), the scale m / 127 is rounded
once to f32.
"""
import torch

import experts_bounds as bounds
from experts_ref import BF16, F32

LEAST = 127.0 * 2.0 ** -126
NAN = float("nan")


def segments(offsets):
    b = offsets.tolist()
    return [(e, b[e], b[e + 1]) for e in range(len(b) - 1) if b[e + 1] > b[e]]


# ----------------------------------------------------------------- rows to integers
def integers(x):
    """x [..., H] -> (integers as f64, scales f64).  The quotient in f64 is off by 2^-52 of itself at most, and a
    half integer or 2^-16 of itself away from one (x and m have 8 bits): its rounding is exact."""
    v = x.double()
    ok = torch.isfinite(v).all(-1)
    v = torch.where(ok[..., None], v, torch.zeros_like(v))
    m = v.abs().amax(-1).clamp(min=LEAST)
    scale = torch.where(ok, m / 127.0, torch.full_like(m, NAN))
    return torch.round(v * 127.0 / m[..., None]), scale


def check_rows(q, scale, x, what="rows"):
    want, unit = integers(x)
    assert torch.equal(q.double(), want), f"{what}: {int((q.double() != want).sum())} integers differ"
    nan = torch.isnan(unit)
    assert torch.equal(torch.isnan(scale), nan), f"{what}: scales"
    off = (scale.double() - unit).abs()[~nan]
    assert (off <= F32 * unit[~nan]).all(), f"{what}: scales"


# ----------------------------------------------------------------- products
def product_bf16(a, w):
    """Rows a [S][K], weights w [N][K] -> (a W^T in f64, what its f32 sum is off by at most)."""
    a, w = a.double(), w.double()
    return a @ w.t(), bounds.additions(a.shape[1]) * 2.0 ** -23 * (a.abs() @ w.abs().t())


def product_int8(a, a_scale, w, w_scale):
    y = (a.double() @ w.double().t()) * torch.outer(a_scale.double(), w_scale.double())
    return y, 4 * F32 * y.abs()


def rounded(y, err):
    """What a value off by err, rounded to bf16, is off by at most."""
    return BF16 * (y.abs() + err) + err


def gated(gu, err):
    """h = silu(g) u in f64 and what the f32 result is off by."""
    return bounds.gated(gu, err)


def check(got, want, limit, what):
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = ((got - want).abs() - limit).max().item() if got.numel() else -1.0
    assert over <= 0, f"{what}: {over:.3g} over the bound"


def check_quantised(q, scale, h, err, what):
    """Rows that were off by err, rounded to bf16 and then quantised: the scale is that of the largest
    magnitude, an integer half a step off at most (and 2^-23 of its 127 steps, the scale's own)."""
    limit = rounded(h, err)
    m, dm = h.abs().amax(-1), limit.amax(-1)
    low = torch.clamp(m - dm, min=LEAST) / 127.0
    high = torch.clamp(m + dm, min=LEAST) / 127.0
    s = scale.double()
    assert ((s >= low * (1 - F32)) & (s <= high * (1 + F32))).all(), f"{what}: scales"
    check(q.double() * s[..., None], h, limit + s[..., None] * (0.5 + 127 * 2.0 ** -23), what)
