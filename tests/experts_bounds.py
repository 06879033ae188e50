"""Error bounds of the expert operators that stay well below what a lost piece of a sum changes
(test_experts_bounds.py plants such mistakes), from what the matrix units do.

8-bit unit (e4m3, block-scaled, 16 x 16 x 128 and 32 x 32 x 64 alike): it adds the products of eight
neighbouring k at a time.  Before that it cuts each of them, towards zero, to a multiple of 2^-13 of 2^E,
E the largest sum of two operands' exponents among the eight; what it adds up beyond that, and to the
accumulator, is f32.  (Measured by products 2^12 + 2^-s: 2^-1 stays and 2^-2 goes within a group of
eight, all of 2^-11 stay in other groups.)  A normal operand is at least 2^exponent; a subnormal's
exponent is that of 2^-6 in units of its scale.  With A and W the largest magnitudes of the eight
operands, 2^-6 of the scale at least: 2^E <= A W, and eight products lose less than 8 * 2^-13 A W.

bf16 unit: it adds eight products at a time to f32 accuracy.  So does f32 itself: one addition is off
by at most 2^-23 of its result (cut, or rounded with half that), and n / 8 groups take n / 4 additions
at most, one for the group's own sum and one to the accumulator.
"""
import torch

from experts_ref import BF16, E4M3, BLOCK, blocks

GROUP = 8


def _tops(v, byte_scale):
    """[rows][k] f64 -> [rows][ceil(k / 8)]: the largest magnitude of eight, 2^-6 of the scale at least."""
    n = v.shape[-1]
    m = torch.maximum(v.abs(), 2.0 ** -6 * byte_scale)
    if n % GROUP:
        m = torch.cat([m, m.new_zeros(*m.shape[:-1], GROUP - n % GROUP)], -1)
    return m.view(*m.shape[:-1], -1, GROUP).amax(-1)


def row_scales(byte, n):
    return torch.exp2(byte.double() - 127).repeat_interleave(BLOCK, -1)[..., :n]


def weight_scales(byte, N, K):
    s = torch.exp2(byte.double() - 127)
    return s.repeat_interleave(BLOCK, -2)[..., :N, :].repeat_interleave(BLOCK, -1)[..., :, :K]


def additions(n):
    return n / 4 + 2


def product(a, a_byte, w, w_byte):
    """Rows a [S][K], one expert's weights w [N][K] as f64 values with their scale bytes ->
    (a W^T, what its f32 sum is off by at most)."""
    y = a @ w.t()
    cut = _tops(a, row_scales(a_byte, a.shape[1])) @ _tops(w, weight_scales(w_byte, *w.shape)).t()
    err = GROUP * 2.0 ** -13 * cut + additions(a.shape[1]) * 2.0 ** -23 * (a.abs() @ w.abs().t())
    return y, err


def product_bound(y, err):
    """... rounded to bf16."""
    return BF16 * (y.abs() + err) + err


def gated(gu, err):
    """h = silu(g) u in f64 and what the f32 result is off by, g and u off by `err`.  |silu'| <= 1.1;
    exp(-g) in f32 is off by (|g| + 4) steps relatively, and the remaining operations by 8 more."""
    I = gu.shape[-1] // 2
    g, u, dg, du = gu[..., :I], gu[..., I:], err[..., :I], err[..., I:]
    silu = g * torch.sigmoid(g)
    h = silu * u
    return h, 1.1 * dg * u.abs() + silu.abs() * du + 1.1 * dg * du + (g.abs() + 12) * 2.0 ** -23 * h.abs()


def quantised_bound(h, err, unit):
    """e4m3 of a value off by err: half a step of the value, or of the smallest step in units of the
    scale (`unit`, the scale at each place)."""
    return E4M3 * (h.abs() + err) + 2.0 ** -10 * unit + err


# ----------------------------------------------------------------- 2-norms
# Sums of terms with independent signs: a partial sum is in the 2-norm over the outputs no larger than
# the whole (the terms' squares add up), so that n additions, each off by 2^-23 of a partial sum, are off
# by n 2^-23 of the result's 2-norm even if all their errors point one way.
def wgrad_norm(n):
    """Relative 2-norm of a weight gradient's error, n rows."""
    return additions(n) * 2.0 ** -23 + 2.0 ** -24


# The few-token layer, relative 2-norm over up to 128 neighbouring outputs of one token.  Rounding the
# output: each value by at most 2^-8 of itself, so the norm by that.  All else: f32 sums as above, gate
# and up each in four parts of H (twice H / 16 additions in a row), the second product I / 4, so
# (H / 2 + I) / 4 * 2^-23 < 2^-10 for H / 2 + I < 32768; h held to 2^-16 twice, exponentials of |g| <= 16
# to (16 + 12) 2^-23 and the picks' sum: below 2^-14.  Errors of h meet random weights and pass the norm
# as h itself does.
MOE_NORM = 2.0 ** -8 + 2.0 ** -10 + 2.0 ** -14


def norm_excess(got, want, limit, chunk=128):
    """The largest of |got - want| - limit |want| over pieces of `chunk` values (2-norms)."""
    n = want.shape[-1]
    d = got.double() - want.double()
    worst = -float("inf")
    for c in range(0, n, chunk):
        e = d[..., c:c + chunk].norm(dim=-1) - limit * want[..., c:c + chunk].double().norm(dim=-1)
        worst = max(worst, e.max().item() if e.numel() else worst)
    return worst
