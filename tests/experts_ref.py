"""The expert operators' definitions in 64 bits (plain torch, any device) and the error bounds that
their tests use.

Bounds.  Every product of two e4m3 or bf16 values is exact in f32.  A sum of n f32 terms, in any
order, each addition off by at most 2^-23 of its result (one f32 step: a matrix unit may cut
instead of rounding), is off by at most n 2^-23 sum|terms| to first order; n 2^-22 covers the rest
for n < 2^20.  The 8-bit matrix unit does better or worse than that with the values: it aligns the
products that it sums at once and keeps some 17 bits of the largest, so that its results are
measured 1.6e-5 of the magnitude off, for 128 products as for 7168; n 2^-22 sum|terms| is 3e-5 of it
at n = 128 and more beyond (below, random signs leave less than either).  A rounding to type t is off by at most eps(t) / 2 relative to the value: bf16 2^-8,
e4m3 2^-4 (and half of its smallest step, 2^-10, in units of the block's scale).
"""
import torch

BLOCK = 128
BF16, E4M3, F32 = 2.0 ** -8, 2.0 ** -4, 2.0 ** -24


def blocks(n):
    return -(-n // BLOCK)


def sum_bound(n, mag):
    return n * 2.0 ** -22 * mag


def scale_exponent(amax):
    """Exponent of the least power of two s with amax / s <= 448, at least -126; 0 for no magnitude."""
    m, e = torch.frexp(amax.double())            # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    return torch.where(amax == 0, torch.zeros_like(e), e)


def round_e4m3(u):
    """Nearest e4m3 value, ties to even (u within +-448; NaN stays)."""
    step = torch.exp2((torch.frexp(u)[1] - 1).clamp(min=-6).double() - 3)
    return torch.round(u / step) * step


def quantize_rows(x):
    """x [..., n] -> (e4m3 values in units of the scale [..., n], scale bytes [..., blocks])."""
    n, nb = x.shape[-1], blocks(x.shape[-1])
    v = x.double()
    finite = torch.where(torch.isfinite(v), v, torch.zeros_like(v)).abs()
    pad = finite.new_zeros(*x.shape[:-1], nb * BLOCK)
    pad[..., :n] = finite
    e = scale_exponent(pad.view(*x.shape[:-1], nb, BLOCK).amax(-1))
    s = torch.exp2(e.double()).repeat_interleave(BLOCK, -1)[..., :n]
    q = torch.where(torch.isfinite(v), round_e4m3(v / s), torch.full_like(v, float("nan")))
    return q, (e + 127).to(torch.uint8)


def quantize_weight(w):
    """w [E][N][K] -> (values in units of the scale, scale bytes [E][NB][KB])."""
    E, N, K = w.shape
    nb, kb = blocks(N), blocks(K)
    v = w.double()
    pad = v.new_zeros(E, nb * BLOCK, kb * BLOCK)
    pad[:, :N, :K] = v.abs()
    e = scale_exponent(pad.view(E, nb, BLOCK, kb, BLOCK).amax((2, 4)))
    return round_e4m3(v / weight_scale(e, N, K)), (e + 127).to(torch.uint8)


def weight_scale(e, N, K):
    s = torch.exp2(e.double())
    return s.repeat_interleave(BLOCK, 1)[:, :N].repeat_interleave(BLOCK, 2)[:, :, :K]


def values(q, byte):
    """Rows' values in f64."""
    s = torch.exp2(byte.double() - 127).repeat_interleave(BLOCK, -1)
    return q.double() * s[..., :q.shape[-1]]


def weight_values(w, byte):
    if byte is None:
        return w.double()
    return w.double() * weight_scale(byte.double() - 127, w.shape[1], w.shape[2])


def segments(offsets):
    b = offsets.tolist()
    return [(e, b[e], b[e + 1]) for e in range(len(b) - 1)]


def grouped(a, w, offsets):
    """(a W^T by segment [rows][N], the sums of magnitudes) in f64; rows outside are zero."""
    y = a.new_zeros(a.shape[0], w.shape[1])
    mag = torch.zeros_like(y)
    for e, lo, hi in segments(offsets):
        y[lo:hi] = a[lo:hi] @ w[e].t()
        mag[lo:hi] = a[lo:hi].abs() @ w[e].abs().t()
    return y, mag


def gated(gu, mag, n):
    """h = silu(g) u in f64 and a bound on the f32 result's error from sums of n terms with
    magnitudes `mag` ([g; u] as gu).  |silu'| <= 1.1; exp(-g) in f32 is off by (|g| + 4) steps
    relatively, and the remaining operations by 8 more."""
    I = gu.shape[-1] // 2
    g, u = gu[..., :I], gu[..., I:]
    dg, du = sum_bound(n, mag[..., :I]), sum_bound(n, mag[..., I:])
    silu = g * torch.sigmoid(g)
    h = silu * u
    err = 1.1 * dg * u.abs() + silu.abs() * du + 1.1 * dg * du + (g.abs() + 12) * 2.0 ** -23 * h.abs()
    return h, err
