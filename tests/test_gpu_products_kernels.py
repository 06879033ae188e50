"""Every kernel that the bf16 and int8 products choose from (sizes found by the rules themselves): values, NaN and
infinities that stay with their rows, offsets that make no sense, the same bits on every call."""
import pytest
import torch

import product_choice as choice
import products_ref as ref
import test_gpu_products as gpu
from gpu_util import DEV, say
from test_gpu_experts import ep, gen, offsets_of  # noqa: F401
from test_gpu_experts_isolation import nonsense

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
BEHIND = 7


class Case:
    """Operands of one kernel, and the call on them with all outputs: [(tensor [S][..], columns of it that
    stand for one channel)]."""

    def __init__(self, ep, c, behind=BEHIND, save=False, sizes=None):  # noqa: F811
        self.ep, self.bytes, self.kind, self.save = ep, c[0], c[1], save
        self.counts, self.N, self.K = sizes or choice.case(c[2], c[3], c[0], c[1], behind)
        self.E, self.S, self.n = len(self.counts), sum(self.counts) + behind, sum(self.counts)
        g = gen(self.S + self.N)
        self.off = offsets_of(self.counts)
        self.channels = 2 * self.N if self.kind == "gated" else self.N
        shape = (self.E, self.K, self.N) if self.kind == "transposed" else (self.E, self.channels, self.K)
        x = gpu.tokens(g, self.S, self.K)
        if self.bytes == 2:
            self.a, self.a_s, self.w, self.w_s = x, None, gpu.matrices(g, *shape), None
            if self.kind == "gated":
                self.w *= self.K ** -0.5
        else:
            self.a, self.a_s = gpu.int8_rows(x)
            self.w, self.w_s = gpu.int8_matrices(g, *shape)
            self.w_s *= self.K ** -0.5

    def buffers(self, pad=0):
        """Outputs filled with a value that no call leaves, `pad` rows of guard on both sides."""
        bf = lambda w: torch.full((self.S + 2 * pad, w), 7.0, dtype=torch.bfloat16, device=DEV)  # noqa: E731
        if self.kind != "gated":
            return [bf(self.N)]
        if self.bytes == 2:
            return [bf(self.N)] + ([bf(2 * self.N)] if self.save else [])
        return [torch.full((self.S + 2 * pad, self.N), 0x55, dtype=torch.int8, device=DEV),
                torch.full((self.S + 2 * pad,), 7.0, device=DEV)]

    def run(self, out, off=None, pad=0):
        off = self.off if off is None else off
        o = [t[pad:pad + self.S] for t in out]
        if self.kind != "gated":
            if self.bytes == 2:
                self.ep.ep_expert_gemm_bf16(self.a, self.w, off, transposed=self.kind == "transposed", y=o[0])
            else:
                self.ep.ep_expert_gemm_int8(self.a, self.a_s, self.w, self.w_s, off, y=o[0])
        elif self.bytes == 2:
            self.ep.ep_expert_swiglu_bf16(self.a, self.w, off, h=o[0], gate_up=o[1] if self.save else None)
        else:
            self.ep.ep_expert_swiglu_int8(self.a, self.a_s, self.w, self.w_s, off, h=o[0], h_scale=o[1])
        torch.cuda.synchronize()
        return out

    def products(self, e, lo, hi):
        if self.bytes == 1:
            return ref.product_int8(self.a[lo:hi], self.a_s[lo:hi], self.w[e], self.w_s[e])
        return ref.product_bf16(self.a[lo:hi], self.w[e].t() if self.kind == "transposed" else self.w[e])


CASES = choice.cases()
SAVED = [(c, save) for c in CASES for save in ((False, True) if c[:2] == (2, "gated") else (False,))]


def name(c):
    return choice.label(c[0]) + ("-saved" if c[1] else "") if isinstance(c[1], bool) else choice.label(c)


def check_values(k):
    out = k.run(k.buffers())
    for t, fresh in zip(out, k.buffers()):
        assert torch.equal(t[k.n:], fresh[k.n:]), "rows behind the last segment"
    for e, lo, hi in ref.segments(k.off):
        y, err = k.products(e, lo, hi)
        if k.kind != "gated":
            ref.check(out[0][lo:hi], y, ref.rounded(y, err), f"expert {e}")
            continue
        h, herr = ref.gated(y, err)
        if k.bytes == 1:
            ref.check_quantised(out[0][lo:hi], out[1][lo:hi], h, herr, f"expert {e}")
            continue
        ref.check(out[0][lo:hi], h, ref.rounded(h, herr), f"h of expert {e}")
        if k.save:
            ref.check(out[1][lo:hi], y, ref.rounded(y, err), f"gate_up of expert {e}")
    again = k.run(k.buffers())
    assert all(torch.equal(a, b) for a, b in zip(out, again)), "another call, other bits"


@pytest.mark.parametrize("c", SAVED, ids=name)
def test_values(ep, c):  # noqa: F811
    say(f"values on {name(c)}")
    check_values(Case(ep, c[0], save=c[1]))


# More experts than a wave has lanes, whose tiles are found by a scan, and a last round in pieces:
# (bytes, kind, halvings, rows of each expert, columns, K)
SCANNED = [(2, "plain", 1, 520, 520, 272), (2, "transposed", 1, 520, 520, 272), (2, "gated", 1, 520, 264, 272),
           (1, "plain", 1, 520, 528, 528), (1, "gated", 1, 520, 272, 528), (2, "plain", 2, 700, 1040, 144),
           (2, "transposed", 2, 700, 1040, 144), (1, "plain", 2, 700, 1040, 272), (1, "gated", 2, 700, 528, 272)]


@pytest.mark.parametrize("c", SCANNED, ids=lambda c: "-".join(map(str, c)))
def test_last_round_of_many_experts(ep, c):  # noqa: F811
    bytes_, kind, halved, rows, N, K = c
    counts = [rows + i % 3 for i in range(70)]
    counts[11], counts[12], counts[13] = 0, 2 * counts[12], counts[13] - 1
    assert choice.product(counts, N, K, bytes_, kind, BEHIND)[0] == choice.TAILS[halved]
    say(f"{c}")
    check_values(Case(ep, c, sizes=(counts, N, K)))


def spoil(k):
    """NaN in one row of the first expert with rows, infinity in the last row of another, NaN in channel 5 of that
    other's weights, in all weights of the last expert, and in the rows behind.  Returns (rows that are lost
    throughout, the expert whose channel 5 is NaN)."""
    b = k.off.tolist()
    used = [e for e in range(k.E) if b[e + 1] > b[e]]
    first, other, last = used[0], used[1], used[-1]
    if other == last:
        other = first
    bad = torch.zeros(k.S, dtype=torch.bool, device=DEV)
    bad[b[first]] = True
    bad[b[other + 1] - 1] = True
    bad[b[last]:b[last + 1]] = True
    if k.bytes == 2:
        k.a[b[first]] = NAN
        k.a[b[other + 1] - 1, k.K - 1] = INF
        k.a[b[-1]:] = NAN
        if k.kind == "transposed":
            k.w[other, :, 5] = NAN
        else:
            k.w[other, 5] = NAN
        k.w[last] = NAN
    else:
        k.a_s[b[first]] = NAN
        k.a_s[b[other + 1] - 1] = INF
        k.a_s[b[-1]:] = NAN
        k.w_s[other, 5] = NAN
        k.w_s[last] = NAN
    return bad, other


@pytest.mark.parametrize("c", SAVED, ids=name)
def test_keeps_nan_to_its_rows(ep, c):  # noqa: F811
    say(f"NaN on {name(c)}")
    k = Case(ep, c[0], save=c[1])
    clean = k.run(k.buffers())
    rows, other = spoil(k)
    out = k.run(k.buffers())
    b, n = k.off.tolist(), k.n
    channel = torch.zeros(k.S, dtype=torch.bool, device=DEV)
    channel[b[other]:b[other + 1]] = True
    fresh = k.buffers()
    for t, f in zip(out, fresh):
        assert torch.equal(t[n:], f[n:]), "rows behind the last segment"
    if k.bytes == 1 and k.kind == "gated":
        # a channel that is NaN makes the row's scale NaN
        lost = rows | channel
        assert torch.isnan(out[1][:n][lost[:n]]).all() and not out[0][:n][lost[:n]].any()
        for t, u in zip(out, clean):
            assert torch.equal(t[:n][~lost[:n]], u[:n][~lost[:n]])
        return
    for i, (t, u) in enumerate(zip(out, clean)):
        lost = rows[:n, None].expand(n, t.shape[1]).clone()
        lost[channel[:n], 5] = True                  # gate's channel 5: h's and gate_up's column 5
        assert not torch.isfinite(t[:n][lost]).any(), i
        assert torch.equal(t[:n][~lost], u[:n][~lost]), i


@pytest.mark.parametrize("c", SAVED, ids=name)
def test_stays_inside(ep, c):  # noqa: F811
    """Offsets that decrease, overlap or leave the buffer: unspecified rows, never an access outside."""
    k, pad = Case(ep, c[0], behind=0, save=c[1]), 64
    for i, off in enumerate(nonsense(k.S, k.E)):
        say(f"offsets {i} on {name(c)}")
        out = k.run(k.buffers(pad), off, pad)
        for t, f in zip(out, k.buffers(pad)):
            assert torch.equal(t[:pad], f[:pad]) and torch.equal(t[pad + k.S:], f[pad + k.S:])
