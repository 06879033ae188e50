"""The few-token layer where h = w silu(g) u leaves bf16's range or f32's: its two bf16 halves hold every
finite f32 value, and an infinite one stays infinite."""
import pytest
import torch

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
INF = float("inf")
GATE = 64.0        # silu(64) is 64 in f32


@pytest.fixture(scope="module")
def ep():
    from combine_ep_route_topk_amd import ep as mod
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    return mod


def case(ep, T, up, fp8):
    """One expert.  Odd tokens read column 0 of the first weights, h = w GATE up at position 5 and zero
    elsewhere; even ones column 1, h = w GATE everywhere.  The second weights are +-2^-100."""
    H, I = 272, 128
    x = torch.zeros((T, H), device=DEV)
    x[0::2, 1], x[1::2, 0] = 1.0, 1.0
    if T == 1:
        x[0] = 0
        x[0, 0] = 1.0
    w13 = torch.zeros((1, 2 * I, H), device=DEV)
    w13[0, :I, :2] = GATE
    w13[0, I + 5, 0] = up
    w13[0, I:, 1] = 1.0
    sign = torch.where(torch.arange(H, device=DEV) % 3 == 0, -1.0, 1.0)
    w2 = (sign * 2.0 ** -100)[None, :, None].expand(1, H, I)
    w13, w2 = w13.to(torch.bfloat16), w2.to(torch.bfloat16).contiguous()
    s13 = s2 = None
    if fp8:
        # column 1's values would vanish next to a large one in their block: 1.0 there only where it is small
        if abs(up) > 1e6:
            w13[0, I:, 1] = 0.0
        d13, d2 = ep.ep_quantize_weight_fp8(w13), ep.ep_quantize_weight_fp8(w2)
        w13, s13, w2, s2 = d13["q"], d13["scale"], d2["q"], d2["scale"]
    odd = x[:, 0] == 1.0
    return x.to(torch.bfloat16), odd, sign, dict(w13=w13, w2=w2, w13_scale=s13, w2_scale=s2)


def run(ep, x, w, W):
    T = x.shape[0]
    idx = torch.zeros((T, 1), dtype=torch.int32, device=DEV)
    out = ep.ep_moe_tokens(x, idx, torch.full((T, 1), w, device=DEV), **W)
    torch.cuda.synchronize()
    return out.double()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 3, 12, 40])
@pytest.mark.parametrize("up", [2.0 ** 121, -2.0 ** 121])
def test_h_past_bf16(ep, T, up, fp8):
    """|h| = w 2^127 up to f32's largest value.  h is held to 2^-15, the sums are exact, and the output
    rounds once: 2^-8 + 2^-15 of the value."""
    x, odd, sign, W = case(ep, T, up, fp8)
    for w in (1.0, 1.9921875, 1.995, 1.9965, 1.998, 1.99999988):
        say(f"moe tokens T={T} h={w} * 2^127 fp8={fp8}")
        out = run(ep, x, w, W)
        h = torch.tensor(w, dtype=torch.float32).double().item() * GATE * up
        want = h * sign.double() * 2.0 ** -100
        assert ((out[odd] - want).abs() <= (2.0 ** -8 + 2.0 ** -15) * want.abs()).all(), (w, out[odd][0])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 3, 12, 40])
@pytest.mark.parametrize("up", [2.0 ** 127, -2.0 ** 127])
def test_h_infinite(ep, T, up, fp8):
    """h = +-inf at one place: the outputs are the infinities of its sign times the weights', and the
    tokens beside it keep their bits."""
    x, odd, sign, W = case(ep, T, up, fp8)
    say(f"moe tokens T={T} infinite h fp8={fp8}")
    out = run(ep, x, 1.0, W)
    want = torch.copysign(torch.full_like(sign, INF), sign * up).double()
    assert (out[odd] == want).all(), out[odd][0]
    if not odd.all():
        alone = run(ep, x[~odd].contiguous(), 1.0, W)
        assert torch.isfinite(alone).all() and torch.equal(out[~odd], alone)


def test_h_nan_stays(ep):
    """A NaN among the first weights meets every token of its expert (also times zero), and stays one
    through the halves of h."""
    x, _, _, W = case(ep, 4, 2.0 ** 121, False)
    W["w13"][0, 3, 0] = float("nan")
    say("moe tokens NaN h")
    assert torch.isnan(run(ep, x, 1.0, W)).all()
