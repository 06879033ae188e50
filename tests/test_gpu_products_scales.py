"""Scales of the int8 products at the ends of what is documented: the largest channel scale with the largest sum, small
and large token scales beside them, and the least ones."""
import pytest
import torch

import products_ref as ref
from gpu_util import DEV, say
from test_gpu_experts import ep, gen, offsets_of  # noqa: F401
from test_gpu_products import int8_rows, tokens

pytestmark = pytest.mark.gpu
MOST, LEAST = 2.0 ** 97, 2.0 ** -126


@pytest.mark.parametrize("rows", [3, 300, 20_000])
@pytest.mark.parametrize("v,x", [(-128, -128), (127, -128), (127, 127)])
def test_gemm(ep, v, x, rows):  # noqa: F811
    """Sums of 2^31 - 2^18 and less, whose product with the scale 2^97 is 2^128 - 2^115, finite.  Rows on the
    narrow kernel, on small tiles and on large ones."""
    K = (1 << 17) - 16
    say(f"int8 scales' ends {v} {x} rows={rows}")
    a = torch.full((rows, K), v, dtype=torch.int8, device=DEV)
    w = torch.full((1, 64, K), x, dtype=torch.int8, device=DEV)
    w[0, 1::2] = 0
    w[0, 1::2, 5] = 1                               # the least sums
    a_s = torch.tensor([2.0 ** -126, 2.0 ** -100, 2.0 ** -3], device=DEV).repeat(-(-rows // 3))[:rows].contiguous()
    w_s = torch.tensor([MOST, MOST, 0.75 * MOST, LEAST, 1.0, 2.0 ** 60, 2.0 ** -60, LEAST], device=DEV).repeat(8)[None]
    y = ep.ep_expert_gemm_int8(a, a_s, w, w_s.contiguous(), offsets_of([rows]))
    torch.cuda.synchronize()
    sums = torch.where(torch.arange(64, device=DEV) % 2 == 0, float(v * x * K), float(v))
    want = sums * torch.outer(a_s.double(), w_s[0].double())
    # a result below bf16's normal numbers is off by half of their least step, 2^-134; above its range, infinite
    top = torch.finfo(torch.bfloat16).max
    inside = want.abs() < top * (1 - 2.0 ** -20)
    limit = ref.rounded(want, 4 * 2.0 ** -24 * want.abs()) + 2.0 ** -134
    assert inside[0].all() and inside.double().mean() > 0.8
    assert ((y.double() - want).abs() <= limit)[inside].all()
    over = want.abs() > top * (1 + 2.0 ** -7)
    assert torch.equal(y[over].double(), torch.sign(want[over]) * float("inf"))


@pytest.mark.parametrize("rows", [3, 300])
def test_swiglu(ep, rows):  # noqa: F811
    """The same through the gate: g and u near 1 from the largest channel scales."""
    K, I = 4096, 32
    say(f"int8 gated scales' ends rows={rows}")
    g = gen(rows)
    a, s = int8_rows(tokens(g, rows, K))
    w = torch.randint(-127, 128, (1, 2 * I, K), generator=g, device=DEV, dtype=torch.int8)
    w_s = torch.full((1, 2 * I), MOST, device=DEV)
    w_s[0, ::3] = MOST / 8
    a_s = s / s.mean() * 2.0 ** -(97 + 18)
    h, h_s = ep.ep_expert_swiglu_int8(a, a_s, w, w_s, offsets_of([rows]))
    torch.cuda.synchronize()
    gu, err = ref.product_int8(a, a_s, w[0], w_s[0])
    assert gu.abs().mean() > 0.1
    ref.check_quantised(h, h_s, *ref.gated(gu, err), "h")
