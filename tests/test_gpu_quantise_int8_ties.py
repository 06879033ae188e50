"""Every bf16 value below every mantissa of a row's maximum, quantised to int8 by each form of the kernel."""
import pytest
import torch

import products_ref as ref
from gpu_util import DEV, say
from test_gpu_experts import ep  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("exponent", [7, 127, 254])
@pytest.mark.parametrize("H", [2048, 8192, 16384])
def test_every_value(ep, H, exponent):  # noqa: F811
    say(f"every value, H={H}, maximum's exponent {exponent}")
    for low in range(0, 128, 32):
        rows = []
        for mantissa in range(low, low + 32):
            top = exponent << 7 | mantissa
            x = torch.arange(0, top + 1, device=DEV, dtype=torch.int32)
            x = torch.cat([x, x | 0x8000])
            x = torch.cat([x, x.new_zeros(-x.numel() % (H - 1))]).view(-1, H - 1)
            rows.append(torch.cat([x, x.new_full((x.shape[0], 1), top)], 1))
        x = torch.cat(rows).to(torch.int16).view(torch.bfloat16)
        q, scale = ep.ep_quantize_int8(x)
        torch.cuda.synchronize()
        ref.check_rows(q, scale, x, f"mantissas from {low}")
