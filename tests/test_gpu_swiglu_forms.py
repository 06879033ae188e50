"""The activation's gradient with and without h, the value that the second weights' gradient takes."""
import pytest
import torch

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S,I", [(1, 8), (257, 1408), (0, 16)])
def test_h_is_optional(S, I):
    from combine_ep_route_topk_amd import ep
    g = torch.Generator(device=DEV).manual_seed(S + I)
    dh, gu = (torch.randn((S, n), generator=g, device=DEV).to(torch.bfloat16) for n in (I, 2 * I))
    say(f"swiglu grad without h S={S} I={I}")
    want, h = ep.ep_swiglu_grad(dh, gu)
    got, none = ep.ep_swiglu_grad(dh, gu, save_h=False)
    mine = torch.full((S, I), -1, dtype=torch.int16, device=DEV).view(torch.bfloat16)
    again, same = ep.ep_swiglu_grad(dh, gu, h=mine, save_h=False)
    torch.cuda.synchronize()
    assert none is None and same is mine
    assert torch.equal(got, want) and torch.equal(again, want) and torch.equal(mine, h)
