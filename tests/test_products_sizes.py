"""Sizes that the bf16 and int8 expert operators refuse, without a GPU: what the ABI's 32 bits cannot hold."""
import pytest
import torch

from test_experts_refusals import ep  # noqa: F401


def many(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("shape", [(1, (1 << 32) + 16), (2, 3, 1 << 31), (0, (1 << 32) + 16),
                                   ((1 << 31) - 1, 2, 16)], ids=str)
def test_rows_to_quantise(ep, shape):  # noqa: F811
    """A row's length as well as their number: 2^32 + 16 values were cut to 16."""
    with pytest.raises(ValueError, match="2\\^31"):
        ep.ep_quantize_int8(many(*shape))
