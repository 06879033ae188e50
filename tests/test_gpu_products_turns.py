"""The products' persistent kernel where a workgroup has several tiles, every shape of it at lengths of k on both sides of
how far its loads are ahead: values, rows behind the last segment, the same bits on every call."""
import pytest

import product_choice as choice
import product_turns as turns
from gpu_util import say
from test_gpu_experts import ep  # noqa: F401
from test_gpu_products_kernels import Case, check_values

pytestmark = pytest.mark.gpu
CASES = [(c, save) for c in turns.cases() for save in ((False, True) if c[:2] == (2, "gated") else (False,))]


@pytest.mark.parametrize("c", CASES, ids=lambda c: turns.label(c[0]) + ("-saved" if c[1] else ""))
def test_values(ep, c):  # noqa: F811
    key, save = c
    counts, N, K = sizes = turns.case(key)
    assert choice.product(counts, N, K, key[0], key[1], turns.BEHIND) == key[2:4]
    say(f"{turns.label(key)}{' saved' if save else ''}: E={len(counts)} S={sum(counts)} N={N} K={K}")
    check_values(Case(ep, key[:4], behind=turns.BEHIND, save=save, sizes=sizes))
