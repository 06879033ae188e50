"""Which kernel a call takes: every one is reached, at the sizes that its measurements speak for."""
import pytest

import expert_choice as choice


@pytest.mark.parametrize("S,N,E,gated,kernel", [
    (32768, 7168, 8, False, "large"), (32768, 4096, 8, True, "large"), (8 * 192, 4096, 8, False, "large"),
    (16 * 128, 2816, 16, False, "128x256"), (16 * 128, 2816, 16, True, "128x256"),
    (2048, 4096, 1, False, "large"), (1024, 4096, 1, False, "64x256"),
    (16 * 30, 2816, 16, False, "32x256"), (18 * 45, 3584, 18, True, "64x256"),
    (64, 4096, 1, True, "32x256"), (8 * 48, 4096, 8, True, "32x256"),
    (8 * 32, 4096, 8, False, "128x128"), (8 * 8, 4096, 8, False, "64x128"), (32 * 16, 4096, 32, False, "64x128"),
    (2 * 8, 4096, 2, False, "32x64"), (1, 16, 1, False, "32x64"),
])
def test_product(S, N, E, gated, kernel):
    assert choice.gemm(S, N, E, gated) == kernel


def test_every_kernel_is_reached():
    assert {choice.gemm(rows * E, N, E) for rows in (1, 8, 30, 32, 96, 128, 512, 4096)
            for N in (128, 2816, 4096) for E in (1, 8, 16, 32)} == set(choice.GEMM)
    assert {choice.gemm(rows * E, N, E, True) for rows in (1, 32, 45, 96, 4096) for N in (256, 4096)
            for E in (1, 8, 18)} == {"large", "128x256", "64x256", "32x256"}


def test_experts_without_rows_do_not_count():
    """At most S experts have rows: more experts than that change nothing."""
    assert choice.gemm(8, 2048, 64) == "32x64"
    for gated in (False, True):
        for S in (1, 2, 3, 8, 17, 40, 63, 200):
            for N in (256, 1024, 2048, 2816, 4096, 7168):
                for E in (2, 8, 64, 256, 1024):
                    assert choice.gemm(S, N, E, gated) == choice.gemm(S, N, min(S, E), gated), (S, N, E)


def test_weight_gradients():
    assert choice.wgrad(32768, 4096, 7168, 8) == "large"
    assert choice.wgrad(2000, 2816, 4096, 16) == 1
    assert choice.wgrad(32768, 256, 512, 1) == 64
    assert choice.wgrad(100, 256, 512, 1) == 1
