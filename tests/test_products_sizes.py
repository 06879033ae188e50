"""The sizes of the bf16 and int8 expert operators, without a GPU: what the ABI's 32 bits or a launch cannot hold is
refused, and the rules that choose a kernel hold at every size that is not."""
import subprocess

import pytest
import torch

import product_choice as choice
from expert_choice import CUS, HEADER
from test_experts_refusals import F, ep, refused  # noqa: F401


def many(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("shape", [(1, (1 << 32) + 16), (2, 3, 1 << 31), (0, (1 << 32) + 16),
                                   ((1 << 31) - 1, 2, 16)], ids=str)
def test_rows_to_quantise(ep, shape):  # noqa: F811
    """A row's length as well as their number: 2^32 + 16 values were cut to 16."""
    with pytest.raises(ValueError, match="2\\^31"):
        ep.ep_quantize_int8(many(*shape))


# The rules that choose a kernel, as a program of its own, where arithmetic that C++ does not define ends it:
# lines of S, columns, bytes of a row of k, E, gated, row tiles of 64, 128 and 256 rows; answers are the kernel, the
# persistent tile, their estimates, the least of all estimates of a persistent one, and the most tiles.
PROGRAM = f"""
#include "{HEADER}"
#include <stdio.h>
int main() {{
    long long S, N, bytes, E, t64, t128, t256;
    int gated;
    while (scanf("%lld %lld %lld %lld %d %lld %lld %lld", &S, &N, &bytes, &E, &gated, &t64, &t128, &t256) == 8) {{
        const int blocks = int((bytes + 127) / 128);
        const int kernel = ep::choose_product(S, N, bytes, E, gated != 0, {CUS});
        const int tile = ep::choose_product_tile(int(t64), int(t128), int(t256), int(N), blocks, gated != 0, {CUS});
        const long long rows[] = {{t64, t128, t256}};
        float took[ep::kProductTiles];
        for (int k = 0; k < ep::kProductTiles; ++k) {{
            const ep::ProductTile t = ep::product_tile(k);
            const long long columns = gated ? t.weights / 2 : t.weights;
            const long long n = rows[t.tokens / 128] * ((N + columns - 1) / columns);
            took[k] = ep::product_us(k, float(n), blocks, {CUS});
        }}
        float least = took[0];
        for (float v : took) least = v < least ? v : least;
        printf("%d %d %g %g %lld\\n", kernel, tile, took[tile], least,
               (long long)ep::product_most_tiles(S, N, E, gated != 0));
    }}
}}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    d = tmp_path_factory.mktemp("rules")
    source, program = d / "rules.cpp", d / "rules"
    source.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined,float-cast-overflow",
                    "-fno-sanitize-recover=all", "-o", str(program), str(source)], check=True)

    def ask(cases):
        lines = []
        for rows, E, N, bytes_, gated in cases:      # rows: of each of E experts
            tiles = [E * -(-rows // t) for t in (64, 128, 256)]
            lines.append(" ".join(map(str, (rows * E, N, bytes_, E, int(gated), *tiles))))
        r = subprocess.run([str(program)], input="\n".join(lines), capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return [[float(v) for v in line.split()] for line in r.stdout.splitlines()]

    return ask


SIZES = [(rows, E, N, bytes_, gated) for E in (1, 3, 64, 1024)
         for rows in sorted({1, 2, 63, 1000, 100_000, ((1 << 30) - 1) // E})
         for N in (8, 16, 1000, 8064, 8200, 1 << 17) for bytes_ in (16, 2000, 1 << 18) for gated in (False, True)]


def test_rules_at_every_size(rules):
    """No overflow, the tile is the one of the least estimate, and a narrow kernel's grid stays below its limit
    wherever the persistent one's does."""
    answers = rules(SIZES)
    assert len(answers) == len(SIZES)
    past = 0
    for (rows, E, N, bytes_, gated), (kernel, tile, took, least, most) in zip(SIZES, answers):
        case = (rows, E, N, bytes_, gated)
        assert took <= least * (1 + 1e-6), case
        past += most >= 1 << 30
        name = choice.KERNELS[int(kernel)]
        if name.startswith("narrow") and most < 1 << 30:
            side = 64 if name == "narrow 64x64" else 32
            columns = side // 2 if gated else side
            grid = (rows * E // side + min(E, rows * E)) * -(-N // columns)
            assert grid < 1 << 23, case
    assert 0 < past < len(SIZES)


@pytest.mark.parametrize("name", ["ep_expert_gemm_bf16", "ep_expert_swiglu_bf16", "ep_expert_gemm_int8",
                                  "ep_expert_swiglu_int8"])
def test_tiles_past_the_launch_limits(ep, name):  # noqa: F811
    """Refused as documented, before anything is launched."""
    gated = "swiglu" in name
    rows = (F, F) if name.endswith("bf16") else (F, F, F, F)
    tail = {"ep_expert_gemm_bf16": (0, F, None), "ep_expert_swiglu_bf16": (F, None, None),
            "ep_expert_gemm_int8": (F, None), "ep_expert_swiglu_int8": (F, F, F, 1 << 62, None)}[name]
    for S, N, E in (((1 << 30) - 1, 1 << 17, 1024), (1 << 29, 8192 if gated else 16384, 1)):
        refused(ep, name, rows + (F, S, N, 64, E) + tail, ep.EP_ERR_LAUNCH, "invalid configuration")
