"""The library's choice of kernel for given sizes (csrc/experts/expert_choice.h), compiled for the host:
tests use it to know that their sizes reach the kernel they are for."""
import ctypes
import functools
import os
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "combine_ep_route_topk_amd", "csrc", "experts", "expert_choice.h")
GEMM = ["large", "128x256", "64x256", "32x256", "128x128", "64x128", "32x64"]
CUS = 256

SHIM = f"""
#include "{HEADER}"
extern "C" int gemm(long long S, long long N, long long E, int gated, long long cus) {{
    return ep::choose_gemm(S, N, E, gated != 0, cus);
}}
extern "C" int wgrad_is_large(int S, int N, int K, int E) {{ return ep::wgrad_large(S, N, K, E); }}
extern "C" int wgrad_parts(int S, int N, int K, int E) {{ return ep::wgrad_parts(S, N, K, E); }}
"""


@functools.lru_cache(maxsize=None)
def _lib():
    with tempfile.TemporaryDirectory() as d:
        src, lib = os.path.join(d, "shim.cpp"), os.path.join(d, "shim.so")
        with open(src, "w") as f:
            f.write(SHIM)
        subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-Werror", "-o", lib, src],
                       check=True)
        h = ctypes.CDLL(lib)
    h.gemm.argtypes = [ctypes.c_longlong] * 3 + [ctypes.c_int, ctypes.c_longlong]
    return h


def gemm(S, N, E, gated=False):
    """N: rows of one expert's weights (2 I when gated)."""
    return GEMM[_lib().gemm(S, N, E, int(gated), CUS)]


def wgrad(S, N, K, E):
    """'large', or the parts that the small tiles split the rows into."""
    return "large" if _lib().wgrad_is_large(S, N, K, E) else _lib().wgrad_parts(S, N, K, E)
