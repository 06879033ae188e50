"""The bf16 and int8 expert operators refuse bad arguments synchronously, without a GPU: no call here reaches a
launch.  And their workspace query, and the Python binding's own checks."""
import ctypes

import pytest
import torch

from test_experts_refusals import F, ODD, P, ep, refused  # noqa: F401

OFF4 = P(0x10002)        # not 4-byte aligned


def test_quantize(ep):  # noqa: F811
    bad, big = ep.EP_ERR_INVALID_ARG, ep.EP_ERR_UNSUPPORTED
    refused(ep, "ep_quantize_int8", (F, -1, 16, F, F, None), bad, "S=-1")
    refused(ep, "ep_quantize_int8", (F, 4, 24, F, F, None), bad, "H=24")
    refused(ep, "ep_quantize_int8", (F, 4, 0, F, F, None), bad, "H=0")
    refused(ep, "ep_quantize_int8", (F, 4, 1 << 21, F, F, None), big, "H=")
    refused(ep, "ep_quantize_int8", (F, 1 << 30, 16, F, F, None), big, "T*k")
    refused(ep, "ep_quantize_int8", (None, 4, 16, F, F, None), bad, "x is NULL")
    refused(ep, "ep_quantize_int8", (F, 4, 16, ODD, F, None), bad, "aligned")
    refused(ep, "ep_quantize_int8", (F, 4, 16, F, OFF4, None), bad, "scale")
    refused(ep, "ep_quantize_int8", (F, 4, 16, F, None, None), bad, "scale")
    refused(ep, "ep_dispatch_int8", (F, 0, 16, 2, F, F, F, None), bad, "T=0")
    refused(ep, "ep_dispatch_int8", (F, 4, 16, 0, F, F, F, None), bad, "k=0")
    refused(ep, "ep_dispatch_int8", (F, 4, 16, 65, F, F, F, None), big, "k=65")
    refused(ep, "ep_dispatch_int8", (F, 1 << 28, 16, 8, F, F, F, None), big, "T*k")
    refused(ep, "ep_dispatch_int8", (F, 4, 16, 2, None, F, F, None), bad, "pos")
    refused(ep, "ep_dispatch_int8", (F, 4, 16, 2, F, F, None, None), bad, "scale")
    assert ep.library().ep_quantize_int8(None, 0, 16, None, None, None) == ep.EP_OK


CALLS = {      # name -> (arguments around S, N, K, E, those behind, the step of N and K)
    "ep_expert_gemm_bf16": (2, 0, (0, F, None), 8),
    "ep_expert_swiglu_bf16": (2, 0, (F, None, None), 8),
    "ep_expert_gemm_int8": (4, 1, (F, None), 16),
    "ep_expert_swiglu_int8": (4, 1, (F, F, F, 1 << 40, None), 16),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_products(ep, name):  # noqa: F811
    bad, big = ep.EP_ERR_INVALID_ARG, ep.EP_ERR_UNSUPPORTED
    ops, _, tail, step = CALLS[name]

    def args(S=8, N=128, K=64, E=2, a=F, w=F, offsets=F, tail=tail):
        rows = (a, w) if ops == 2 else (a, F, w, F)
        return rows + (offsets, S, N, K, E) + tail

    refused(ep, name, args(S=-1), bad, "S=-1")
    refused(ep, name, args(S=1 << 30), big, "S=")
    refused(ep, name, args(E=0), bad, "E=0")
    refused(ep, name, args(E=1025), big, "E=1025")
    refused(ep, name, args(N=step // 2), bad, f"={step // 2}")
    refused(ep, name, args(N=128 + step // 2), bad, f"={128 + step // 2}")
    refused(ep, name, args(K=64 + step // 2), bad, f"K={64 + step // 2}")
    refused(ep, name, args(K=0), bad, "K=0")
    refused(ep, name, args(K=1 << 18), big, "2^17")
    refused(ep, name, args(N=1 << 18), big, "2^17")
    refused(ep, name, args(a=None), bad, "a is NULL")
    refused(ep, name, args(a=ODD), bad, "aligned")
    refused(ep, name, args(w=None), bad, "NULL")
    refused(ep, name, args(w=ODD), bad, "aligned")
    refused(ep, name, args(offsets=None), bad, "expert_offsets")
    for i, v in enumerate(tail):
        if v is F:
            refused(ep, name, args(tail=tail[:i] + (None,) + tail[i + 1:]), bad, "NULL")
    # no rows: nothing to do, and the row buffers may be NULL
    lib = ep.library()
    none = tuple(None if v is F else v for v in tail)
    assert getattr(lib, name)(*args(S=0, a=None, tail=none)) == ep.EP_OK


def test_int8_alone(ep):  # noqa: F811
    bad, big = ep.EP_ERR_INVALID_ARG, ep.EP_ERR_UNSUPPORTED
    tails = {"ep_expert_gemm_int8": (F, None), "ep_expert_swiglu_int8": (F, F, F, 1 << 40, None)}
    for name, tail in tails.items():
        refused(ep, name, (F, F, F, F, F, 8, 128, 1 << 17, 2) + tail, big, "K=131072")
        refused(ep, name, (F, None, F, F, F, 8, 128, 64, 2) + tail, bad, "a_scale")
        refused(ep, name, (F, OFF4, F, F, F, 8, 128, 64, 2) + tail, bad, "a_scale")
        refused(ep, name, (F, F, F, ODD, F, 8, 128, 64, 2) + tail, bad, "_scale")
    refused(ep, "ep_expert_swiglu_int8", (F, F, F, F, F, 8, 128, 64, 2, F, F, P(0x10010), 1 << 40, None),
            bad, "workspace")
    need = ep.ep_expert_swiglu_int8_workspace_bytes(8, 128)
    assert need == 8 * 128 * 2
    refused(ep, "ep_expert_swiglu_int8", (F, F, F, F, F, 8, 128, 64, 2, F, F, F, need - 1, None),
            ep.EP_ERR_WORKSPACE, "needs")
    size = ep.ep_expert_swiglu_int8_workspace_bytes
    assert size(0, 128) == size(-1, 128) == size(5, 0) == 0
    assert size((1 << 30) - 1, 1 << 17) == ((1 << 30) - 1) * 2 ** 18


def test_gate_up_alignment(ep):  # noqa: F811
    refused(ep, "ep_expert_swiglu_bf16", (F, F, F, 8, 128, 64, 2, F, ODD, None), ep.EP_ERR_INVALID_ARG,
            "gate_up")


def test_binding(ep):  # noqa: F811
    """Shapes, types and places, before the library is called."""
    bf, i8, f = torch.bfloat16, torch.int8, torch.float32
    t = lambda *s, d=bf: torch.zeros(s, dtype=d)  # noqa: E731
    off = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: ep.ep_expert_gemm_bf16(t(4, 64), t(2, 16, 64), off),
                 lambda: ep.ep_expert_swiglu_bf16(t(4, 64), t(2, 16, 64), off),
                 lambda: ep.ep_quantize_int8(t(4, 64)),
                 lambda: ep.ep_dispatch_int8(t(4, 64), torch.zeros(4, 2, dtype=torch.int32)),
                 lambda: ep.ep_expert_gemm_int8(t(4, 64, d=i8), t(4, d=f), t(2, 16, 64, d=i8),
                                                t(2, 16, d=f), off)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(ValueError, match="3 dimensions"):
        ep.ep_expert_gemm_bf16(_gpu_like(t(4, 64)), t(16, 64), off)
    with pytest.raises(TypeError, match="bf16"):
        ep.ep_expert_gemm_bf16(t(4, 64, d=f), t(2, 16, 64), off)
    with pytest.raises(ValueError, match="2 dimensions"):
        ep.ep_quantize_int8(t(64))
    with pytest.raises(TypeError, match="torch.Tensor"):
        ep.ep_quantize_int8([1.0])


def _gpu_like(tensor):
    """A tensor that passes the check of its place (the next argument's is what fails)."""
    class Placed(torch.Tensor):
        is_cuda = property(lambda self: True)

        @staticmethod
        def __new__(cls, v):
            return v.as_subclass(cls)
    return Placed(tensor)


def test_sizes_past_the_abi(ep):  # noqa: F811
    """Sizes are 32 bits in C: larger ones are refused before they are cut."""
    def many(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="meta")

    few = many(2, 16, 16)
    for call in (lambda: ep.ep_quantize_int8(many((1 << 32) + 4, 16)),
                 lambda: ep.ep_quantize_int8(many(1 << 12, 1 << 20, 16)),
                 lambda: ep.ep_dispatch_int8(many((1 << 32) + 4, 16), many(4, 2, dtype=torch.int32)),
                 lambda: ep.ep_expert_gemm_bf16(many((1 << 32) + 4, 16), few, many(3, dtype=torch.int32)),
                 lambda: ep.ep_expert_swiglu_bf16(many((1 << 32) + 4, 16), few, many(3, dtype=torch.int32)),
                 lambda: ep.ep_expert_gemm_int8(many((1 << 32) + 4, 16, dtype=torch.int8), None, few, None, None)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()
