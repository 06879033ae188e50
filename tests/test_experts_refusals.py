"""The expert operators refuse bad arguments synchronously, without a GPU: no call here reaches a
launch.  And their workspace query."""
import ctypes

import pytest

P = ctypes.c_void_p
F = P(0x10000)          # aligned, never dereferenced: validation fails first
ODD = P(0x10004)


@pytest.fixture(scope="module")
def ep():
    from combine_ep_route_topk_amd import ep as mod
    return mod


def refused(ep, name, args, status, text=""):
    lib = ep.library()
    rc = getattr(lib, name)(*args)
    assert rc == status, (name, rc, lib.ep_last_error())
    assert text in lib.ep_last_error().decode(), lib.ep_last_error()


def test_quantize(ep):
    bad, big = ep.EP_ERR_INVALID_ARG, ep.EP_ERR_UNSUPPORTED
    refused(ep, "ep_quantize_fp8", (F, -1, 16, F, F, None), bad, "S=-1")
    refused(ep, "ep_quantize_fp8", (F, 4, 24, F, F, None), bad, "H=24")
    refused(ep, "ep_quantize_fp8", (F, 4, 1 << 21, F, F, None), big, "H=")
    refused(ep, "ep_quantize_fp8", (None, 4, 16, F, F, None), bad, "NULL")
    refused(ep, "ep_quantize_fp8", (F, 4, 16, ODD, F, None), bad, "aligned")
    refused(ep, "ep_quantize_fp8", (F, 4, 16, F, None, None), bad, "scale")
    refused(ep, "ep_dispatch_fp8", (F, 0, 16, 2, F, F, F, None), bad, "T=0")
    refused(ep, "ep_dispatch_fp8", (F, 4, 16, 0, F, F, F, None), bad, "k=0")
    refused(ep, "ep_dispatch_fp8", (F, 4, 16, 65, F, F, F, None), big, "k=65")
    refused(ep, "ep_dispatch_fp8", (F, 1 << 28, 16, 8, F, F, F, None), big, "T*k")
    refused(ep, "ep_dispatch_fp8", (F, 4, 16, 2, None, F, F, None), bad, "pos")
    refused(ep, "ep_quantize_weight_fp8", (F, 0, 16, 16, F, F, None, None, None), bad, "E=0")
    refused(ep, "ep_quantize_weight_fp8", (F, 2, 20, 16, F, F, None, None, None), bad, "N=20")
    refused(ep, "ep_quantize_weight_fp8", (F, 2, 16, 16, F, F, F, None, None), bad, "together")
    refused(ep, "ep_quantize_weight_fp8", (F, 2, 16, 16, F, F, ODD, F, None), bad, "aligned")


@pytest.mark.parametrize("name", ["ep_expert_gemm_fp8", "ep_expert_swiglu_fp8"])
def test_products(ep, name):
    bad, big = ep.EP_ERR_INVALID_ARG, ep.EP_ERR_UNSUPPORTED
    tail = (F, None) if name == "ep_expert_gemm_fp8" else (F, F, None, None)

    def args(S=8, N=128, K=64, E=2, a=F, offsets=F):
        return (a, F, F, F, offsets, S, N, K, E) + tail

    refused(ep, name, args(S=-1), bad, "S=-1")
    refused(ep, name, args(S=1 << 30), big, "S=")
    refused(ep, name, args(E=0), bad, "E=0")
    refused(ep, name, args(E=1025), big, "E=1025")
    refused(ep, name, args(N=120), bad, "=120")
    refused(ep, name, args(K=8), bad, "K=8")
    refused(ep, name, args(K=1 << 18), big, "2^17")
    refused(ep, name, args(a=None), bad, "NULL")
    refused(ep, name, args(a=ODD), bad, "aligned")
    refused(ep, name, args(offsets=None), bad, "expert_offsets")
    # no rows: nothing to do, and the row buffers may be NULL
    lib = ep.library()
    none = (None, None, F, F, F, 0, 128, 64, 2) + ((None, None) if len(tail) == 2 else (None,) * 4)
    assert getattr(lib, name)(*none) == ep.EP_OK


def test_swiglu_blocks(ep):
    refused(ep, "ep_expert_swiglu_fp8", (F, F, F, F, F, 8, 80, 64, 2, F, F, None, None),
            ep.EP_ERR_INVALID_ARG, "multiple of 128")
    refused(ep, "ep_expert_swiglu_fp8",
            (F, F, F, F, F, 8, 1 << 15, 1 << 16, 2, F, F, None, None), ep.EP_ERR_UNSUPPORTED, "2^31")
    refused(ep, "ep_expert_swiglu_fp8", (F, F, F, F, F, 8, 128, 64, 2, F, F, ODD, None),
            ep.EP_ERR_INVALID_ARG, "gate_up")


def test_gradients(ep):
    bad = ep.EP_ERR_INVALID_ARG
    refused(ep, "ep_swiglu_grad", (F, F, 4, 12, F, F, None), bad, "I=12")
    refused(ep, "ep_swiglu_grad", (F, F, 4, 16, None, F, None), bad, "grad_gate_up")
    refused(ep, "ep_swiglu_grad", (F, F, 4, 16, F, ODD, None), bad, "aligned")
    assert ep.library().ep_swiglu_grad(None, None, 0, 16, None, None, None) == ep.EP_OK
    refused(ep, "ep_expert_wgrad", (F, F, F, 4, 12, 16, 2, 0, F, None, 0, None), bad, "N=12")
    refused(ep, "ep_expert_wgrad", (F, F, F, 4, 16, 16, 2, 0, None, None, 0, None), bad, "grad_w")
    refused(ep, "ep_expert_wgrad", (None, F, F, 4, 16, 16, 2, 0, F, None, 0, None), bad, "grad_y")
    refused(ep, "ep_expert_wgrad", (F, F, None, 4, 16, 16, 2, 0, F, None, 0, None), bad, "expert_offsets")


def test_wgrad_workspace(ep):
    query = ep.library().ep_expert_wgrad_workspace_bytes
    assert query(32768, 4096, 7168, 8) == 0          # many tiles: not split
    assert query(100, 256, 512, 1) == 0              # few rows
    need = query(32768, 256, 512, 1)
    assert need > 0 and need % (256 * 512 * 4) == 0
    assert query(0, 256, 512, 1) == 0
    args = lambda ws, n: (F, F, F, 32768, 256, 512, 1, 0, F, ws, n, None)  # noqa: E731
    refused(ep, "ep_expert_wgrad", args(F, need - 1), ep.EP_ERR_WORKSPACE, "needs")
    refused(ep, "ep_expert_wgrad", args(P(0x10010), need), ep.EP_ERR_INVALID_ARG, "256")


def test_moe_tokens(ep):
    bad, big = ep.EP_ERR_INVALID_ARG, ep.EP_ERR_UNSUPPORTED
    lib = ep.library()
    need = lib.ep_moe_tokens_workspace_bytes(8, 2, 128)
    assert need >= 2 * 2 * 8 * 2 * 128 and need % 256 == 0
    assert lib.ep_moe_tokens_workspace_bytes(65, 2, 128) == 0
    assert lib.ep_moe_tokens_workspace_bytes(8, 0, 128) == 0

    def args(T=8, H=64, I=128, E=4, k=2, s13=F, s2=F, ws=F, nbytes=need, x=F):
        return (x, F, F, T, H, I, E, k, F, s13, F, s2, F, ws, nbytes, None)

    refused(ep, "ep_moe_tokens", args(T=0), bad, "T=0")
    refused(ep, "ep_moe_tokens", args(T=65), big, "T=65")
    refused(ep, "ep_moe_tokens", args(H=24), bad, "H=24")
    refused(ep, "ep_moe_tokens", args(I=80), bad, "I=80")
    refused(ep, "ep_moe_tokens", args(k=5), bad, "k=5")
    refused(ep, "ep_moe_tokens", args(s2=None), bad, "together")
    refused(ep, "ep_moe_tokens", args(x=None), bad, "NULL")
    refused(ep, "ep_moe_tokens", args(ws=P(0x10080)), bad, "256")
    refused(ep, "ep_moe_tokens", args(nbytes=need - 1), ep.EP_ERR_WORKSPACE, "needs")


def test_binding(ep):
    import torch
    x = torch.zeros((4, 32), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        ep.ep_quantize_fp8(x)
    with pytest.raises(TypeError, match="bf16"):
        ep.ep_quantize_fp8(x.float())
    with pytest.raises(ValueError, match="dimensions"):
        ep.ep_quantize_fp8(x[0])
    with pytest.raises(ValueError, match="GPU"):
        ep.ep_moe_tokens(x, torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2)),
                         torch.zeros((2, 64, 32), dtype=torch.bfloat16),
                         torch.zeros((2, 32, 32), dtype=torch.bfloat16))
