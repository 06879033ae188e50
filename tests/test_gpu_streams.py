"""stream=: what a call makes for itself belongs to the stream that its kernels run on, so that neither
work pending on the current stream nor a later owner of the memory meets the call."""
import pytest
import torch

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    from combine_ep_route_topk_amd import ep as mod
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    return mod


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def pool_of(t):
    """The raw handle of the stream whose memory holds the tensor."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's memory")


def tensors(v):
    if isinstance(v, torch.Tensor):
        return [v]
    if isinstance(v, dict):
        v = list(v.values())
    return [t for x in v for t in tensors(x)] if isinstance(v, (list, tuple)) else []


def calls(ep):
    """name -> (a call with stream=, whose outputs are all its own): small inputs of every operator."""
    g = gen(7)
    T, H, I, E, k = 24, 256, 128, 4, 2
    x, logits = normal(g, T, H), torch.randn((T, E), generator=g, device=DEV)
    idx, tw = ep.ep_route_topk(logits, k)
    lay = ep.ep_dispatch_layout(idx, E, 2)
    pos, off = lay["pos"], lay["expert_offsets"]
    w13, w2 = normal(g, E, 2 * I, H), normal(g, E, H, I)
    d13, d2 = ep.ep_quantize_weight_fp8(w13), ep.ep_quantize_weight_fp8(w2)
    a, a_s = ep.ep_dispatch_fp8(x, pos)
    gu, dh = normal(g, T * k, 2 * I), normal(g, T * k, I)
    rows = normal(g, 4096, 256)
    y, masks = normal(g, T * k, H), torch.arange(T, device=DEV) % 16
    one = torch.tensor([0, 4096], dtype=torch.int32, device=DEV)
    return {
        "quantize": lambda s: ep.ep_quantize_fp8(x, stream=s),
        "dispatch_fp8": lambda s: ep.ep_dispatch_fp8(x, pos, stream=s),
        "quantize_weight": lambda s: ep.ep_quantize_weight_fp8(w13, transposed=True, stream=s),
        "gemm": lambda s: ep.ep_expert_gemm_fp8(a, a_s, d13["q"], d13["scale"], off, stream=s),
        "swiglu": lambda s: ep.ep_expert_swiglu_fp8(a, a_s, d13["q"], d13["scale"], off,
                                                    save_gate_up=True, stream=s),
        "swiglu_grad": lambda s: ep.ep_swiglu_grad(dh, gu, stream=s),
        "wgrad": lambda s: ep.ep_expert_wgrad(gu, a.view(torch.uint8).to(torch.bfloat16), off, stream=s),
        "wgrad_parts": lambda s: ep.ep_expert_wgrad(rows, rows, one, stream=s),
        "moe_tokens": lambda s: ep.ep_moe_tokens(x, idx, tw, w13, w2, stream=s),
        "moe_tokens_fp8": lambda s: ep.ep_moe_tokens(x, idx, tw, d13["q"], d2["q"], d13["scale"],
                                                     d2["scale"], stream=s),
        "route": lambda s: ep.ep_route_topk(logits, k, stream=s),
        "layout": lambda s: ep.ep_dispatch_layout(idx, E, 2, stream=s),
        "dispatch": lambda s: ep.ep_dispatch(x, pos, stream=s),
        "combine": lambda s: ep.ep_combine(y, pos, tw, stream=s),
        "combine_grad": lambda s: ep.ep_combine_grad(x, y, pos, tw, stream=s),
        "dispatch_grad": lambda s: ep.ep_dispatch_grad(y, pos, stream=s),
        "fused": lambda s: ep.ep_fused_dispatch_combine(x, idx, tw, E, 2, stream=s),
        "slices": lambda s: ep.ep_expert_slices(off, 3, stream=s),
        "coalesce": lambda s: ep.ep_rank_coalesce(idx, E, 2, stream=s),
        "expand": lambda s: ep.ep_expand_records(x, masks, E, T * E, stream=s),
    }


def known(v):
    """Without what a call leaves undefined in part: workspaces, row tails, rows behind the last."""
    if not isinstance(v, dict):
        return tensors(v)
    return [t for n, t in v.items()
            if n not in ("workspace", "send_rows", "row_src", "row_experts", "recv")]


NAMES = ["quantize", "dispatch_fp8", "quantize_weight", "gemm", "swiglu", "swiglu_grad", "wgrad",
         "wgrad_parts", "moe_tokens", "moe_tokens_fp8"]
EARLIER = ["route", "layout", "dispatch", "combine", "combine_grad", "dispatch_grad", "fused", "slices",
           "coalesce", "expand"]


@pytest.mark.parametrize("handle", ["stream", "integer"])
@pytest.mark.parametrize("name", NAMES + EARLIER)
def test_outputs_belong_to_the_calls_stream(ep, name, handle):
    call = calls(ep)[name]
    want = [t.clone() for t in known(call(None))]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    say(f"{name} on another stream ({handle})")
    got = call(s if handle == "stream" else s.cuda_stream)
    torch.cuda.synchronize()
    assert all(pool_of(t) == s.cuda_stream for t in tensors(got)), name
    assert len(known(got)) == len(want) > 0
    for a, b in zip(known(got), want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name


@pytest.mark.parametrize("name", NAMES + EARLIER)
def test_null_stream_from_another_current_one(ep, name):
    call = calls(ep)[name]
    torch.cuda.synchronize()
    say(f"{name} on the null stream")
    with torch.cuda.stream(torch.cuda.Stream()):
        got = tensors(call(0))
    torch.cuda.synchronize()
    assert got and all(pool_of(t) == 0 for t in got)


@pytest.mark.parametrize("name", ["gemm", "moe_tokens", "swiglu_grad", "quantize", "dispatch", "combine",
                                  "dispatch_grad", "route"])
def test_pending_work_of_the_current_stream(ep, name):
    """A block that a write still waits for on the current stream, dropped by its owner, is not handed
    to a call on another stream."""
    call = calls(ep)[name]
    want = [t.clone() for t in tensors(call(None))]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    say(f"{name} beside pending writes")
    blocks = [torch.empty(t.numel() * t.element_size(), dtype=torch.uint8, device=DEV) for t in want]
    torch.cuda._sleep(20_000_000)
    for b in blocks:
        b.fill_(0x5A)
    del blocks, b
    got = tensors(call(s))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name


@pytest.mark.parametrize("name", ["gemm", "moe_tokens", "swiglu_grad", "quantize", "layout", "dispatch", "fused",
                                  "combine"])
def test_dropped_outputs_wait_for_their_reader(ep, name):
    """Results read by work that is pending on the current stream and dropped: the call's stream does not
    get their memory before that work is done."""
    call = calls(ep)[name]
    want = [t.clone() for t in known(call(None))]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    say(f"{name} dropped beside pending reads")
    got = call(s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(20_000_000)
    mine = [t.clone() for t in known(got)]
    sizes = [t.numel() * t.element_size() for t in tensors(got)]
    del got
    with torch.cuda.stream(s):
        blocks = [torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV) for n in sizes]
    torch.cuda.synchronize()
    for a, b in zip(mine, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
    del blocks


@pytest.mark.parametrize("name", ["gemm", "moe_tokens", "wgrad_parts", "layout"])
def test_captured_on_a_forked_stream(ep, name):
    """A call on a stream that a capture forked to: replays equal the eager results."""
    call = calls(ep)[name]
    want = [t.clone() for t in known(call(None))]
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    say(f"{name} captured on a forked stream")
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        got = call(s)
        torch.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        for t in known(got):
            t.view(torch.uint8).fill_(0x5A)
        call(None)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(known(got), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
