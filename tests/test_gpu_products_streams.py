"""stream= of the bf16 and int8 expert operators: what a call makes for itself belongs to the stream that its
kernels run on; overlapping calls, captured ones, and the timing hook."""
import pytest
import torch

import test_gpu_products as gpu
from gpu_util import say
from test_gpu_experts import ep, gen, normal  # noqa: F401
from test_gpu_streams import pool_of, tensors

pytestmark = pytest.mark.gpu
NAMES = ["gemm_bf16", "dgrad_bf16", "swiglu_bf16", "quantize", "dispatch", "gemm_int8", "swiglu_int8"]


def calls(ep, seed=7):  # noqa: F811
    """name -> (a call with stream=, whose outputs are all its own)."""
    g = gen(seed)
    T, H, I, E, k = 24, 256, 128, 4, 2
    x, logits = normal(g, T, H), normal(g, T, E, dtype=torch.float32)
    idx, _ = ep.ep_route_topk(logits, k)
    lay = ep.ep_dispatch_layout(idx, E, 2)
    pos, off = lay["pos"], lay["expert_offsets"]
    w13 = gpu.matrices(g, E, 2 * I, H)
    a, gu = ep.ep_dispatch(x, pos), normal(g, T * k, 2 * I)
    q, s = ep.ep_dispatch_int8(x, pos)
    W = ep.ep_quantize_int8(w13)
    return {
        "gemm_bf16": lambda st: ep.ep_expert_gemm_bf16(a, w13, off, stream=st),
        "dgrad_bf16": lambda st: ep.ep_expert_gemm_bf16(gu, w13, off, transposed=True, stream=st),
        "swiglu_bf16": lambda st: ep.ep_expert_swiglu_bf16(a, w13, off, save_gate_up=True, stream=st),
        "quantize": lambda st: ep.ep_quantize_int8(w13, stream=st),
        "dispatch": lambda st: ep.ep_dispatch_int8(x, pos, stream=st),
        "gemm_int8": lambda st: ep.ep_expert_gemm_int8(q, s, *W, off, stream=st),
        "swiglu_int8": lambda st: ep.ep_expert_swiglu_int8(q, s, *W, off, stream=st),
    }


def same(got, want, name):
    got = tensors(got)
    assert len(got) == len(want) > 0
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name


@pytest.mark.parametrize("handle", ["stream", "integer"])
@pytest.mark.parametrize("name", NAMES)
def test_outputs_belong_to_the_calls_stream(ep, name, handle):  # noqa: F811
    call = calls(ep)[name]
    want = [t.clone() for t in tensors(call(None))]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    say(f"{name} on another stream ({handle})")
    got = call(s if handle == "stream" else s.cuda_stream)
    torch.cuda.synchronize()
    assert all(pool_of(t) == s.cuda_stream for t in tensors(got)), name
    same(got, want, name)


@pytest.mark.parametrize("name", NAMES)
def test_null_stream_from_another_current_one(ep, name):  # noqa: F811
    call = calls(ep)[name]
    torch.cuda.synchronize()
    say(f"{name} on the null stream")
    with torch.cuda.stream(torch.cuda.Stream()):
        got = tensors(call(0))
    torch.cuda.synchronize()
    assert got and all(pool_of(t) == 0 for t in got)


def test_own_workspace_belongs_to_the_calls_stream(ep, monkeypatch):  # noqa: F811
    call, seen = calls(ep)["swiglu_int8"], []
    real = ep._scratch

    def scratch(*args):
        seen.append(real(*args))
        return seen[-1]

    monkeypatch.setattr(ep, "_scratch", scratch)
    s = torch.cuda.Stream()
    say("workspace of a call on another stream")
    call(s)
    torch.cuda.synchronize()
    assert len(seen) == 3 and all(pool_of(t) == s.cuda_stream for t in seen)


@pytest.mark.parametrize("name", NAMES)
def test_overlapping_calls(ep, name):  # noqa: F811
    """Calls on two streams at once, each with outputs and workspaces of its own: the same bits as alone."""
    both = [calls(ep, seed)[name] for seed in (1, 2)]
    want = [[t.clone() for t in tensors(c(None))] for c in both]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    say(f"{name} on two streams at once")
    for _ in range(10):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                outs[i].append(both[i](None))
    torch.cuda.synchronize()
    for i in (0, 1):
        for o in outs[i]:
            same(o, want[i], name)


@pytest.mark.parametrize("name", NAMES)
def test_captured_on_a_forked_stream(ep, name):  # noqa: F811
    """A call on a stream that a capture forked to: replays equal the eager results."""
    call = calls(ep)[name]
    want = [t.clone() for t in tensors(call(None))]
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    say(f"{name} captured on a forked stream")
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        got = call(s)
        torch.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        for t in tensors(got):
            t.view(torch.uint8).fill_(0x5A)
        call(None)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        same(got, want, name)


def test_two_graphs_with_one_workspace_in_turn(ep):  # noqa: F811
    """Two captured calls that were given the same workspace, replayed one after the other in both orders."""
    g = gen(11)
    off = torch.tensor([0, 20, 33], dtype=torch.int32, device="cuda")
    ws = torch.empty(ep.ep_expert_swiglu_int8_workspace_bytes(33, 128), dtype=torch.uint8, device="cuda")
    W = ep.ep_quantize_int8(gpu.matrices(g, 2, 256, 128))
    rows = [ep.ep_quantize_int8(normal(g, 33, 128)) for _ in range(2)]
    want = [ep.ep_expert_swiglu_int8(*r, *W, off) for r in rows]
    torch.cuda.synchronize()
    graphs, got = [], []
    say("two graphs, one workspace")
    for r in rows:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(ep.ep_expert_swiglu_int8(*r, *W, off, workspace=ws))
        graphs.append(graph)
    for order in ((0, 1), (1, 0), (1, 1), (0, 0)):
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in set(order):
            for a, b in zip(got[i], want[i]):
                assert torch.equal(a, b), order


@pytest.mark.parametrize("name", NAMES)
def test_timing_events(ep, name):  # noqa: F811
    """The one-shot events bracket all of a call's kernels and no later ones."""
    call = calls(ep)[name]
    call(None)
    torch.cuda.synchronize()
    ev = ep.HipEvents()
    a, b = ev.create(), ev.create()
    say(f"{name} between timing events")
    ep.ep_set_timing_events(a, b)
    call(None)
    ev.synchronize(b)
    first = ev.elapsed_ms(a, b)
    call(None)
    torch.cuda.synchronize()
    assert 0 < first < 50 and ev.elapsed_ms(a, b) == first
    ev.destroy(a)
    ev.destroy(b)
