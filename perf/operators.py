"""Cases of the expert operators: FP8 dispatch, the experts' block-scaled products, their gradients
and the whole layer for a few tokens.

An 8-bit tensor here is e4m3 values with one power-of-two scale (a byte b standing for 2^(b - 127))
for each 128 values of a row, or for each 128 x 128 block of a weight matrix.  A block's scale is the
least power of two that brings its largest magnitude to 448 or less.  The experts' rows lie in one
buffer, expert after expert, as the dispatch layout orders them; `offsets` [E + 1] bounds them.

  dispatch_fp8  x [T][H] -> quantised rows at pos[t][j], and their scales
  expert_gemm   y[s] = W[e(s)] a[s]                        (forward; an input gradient with W transposed)
  expert_ffn    y[s] = W2[e] q(silu(G) * U), [G; U] = W13[e] a[s], q the quantiser
  expert_wgrad  dW[e] = sum over the rows s of e of dy[s] x[s]^T
  swiglu_grad   of h = silu(g) * u: dg, du and h, from dh and the saved [g; u]
  moe_tokens    out[t] = sum_j w[t][j] W2[e] (silu(G) * U), [G; U] = W13[e] x[t], e = idx[t][j]
"""
import math

import torch

own = False     # True: run() calls the framework; False: run() computes the plain forms

DEV = "cuda:0"
BLOCK = 128
E4M3_MAX = 448.0


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's 128 tokens going out to 256 experts: latency
        dict(name="dispatch_fp8_decode", op="dispatch_fp8", T=128, H=7168, E=256, k=8),
        # a prefill batch of 4096 tokens: half the bytes of the bf16 dispatch
        dict(name="dispatch_fp8_prefill", op="dispatch_fp8", T=4096, H=7168, E=256, k=8),
        # a decode step on one rank's 8 experts: a few rows each, the weights' bytes bound it
        dict(name="expert_gemm_decode", op="expert_gemm", S=256, N=4096, K=7168, E=8, rows="zipf"),
        # a training step's input gradient: 32768 rows against the transposed gate/up weights
        dict(name="expert_gemm_dgrad", op="expert_gemm", S=32768, N=7168, K=4096, E=8, rows="even"),
        # a small ragged batch through narrow experts, one in four without rows, gate_up kept for training
        dict(name="expert_ffn_ragged", op="expert_ffn", S=1000, H=4096, I=1408, E=16, rows="gaps", save=True),
        # a prefill batch (4096 tokens, top-8) through 8 local experts
        dict(name="expert_ffn_prefill", op="expert_ffn", S=32768, H=7168, I=2048, E=8, rows="even", save=False),
        # weight gradients of 16 narrow experts from a short micro-batch
        dict(name="expert_wgrad_short", op="expert_wgrad", S=2000, N=2816, K=4096, E=16, rows="gaps"),
        # weight gradients of 8 gate/up matrices from a full batch
        dict(name="expert_wgrad_train", op="expert_wgrad", S=32768, N=4096, K=7168, E=8, rows="even"),
        # the gated activation's gradient for a short and for a full batch
        dict(name="swiglu_grad_short", op="swiglu_grad", S=1000, I=1408),
        dict(name="swiglu_grad_train", op="swiglu_grad", S=32768, I=2048),
        # one user's token through 8 of 64 experts with 8-bit weights
        dict(name="moe_one_token", op="moe_tokens", T=1, H=7168, I=2048, E=64, k=8, fp8=True),
        # 32 users' tokens through 128 narrow experts with bf16 weights: nearly all are read
        dict(name="moe_32_tokens", op="moe_tokens", T=32, H=4096, I=1408, E=128, k=8, fp8=False),
    ]


def draw(rng):
    def size(lo, hi, step=1):
        return max(1, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step

    op = rng.choice(["dispatch_fp8", "expert_gemm", "expert_ffn", "expert_wgrad", "swiglu_grad",
                     "moe_tokens"])
    if op == "dispatch_fp8":
        E = rng.choice([8, 33, 64, 128, 256])
        return dict(op=op, T=size(1, 8192), H=size(64, 8192, 16), E=E, k=rng.randint(1, 8))
    if op == "swiglu_grad":
        return dict(op=op, S=size(1, 32768), I=size(64, 2048, 8))
    if op == "moe_tokens":
        fp8 = rng.random() < 0.5
        E = rng.randint(8, 96)
        return dict(op=op, T=size(1, 64), H=size(256, 7168, 16),
                    I=size(128, 2048, 128) if fp8 else size(64, 2048, 16), E=E,
                    k=rng.randint(1, 8), fp8=fp8)
    rows = rng.choice(["even", "zipf", "gaps"])
    E, S = rng.randint(1, 32), size(1, 32768)
    if op == "expert_ffn":
        return dict(op=op, S=S, H=size(256, 7168, 16), I=size(128, 2048, 128), E=E, rows=rows,
                    save=rng.random() < 0.5)
    return dict(op=op, S=S, N=size(64, 7168, 16), K=size(64, 4096, 16), E=E, rows=rows)


def work(case):
    c = case
    blocks = lambda n: -(-n // BLOCK)  # noqa: E731
    if c["op"] == "dispatch_fp8":
        T, H, k = c["T"], c["H"], c["k"]
        return {"bytes": 2 * T * H + 4 * T * k + T * k * (H + blocks(H)), "flops": 4 * T * H}
    if c["op"] == "expert_gemm":
        S, N, K, E = c["S"], c["N"], c["K"], _used(c)
        return {"bytes": S * (K + blocks(K) + 2 * N) + E * (N * K + blocks(N) * blocks(K)),
                "flops": 2 * S * N * K}
    if c["op"] == "expert_ffn":
        S, H, I, E = c["S"], c["H"], c["I"], _used(c)
        return {"bytes": S * (H + blocks(H) + 2 * H + (4 * I if c["save"] else 0)) + E * 3 * I * H,
                "flops": 6 * S * H * I}
    if c["op"] == "expert_wgrad":
        S, N, K, E = c["S"], c["N"], c["K"], c["E"]
        return {"bytes": 2 * S * (N + K) + 4 * E * N * K, "flops": 2 * S * N * K}
    if c["op"] == "swiglu_grad":
        return {"bytes": 2 * c["S"] * c["I"] * 6, "flops": 12 * c["S"] * c["I"]}
    T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
    read = E * (1.0 - (1.0 - k / E) ** T)       # experts that T tokens of k picks reach, expected
    return {"bytes": int(read * 3 * I * H * (1 if c["fp8"] else 2)) + 4 * T * H + 8 * T * k,
            "flops": 6 * T * k * I * H}


def _used(c):
    """Experts that have rows, as _counts spreads them."""
    return min(c["S"], c["E"] - c["E"] // 4 if c["rows"] == "gaps" else c["E"])


# --------------------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _quantize(x):
    """x [..., n] -> e4m3 values [..., n] and scale bytes [..., ceil(n / 128)], block by block."""
    n = x.shape[-1]
    nb = -(-n // BLOCK)
    v = x.float()
    if nb * BLOCK != n:
        v = torch.cat([v, v.new_zeros(*v.shape[:-1], nb * BLOCK - n)], -1)
    v = v.view(*v.shape[:-1], nb, BLOCK)
    scale = _scale_of(v.abs().amax(-1))
    q = (v / scale.unsqueeze(-1)).view(*v.shape[:-2], nb * BLOCK)[..., :n]
    return q.to(torch.float8_e4m3fn), _scale_byte(scale)


def _scale_of(amax):
    """The least power of two s with amax / s <= 448 (1 for a block of zeros)."""
    m, e = torch.frexp(amax)                    # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.clamp(torch.where(m <= 0.875, e - 9, e - 8), min=-126)
    s = torch.ldexp(torch.ones_like(amax), e)
    return torch.where(amax == 0, torch.ones_like(s), s)


def _scale_byte(scale):
    return (torch.frexp(scale)[1] + 126).to(torch.uint8)


def _quantize_weight(w):
    """w [n][k] -> e4m3 values [n][k] and scale bytes [ceil(n / 128)][ceil(k / 128)]."""
    n, k = w.shape
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    v = w.new_zeros(nb * BLOCK, kb * BLOCK)
    v[:n, :k] = w
    v = v.view(nb, BLOCK, kb, BLOCK)
    scale = _scale_of(v.abs().amax((1, 3)))
    q = (v / scale[:, None, :, None]).view(nb * BLOCK, kb * BLOCK)[:n, :k]
    return q.to(torch.float8_e4m3fn).contiguous(), _scale_byte(scale)


def _weights(g, E, n, k):
    """E quantised matrices with the spread of a trained layer's weights."""
    q = torch.empty(E, n, k, dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.empty(E, -(-n // BLOCK), -(-k // BLOCK), dtype=torch.uint8, device=DEV)
    for e in range(E):
        q[e], s[e] = _quantize_weight(_normal(g, n, k) * (1.0 / math.sqrt(k)))
    return q, s


def _tokens(g, n, h):
    """Activations: normal values, rows of different size."""
    return (_normal(g, n, h) * torch.exp(0.3 * _normal(g, n, 1))).to(torch.bfloat16)


def _counts(case, seed):
    """Rows of each expert (host): S picks drawn evenly, by a Zipf law, or with a quarter of the
    experts left out."""
    S, E = case["S"], case["E"]
    g = torch.Generator().manual_seed(int(seed) + 7)
    p = torch.ones(E)
    if case["rows"] == "zipf":
        p = 1.0 / torch.arange(1, E + 1).float()
        p = p[torch.randperm(E, generator=g)]
    elif case["rows"] == "gaps":
        p[torch.randperm(E, generator=g)[:E // 4]] = 0.0
    picks = torch.multinomial(p, S, replacement=True, generator=g)
    return torch.bincount(picks, minlength=E)


def _segments(case, seed):
    """The experts' row ranges: `offsets` on the GPU as the dispatch layout gives them, and the same
    plan for padded batches: row of (expert, i), and which of these are real."""
    n = _counts(case, seed)
    ends = torch.cumsum(n, 0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    i = torch.arange(int(n.max()))
    real = i[None, :] < n[:, None]
    row = torch.where(real, offsets[:-1, None] + i[None, :], torch.zeros_like(i)[None, :])
    return dict(offsets=offsets.to(torch.int32).to(DEV), row=row.to(DEV), real=real.to(DEV))


def _picks(g, T, E, k):
    """k different experts for each token, and routing weights that sum to 1."""
    logits = _normal(g, T, E)
    top, idx = torch.topk(logits, k, dim=1)
    return idx.to(torch.int32), torch.softmax(top, 1)


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    if op == "dispatch_fp8":
        T, H, E, k = case["T"], case["H"], case["E"], case["k"]
        idx, _ = _picks(g, T, E, min(k, E))
        order = torch.argsort(idx.reshape(-1), stable=True)     # row -> pick
        pos = torch.empty_like(order)
        pos[order] = torch.arange(T * k, device=DEV)
        return dict(op=op, x=_tokens(g, T, H), pos=pos.view(T, k).to(torch.int32),
                    token=order // k)
    if op == "expert_gemm":
        a, a_scale = _quantize(_tokens(g, case["S"], case["K"]))
        w, w_scale = _weights(g, case["E"], case["N"], case["K"])
        return dict(op=op, a=a, a_scale=a_scale, w=w, w_scale=w_scale, **_segments(case, seed))
    if op == "expert_ffn":
        S, H, I, E = case["S"], case["H"], case["I"], case["E"]
        a, a_scale = _quantize(_tokens(g, S, H))
        w13, w13_scale = _weights(g, E, 2 * I, H)
        w2, w2_scale = _weights(g, E, H, I)
        return dict(op=op, a=a, a_scale=a_scale, w13=w13, w13_scale=w13_scale, w2=w2,
                    w2_scale=w2_scale, save=case["save"], **_segments(case, seed))
    if op == "expert_wgrad":
        return dict(op=op, dy=_tokens(g, case["S"], case["N"]), x=_tokens(g, case["S"], case["K"]),
                    **_segments(case, seed))
    if op == "swiglu_grad":
        return dict(op=op, dh=_tokens(g, case["S"], case["I"]),
                    gate_up=_tokens(g, case["S"], 2 * case["I"]))
    T, H, I, E, k = case["T"], case["H"], case["I"], case["E"], case["k"]
    idx, w = _picks(g, T, E, k)
    st = dict(op=op, x=_tokens(g, T, H), idx=idx, w=w)
    if case["fp8"]:
        st["w13"], st["w13_scale"] = _weights(g, E, 2 * I, H)
        st["w2"], st["w2_scale"] = _weights(g, E, H, I)
    else:
        st["w13"] = (_normal(g, E, 2 * I, H) * (1.0 / math.sqrt(H))).to(torch.bfloat16)
        st["w2"] = (_normal(g, E, H, I) * (1.0 / math.sqrt(I))).to(torch.bfloat16)
        st["w13_scale"] = st["w2_scale"] = None
    return st


# --------------------------------------------------------------------------- plain forms, in 32 bits
def _scale_value(byte):
    return torch.ldexp(torch.ones_like(byte, dtype=torch.float32), byte.to(torch.int32) - 127)


def _values(q, byte):
    """Rows' e4m3 values times their blocks' scales, f32."""
    s = _scale_value(byte).repeat_interleave(BLOCK, -1)
    return q.float() * s[..., :q.shape[-1]]


def _weight_values(w, byte):
    """[E][n][k] values in f32: e4m3 times the blocks' scales, or bf16 as it is."""
    if byte is None:
        return w.float()
    s = _scale_value(byte).repeat_interleave(BLOCK, -1)[..., :w.shape[-1]]
    return w.float() * s.repeat_interleave(BLOCK, -2)[..., :w.shape[-2], :]


def _grouped(a, w, st):
    """a [S][k] f32, w [E][n][k] f32 -> [S][n] f32: the experts' rows padded to one batch."""
    return torch.bmm(a[st["row"]], w.transpose(1, 2).contiguous())[st["real"]]


def _gated(gu):
    gate, up = gu.chunk(2, -1)
    return gate / (1.0 + torch.exp(-gate)) * up


def _plain(st):
    op = st["op"]
    if op == "dispatch_fp8":
        q, scale = _quantize(st["x"])
        send = q.view(torch.uint8)[st["token"]].view(torch.float8_e4m3fn)
        return {"send": send, "scale": scale[st["token"]]}
    if op == "expert_gemm":
        y = _grouped(_values(st["a"], st["a_scale"]), _weight_values(st["w"], st["w_scale"]), st)
        return {"y": y.to(torch.bfloat16)}
    if op == "expert_ffn":
        gu = _grouped(_values(st["a"], st["a_scale"]), _weight_values(st["w13"], st["w13_scale"]),
                      st)
        h = _values(*_quantize(_gated(gu)))
        y = _grouped(h, _weight_values(st["w2"], st["w2_scale"]), st)
        out = {"y": y.to(torch.bfloat16)}
        if st["save"]:
            out["gate_up"] = gu.to(torch.bfloat16)
        return out
    if op == "expert_wgrad":
        real = st["real"].unsqueeze(-1)
        dy = st["dy"].float()[st["row"]] * real
        x = st["x"].float()[st["row"]] * real
        return {"dw": torch.bmm(dy.transpose(1, 2).contiguous(), x)}
    if op == "swiglu_grad":
        gate, up = st["gate_up"].float().chunk(2, -1)
        dh = st["dh"].float()
        sig = 1.0 / (1.0 + torch.exp(-gate))
        silu = gate * sig
        dgate = dh * up * (sig + silu * (1.0 - sig))
        return {"dgate_up": torch.cat([dgate, dh * silu], -1).to(torch.bfloat16),
                "h": (silu * up).to(torch.bfloat16)}
    x, idx, w = st["x"].float(), st["idx"].long(), st["w"]
    T, k, E = x.shape[0], idx.shape[1], st["w13"].shape[0]
    if T * k < E:       # fewer picks than experts: only the picked experts' weights
        flat = idx.reshape(-1)
        pick = lambda v: None if v is None else v.view(torch.uint8 if v.dtype != torch.bfloat16  # noqa: E731
                                                       else v.dtype)[flat].view(v.dtype)
        w13 = _weight_values(pick(st["w13"]), pick(st["w13_scale"]))
        w2 = _weight_values(pick(st["w2"]), pick(st["w2_scale"]))
        xs = x.repeat_interleave(k, 0)
        h = _gated(torch.bmm(w13, xs.unsqueeze(-1)).squeeze(-1)) * w.reshape(-1, 1)
        y = torch.bmm(w2, h.unsqueeze(-1)).squeeze(-1).view(T, k, -1).sum(1)
        return {"out": y.to(torch.bfloat16)}
    w13, w2 = _weight_values(st["w13"], st["w13_scale"]), _weight_values(st["w2"], st["w2_scale"])
    share = torch.zeros(T, E, device=x.device).scatter_add_(1, idx, w)       # [T][E]
    gu = (x @ w13.view(-1, w13.shape[-1]).t()).view(T, E, -1)
    h = (_gated(gu) * share.unsqueeze(-1)).transpose(0, 1).contiguous()      # [E][T][I]
    y = torch.bmm(h, w2.transpose(1, 2).contiguous()).sum(0)
    return {"out": y.to(torch.bfloat16)}


# --------------------------------------------------------------------------- one pass
def run(st):
    if not own:
        return _plain(st)
    from combine_ep_route_topk_amd import ep
    op = st["op"]
    if op == "dispatch_fp8":
        send, scale = ep.ep_dispatch_fp8(st["x"], st["pos"])
        return {"send": send, "scale": scale}
    if op == "expert_gemm":
        return {"y": ep.ep_expert_gemm_fp8(st["a"], st["a_scale"], st["w"], st["w_scale"],
                                           st["offsets"])}
    if op == "expert_ffn":
        h, h_scale, gate_up = ep.ep_expert_swiglu_fp8(st["a"], st["a_scale"], st["w13"],
                                                      st["w13_scale"], st["offsets"],
                                                      save_gate_up=st["save"])
        out = {"y": ep.ep_expert_gemm_fp8(h, h_scale, st["w2"], st["w2_scale"], st["offsets"])}
        if st["save"]:
            out["gate_up"] = gate_up
        return out
    if op == "expert_wgrad":
        return {"dw": ep.ep_expert_wgrad(st["dy"], st["x"], st["offsets"])}
    if op == "swiglu_grad":
        dgate_up, h = ep.ep_swiglu_grad(st["dh"], st["gate_up"])
        return {"dgate_up": dgate_up, "h": h}
    return {"out": ep.ep_moe_tokens(st["x"], st["idx"], st["w"], st["w13"], st["w2"],
                                    st["w13_scale"], st["w2_scale"])}


# --------------------------------------------------------------------------- definitions, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "dispatch_fp8":
        v, exps = _quantize64(st["x"].double())
        step = torch.exp2(exps.double()).repeat_interleave(BLOCK, 1)[:, :v.shape[1]]
        return {"send": (v / step)[st["token"]], "scale": (exps + 127).to(torch.uint8)[st["token"]]}
    if op == "swiglu_grad":
        dh, gu = st["dh"].double(), st["gate_up"].double()
        I = dh.shape[1]
        g, u = gu[:, :I], gu[:, I:]
        s = torch.sigmoid(g)
        return {"dgate_up": torch.cat([dh * u * s * (1 + g * (1 - s)), dh * g * s], 1),
                "h": g * s * u}
    if op == "moe_tokens":
        x, out = st["x"].double(), torch.zeros(case["T"], case["H"], dtype=torch.float64, device=DEV)
        for e in torch.unique(st["idx"]).tolist():
            t, j = torch.nonzero(st["idx"] == e, as_tuple=True)
            w13 = _dense64(st["w13"][e], None if st["w13_scale"] is None else st["w13_scale"][e])
            w2 = _dense64(st["w2"][e], None if st["w2_scale"] is None else st["w2_scale"][e])
            h = _silu_up64(x[t] @ w13.t())
            out.index_add_(0, t, (h @ w2.t()) * st["w"].double()[t, j].unsqueeze(1))
        return {"out": out}
    b = st["offsets"].tolist()
    got = {}
    for e in range(case["E"]):
        lo, hi = b[e], b[e + 1]
        if op == "expert_wgrad":
            got.setdefault("dw", []).append((st["dy"][lo:hi].double().t() @ st["x"][lo:hi].double()
                                             )[None])
            continue
        a = _rows64(st["a"][lo:hi], st["a_scale"][lo:hi])
        if op == "expert_gemm":
            got.setdefault("y", []).append(a @ _dense64(st["w"][e], st["w_scale"][e]).t())
            continue
        gu = a @ _dense64(st["w13"][e], st["w13_scale"][e]).t()
        h, _ = _quantize64(_silu_up64(gu))
        got.setdefault("y", []).append(h @ _dense64(st["w2"][e], st["w2_scale"][e]).t())
        if st["save"]:
            got.setdefault("gate_up", []).append(gu)
    return {k: torch.cat(v) for k, v in got.items()}


def _silu_up64(gu):
    I = gu.shape[1] // 2
    return gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]


def _rows64(q, byte):
    s = torch.exp2(byte.double() - 127)
    return q.double() * s[:, torch.arange(q.shape[1], device=q.device) // BLOCK]


def _dense64(w, byte):
    if byte is None:
        return w.double()
    n = torch.arange(w.shape[0], device=w.device) // BLOCK
    k = torch.arange(w.shape[1], device=w.device) // BLOCK
    return w.double() * torch.exp2(byte.double() - 127)[n][:, k]


def _quantize64(v):
    """The values that the quantised rows stand for, and the scales' exponents: each value is
    rounded, ties to even, to a multiple of 2^-3 of its binade (2^-9 below 2^-6), in units of
    its block's scale."""
    n = v.shape[1]
    k = torch.arange(n, device=v.device) // BLOCK
    nb = -(-n // BLOCK)
    amax = torch.zeros(v.shape[0], nb, dtype=torch.float64, device=v.device)
    amax.scatter_reduce_(1, k.expand(v.shape[0], n), v.abs(), "amax")
    e = torch.ceil(torch.log2(amax / E4M3_MAX))
    e = torch.where(amax <= E4M3_MAX * torch.exp2(e - 1), e - 1, e)     # log2 rounded up
    e = torch.where(amax > E4M3_MAX * torch.exp2(e), e + 1, e)          # log2 rounded down
    e = torch.where(amax == 0, torch.zeros_like(e), torch.clamp(e, min=-126))
    s = torch.exp2(e)[:, k]
    u = v / s
    step = torch.exp2(torch.clamp(torch.frexp(u)[1] - 1, min=-6).double() - 3)
    return torch.round(u / step) * step * s, e.to(torch.int32)
