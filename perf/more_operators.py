"""Cases of the expert operators in bf16 and in 8-bit integers: the products grouped by expert, with
their input gradient and with the gated activation, and the quantiser of rows.

An 8-bit integer tensor here is int8 values with one f32 scale for each row: a token's, or that of an
output channel of a weight matrix.  With m the row's largest magnitude (127 * 2^-126 at least) the
scale is m / 127, and a value is 127 x / m rounded to the nearest integer, ties to even.  The experts'
rows lie in one buffer, expert after expert, as the dispatch layout orders them; `offsets` [E + 1]
bounds them.

  rows_int8   x [T][H] -> quantised rows and scales, in order (k = 0) or at pos[t][j] (dispatch)
  gemm_bf16   y[s] = W[e(s)] a[s], or W[e(s)]^T a[s] (an input gradient from the forward weights)
  ffn_bf16    y[s] = W2[e] bf16(silu(G) * U), [G; U] = W13[e] a[s]
  gemm_int8   y[s][n] = scale[s] scale[e][n] sum_k a[s][k] W[e][n][k]
  ffn_int8    the same feed-forward on int8 rows and weights, bf16(silu(G) * U) quantised by row
"""
import math

import torch

own = False     # True: run() calls the framework; False: run() computes the plain forms

DEV = "cuda:0"
LEAST = 127.0 * 2.0 ** -126     # of a row's largest magnitude: scales stay normal numbers


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's 128 tokens going out to 256 experts: latency
        dict(name="dispatch_int8_decode", op="rows_int8", T=128, H=7168, E=256, k=8),
        # a prefill batch of 4096 tokens
        dict(name="dispatch_int8_prefill", op="rows_int8", T=4096, H=7168, E=256, k=8),
        # the channels of eight experts' gate/up weights, quantised once when a model is loaded
        dict(name="quantize_int8_weights", op="rows_int8", T=32768, H=7168, E=1, k=0),
        # a decode step on one rank's 8 experts: a few rows each, the weights' bytes bound it
        dict(name="gemm_bf16_decode", op="gemm_bf16", S=64, N=4096, K=7168, E=8, rows="zipf",
             transposed=False),
        # input gradient of a short ragged micro-batch, one expert in four without rows
        dict(name="gemm_bf16_dgrad_ragged", op="gemm_bf16", S=1000, N=4096, K=2816, E=16, rows="gaps",
             transposed=True),
        # input gradient of a full batch against the gate/up weights
        dict(name="gemm_bf16_dgrad_train", op="gemm_bf16", S=32768, N=7168, K=4096, E=8, rows="even",
             transposed=True),
        # a short ragged micro-batch through narrow experts, gate_up kept for the backward pass
        dict(name="ffn_bf16_ragged", op="ffn_bf16", S=1000, H=4096, I=1408, E=16, rows="gaps",
             save=True),
        # a training batch (4096 tokens, top-8) through 8 local experts
        dict(name="ffn_bf16_train", op="ffn_bf16", S=32768, H=7168, I=2048, E=8, rows="even", save=True),
        # a decode step in 8 bits
        dict(name="gemm_int8_decode", op="gemm_int8", S=256, N=4096, K=7168, E=8, rows="zipf"),
        # a prefill batch through the down projections
        dict(name="gemm_int8_prefill", op="gemm_int8", S=16384, N=7168, K=2048, E=8, rows="even"),
        # one user's token through 8 of 64 experts
        dict(name="ffn_int8_one_token", op="ffn_int8", S=8, H=7168, I=2048, E=64, rows="one"),
        # a prefill batch (4096 tokens, top-8) through 8 local experts
        dict(name="ffn_int8_prefill", op="ffn_int8", S=32768, H=7168, I=2048, E=8, rows="even"),
    ]


def draw(rng):
    def size(lo, hi, step=1):
        return max(1, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step

    op = rng.choice(["rows_int8", "gemm_bf16", "ffn_bf16", "gemm_int8", "ffn_int8"])
    if op == "rows_int8":
        E = rng.choice([8, 33, 64, 128, 256])
        return dict(op=op, T=size(1, 8192), H=size(64, 8192, 16), E=E, k=rng.randint(0, 8))
    rows = rng.choice(["even", "zipf", "gaps"])
    E, S = rng.randint(1, 32), size(1, 32768)
    if op == "gemm_bf16":
        return dict(op=op, S=S, N=size(64, 7168, 8), K=size(64, 4096, 8), E=E, rows=rows,
                    transposed=rng.random() < 0.5)
    if op == "gemm_int8":
        return dict(op=op, S=S, N=size(64, 7168, 16), K=size(64, 4096, 16), E=E, rows=rows)
    if op == "ffn_bf16":
        return dict(op=op, S=S, H=size(64, 7168, 8), I=size(64, 2048, 8), E=E, rows=rows,
                    save=rng.random() < 0.5)
    return dict(op=op, S=S, H=size(64, 7168, 16), I=size(64, 2048, 16), E=E, rows=rows)


def work(case):
    c = case
    if c["op"] == "rows_int8":
        T, H, k = c["T"], c["H"], c["k"]
        return {"bytes": 2 * T * H + 4 * T * k + T * max(k, 1) * (H + 4), "flops": 4 * T * H}
    S, E = c["S"], _used(c)
    if c["op"] == "gemm_bf16":
        N, K = c["N"], c["K"]
        return {"bytes": 2 * S * (N + K) + 2 * E * N * K, "flops": 2 * S * N * K}
    if c["op"] == "gemm_int8":
        N, K = c["N"], c["K"]
        return {"bytes": S * (K + 4 + 2 * N) + E * N * (K + 4), "flops": 2 * S * N * K}
    H, I = c["H"], c["I"]
    if c["op"] == "ffn_bf16":
        return {"bytes": S * (4 * H + (4 * I if c["save"] else 0)) + 6 * E * I * H,
                "flops": 6 * S * H * I}
    return {"bytes": S * (H + 4 + 2 * H) + E * (3 * I * H + 4 * (2 * I + H)), "flops": 6 * S * H * I}


def _used(c):
    """Experts that have rows, as _counts spreads them."""
    return min(c["S"], c["E"] - c["E"] // 4 if c["rows"] == "gaps" else c["E"])


# --------------------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _tokens(g, n, h):
    """Activations: normal values, rows of different size."""
    return (_normal(g, n, h) * torch.exp(0.3 * _normal(g, n, 1))).to(torch.bfloat16)


def _weights(g, E, n, k, fan_in):
    """E matrices with the spread of a trained layer's weights."""
    w = torch.empty(E, n, k, dtype=torch.bfloat16, device=DEV)
    for e in range(E):
        w[e] = _normal(g, n, k) * (1.0 / math.sqrt(fan_in))
    return w


def _quantize(x):
    """x [n][h] -> int8 values and f32 scales [n].  The quotient in 64 bits: next to a half integer
    32 would decide by their rounding."""
    m = x.double().abs().amax(1).clamp(min=LEAST)
    q = torch.round(x.double() * 127.0 / m[:, None]).to(torch.int8)
    return q, (m / 127.0).float()


def _weights_int8(g, E, n, k):
    q = torch.empty(E, n, k, dtype=torch.int8, device=DEV)
    s = torch.empty(E, n, dtype=torch.float32, device=DEV)
    for e in range(E):
        q[e], s[e] = _quantize(_weights(g, 1, n, k, k)[0])
    return q, s


def _counts(case, seed):
    """Rows of each expert (host): S picks drawn evenly, by a Zipf law, with a quarter of the experts
    left out, or of S different experts."""
    S, E = case["S"], case["E"]
    g = torch.Generator().manual_seed(int(seed) + 7)
    p = torch.ones(E)
    if case["rows"] == "zipf":
        p = 1.0 / torch.arange(1, E + 1).float()
        p = p[torch.randperm(E, generator=g)]
    elif case["rows"] == "gaps":
        p[torch.randperm(E, generator=g)[:E // 4]] = 0.0
    picks = torch.multinomial(p, S, replacement=case["rows"] != "one", generator=g)
    return torch.bincount(picks, minlength=E)


def _segments(case, seed):
    """The experts' row ranges: `offsets` on the GPU as the dispatch layout gives them, and on the host."""
    ends = torch.cumsum(_counts(case, seed), 0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    return dict(offsets=offsets.to(torch.int32).to(DEV), bounds=offsets.tolist())


def prepare(case, seed):
    g = _generator(seed)
    op, E = case["op"], case["E"]
    if op == "rows_int8":
        T, H, k = case["T"], case["H"], min(case["k"], E)
        st = dict(op=op, x=_tokens(g, T, H), pos=None)
        if k:
            idx = torch.topk(_normal(g, T, E), k, dim=1)[1]
            order = torch.argsort(idx.reshape(-1), stable=True)     # row -> pick
            pos = torch.empty_like(order)
            pos[order] = torch.arange(T * k, device=DEV)
            st.update(pos=pos.view(T, k).to(torch.int32), token=order // k)
        return st
    seg = _segments(case, seed)
    if op == "gemm_bf16":
        N, K, t = case["N"], case["K"], case["transposed"]
        w = _weights(g, E, K, N, K) if t else _weights(g, E, N, K, K)
        return dict(op=op, a=_tokens(g, case["S"], K), w=w, transposed=t, **seg)
    if op == "gemm_int8":
        a, a_scale = _quantize(_tokens(g, case["S"], case["K"]))
        w, w_scale = _weights_int8(g, E, case["N"], case["K"])
        return dict(op=op, a=a, a_scale=a_scale, w=w, w_scale=w_scale, **seg)
    H, I = case["H"], case["I"]
    if op == "ffn_bf16":
        return dict(op=op, a=_tokens(g, case["S"], H), w13=_weights(g, E, 2 * I, H, H),
                    w2=_weights(g, E, H, I, I), save=case["save"], **seg)
    a, a_scale = _quantize(_tokens(g, case["S"], H))
    w13, w13_scale = _weights_int8(g, E, 2 * I, H)
    w2, w2_scale = _weights_int8(g, E, H, I)
    return dict(op=op, a=a, a_scale=a_scale, w13=w13, w13_scale=w13_scale, w2=w2, w2_scale=w2_scale,
                **seg)


# --------------------------------------------------------------------------- plain forms, in 32 bits
def _grouped(a, w, bounds, transposed=False):
    """a [S][k] f32, w [E] matrices of any type -> [S][n] f32, expert by expert."""
    out = []
    for e in range(len(bounds) - 1):
        if bounds[e + 1] > bounds[e]:
            m = w[e].float()
            out.append(a[bounds[e]:bounds[e + 1]] @ (m if transposed else m.t()))
    return torch.cat(out)


def _channels(scale, bounds):
    """Channel scales [E][n] -> [S][n], each row its expert's."""
    return torch.cat([scale[e].expand(bounds[e + 1] - bounds[e], -1) for e in range(len(bounds) - 1)])


def _gated(gu):
    gate, up = gu.chunk(2, -1)
    return gate / (1.0 + torch.exp(-gate)) * up


def _plain(st):
    op = st["op"]
    if op == "rows_int8":
        q, scale = _quantize(st["x"])
        if st["pos"] is None:
            return {"q": q, "scale": scale}
        return {"q": q[st["token"]], "scale": scale[st["token"]]}
    b = st["bounds"]
    if op == "gemm_bf16":
        return {"y": _grouped(st["a"].float(), st["w"], b, st["transposed"]).to(torch.bfloat16)}
    if op == "gemm_int8":
        y = _grouped(st["a"].float(), st["w"], b) * st["a_scale"][:, None] * _channels(st["w_scale"], b)
        return {"y": y.to(torch.bfloat16)}
    if op == "ffn_bf16":
        gu = _grouped(st["a"].float(), st["w13"], b)
        h = _gated(gu).to(torch.bfloat16)
        out = {"y": _grouped(h.float(), st["w2"], b).to(torch.bfloat16)}
        if st["save"]:
            out["gate_up"] = gu.to(torch.bfloat16)
        return out
    gu = _grouped(st["a"].float(), st["w13"], b) * st["a_scale"][:, None] * _channels(st["w13_scale"], b)
    h, h_scale = _quantize(_gated(gu).to(torch.bfloat16))
    y = _grouped(h.float(), st["w2"], b) * h_scale[:, None] * _channels(st["w2_scale"], b)
    return {"y": y.to(torch.bfloat16)}


# --------------------------------------------------------------------------- one pass
def run(st):
    if not own:
        return _plain(st)
    from combine_ep_route_topk_amd import ep
    op = st["op"]
    if op == "rows_int8":
        if st["pos"] is None:
            q, scale = ep.ep_quantize_int8(st["x"])
        else:
            q, scale = ep.ep_dispatch_int8(st["x"], st["pos"])
        return {"q": q, "scale": scale}
    off = st["offsets"]
    if op == "gemm_bf16":
        return {"y": ep.ep_expert_gemm_bf16(st["a"], st["w"], off, transposed=st["transposed"])}
    if op == "gemm_int8":
        return {"y": ep.ep_expert_gemm_int8(st["a"], st["a_scale"], st["w"], st["w_scale"], off)}
    if op == "ffn_bf16":
        h, gate_up = ep.ep_expert_swiglu_bf16(st["a"], st["w13"], off, save_gate_up=st["save"])
        out = {"y": ep.ep_expert_gemm_bf16(h, st["w2"], off)}
        if st["save"]:
            out["gate_up"] = gate_up
        return out
    h, h_scale = ep.ep_expert_swiglu_int8(st["a"], st["a_scale"], st["w13"], st["w13_scale"], off)
    return {"y": ep.ep_expert_gemm_int8(h, h_scale, st["w2"], st["w2_scale"], off)}


# --------------------------------------------------------------------------- definitions, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "rows_int8":
        v, unit = _integers64(st["x"].double())
        if st["pos"] is not None:
            v, unit = v[st["token"]], unit[st["token"]]
        return {"q": v.to(torch.int8), "scale": unit}
    off = st["offsets"].tolist()
    y, kept = [], []
    for e in range(case["E"]):
        rows = slice(off[e], off[e + 1])
        a = st["a"][rows].double()
        if op == "gemm_bf16":
            w = st["w"][e].double()
            y.append(a @ w if case["transposed"] else a @ w.t())
            continue
        if op == "gemm_int8":
            y.append((a @ st["w"][e].double().t()) * torch.outer(st["a_scale"][rows].double(),
                                                                 st["w_scale"][e].double()))
            continue
        gu = a @ st["w13"][e].double().t()
        if op == "ffn_int8":
            gu *= torch.outer(st["a_scale"][rows].double(), st["w13_scale"][e].double())
        I = case["I"]
        h = _bf16_64(gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:])
        if op == "ffn_bf16":
            kept.append(gu)
            y.append(h @ st["w2"][e].double().t())
            continue
        v, unit = _integers64(h)
        y.append((v @ st["w2"][e].double().t()) * torch.outer(unit, st["w2_scale"][e].double()))
    out = {"y": torch.cat(y)}
    if kept and case["save"]:
        out["gate_up"] = torch.cat(kept)
    return out


def _bf16_64(v):
    """f64 rounded to 8 bits of mantissa, ties to even (bf16's values above its least normal one)."""
    step = torch.exp2((torch.frexp(v)[1] - 8).clamp(min=-133).double())
    return torch.round(v / step) * step


def _integers64(v):
    """The rows' integers (f64) and their units."""
    top = torch.maximum(v.abs().amax(1), torch.full_like(v[:, 0], LEAST)) if v.shape[0] else v[:, 0]
    return torch.round(v * 127.0 / top[:, None]), top / 127.0
