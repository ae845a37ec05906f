"""A frozen weight in 4 bits and the experts of a mixture, as cases that can be timed and compared.

The 4-bit form of a matrix [rows, cols]: one E2M1 value per element, two a byte
(the even column in the low half), and one power-of-two scale 2^(byte - 127) per
32 columns of a row; the byte 255 stands for NaN.

  form       a weight into the 4-bit form and back
  matmul     y = x W^T, W in 4 bits; with experts, x's rows are sorted by expert and
             each run of them meets its own W
  matmul_t   dx = dy W, the same W
  route      tokens sorted by expert (order, its inverse, offsets), sent to the experts'
             rows, returned as a weighted sum, and the gradients of both

With ``own`` false, run() computes them in elementary torch operations in 32
bits; with ``own`` true it calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 32
MIN_SCALE = 2           # 2^-125, the smallest scale that a store gives


def listed():
    return [
        # the smallest module's weight: latency
        {"name": "form tiny", "op": "form", "act": "bfloat16", "rows": 512, "cols": 512},
        # the MLP's gate/up projection from a float32 checkpoint
        {"name": "form mlp f32", "op": "form", "act": "float32", "rows": 14336, "cols": 4096},
        # one token through the smallest module: latency
        {"name": "matmul token tiny", "op": "matmul", "T": 1, "out": 512, "cols": 512, "experts": 0},
        # serving one token: bound by reading the weight
        {"name": "matmul token", "op": "matmul", "T": 1, "out": 8192, "cols": 8192, "experts": 0},
        # serving an odd batch through the MLP's gate/up projection
        {"name": "matmul batch", "op": "matmul", "T": 37, "out": 14336, "cols": 4096, "experts": 0},
        # an attention projection of a training step
        {"name": "matmul attention", "op": "matmul", "T": 8192, "out": 4096, "cols": 4096, "experts": 0},
        # one token at its eight experts of sixty-four
        {"name": "matmul experts token", "op": "matmul", "T": 8, "out": 2048, "cols": 4096, "experts": 64},
        # a prompt's tokens at their experts, loads uneven, some experts idle
        {"name": "matmul experts prompt", "op": "matmul", "T": 4096, "out": 2048, "cols": 4096, "experts": 32},
        # the gradient of the high-rank module's input
        {"name": "matmul_t high rank", "op": "matmul_t", "T": 15360, "out": 8192, "cols": 8192, "experts": 0},
        # the gradient of a short sequence's tokens at a few experts, odd sizes
        {"name": "matmul_t experts", "op": "matmul_t", "T": 1001, "out": 1040, "cols": 2080, "experts": 8},
        # a decoding batch, some of its tokens padding: latency
        {"name": "route batch", "op": "route", "T": 63, "k": 6, "cols": 4096, "experts": 60, "padded": True},
        # a training step's tokens
        {"name": "route step", "op": "route", "T": 8192, "k": 8, "cols": 4096, "experts": 64, "padded": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["form", "matmul", "matmul", "matmul", "matmul_t", "matmul_t", "route", "route"])
    if op == "form":
        return {"op": op, "act": rng.choice(["bfloat16", "float32"]), "rows": _log(rng, 1, 14336),
                "cols": GROUP * _log(rng, 1, 448)}
    if op == "route":
        return {"op": op, "T": _log(rng, 1, 8192), "k": rng.randint(1, 8), "cols": 8 * _log(rng, 8, 512),
                "experts": _log(rng, 1, 128), "padded": rng.random() < 0.5}
    case = {"op": op, "T": _log(rng, 1, 16384), "out": 16 * _log(rng, 8, 896), "cols": GROUP * _log(rng, 4, 448),
            "experts": rng.choice([0, _log(rng, 2, 128)])}
    E = max(case["experts"], 1)
    while E * case["out"] * case["cols"] > 64 * 2048 * 4096:      # a stack of weights that is quickly made
        E = E // 2
        case["experts"] = E if E > 1 else 0
    while case["T"] * case["out"] * case["cols"] > 15360 * 8192 * 8192:   # no more work than the largest listed case
        case["T"] = case["T"] // 2 + 1
    return case


# ---------------------------------------------------------------------------
# the 4-bit form, in elementary operations
# ---------------------------------------------------------------------------
def _quantize(v):
    """float32 [..., C] -> (bytes [..., C / 2], scale bytes [..., C / 32])."""
    g = v.unflatten(-1, (-1, GROUP))
    finite = torch.isfinite(g).all(-1)
    amax = torch.where(torch.isfinite(g), g.abs(), 0.0).amax(-1)
    # the smallest power of two that brings amax to at most 6 = 1.5 * 2^2
    byte = (((amax.view(torch.int32) + 0x3FFFFF) >> 23) - 2).clamp(min=MIN_SCALE)
    inv = ((254 - byte) << 23).view(torch.float32)
    u = (g * inv[..., None]).abs()
    # 0 .5 1 1.5 2 3 4 6, ties to the even mantissa
    n = ((u > 0.25).int() + (u >= 0.75) + (u > 1.25) + (u >= 1.75) + (u > 2.5) + (u >= 3.5) + (u > 5.0))
    n = n + 8 * torch.signbit(g)
    n = torch.where(finite[..., None], n, 0).flatten(-2).to(torch.uint8)
    byte = torch.where(finite, byte, 255).to(torch.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4), byte


def _dequantize(q, scale):
    """float32 [..., C] of a 4-bit form."""
    n = torch.stack([q & 15, q >> 4], -1).flatten(-2).int()
    m = n & 7
    mag = torch.where(m < 4, 0.5 * m, torch.where(m < 6, m - 2.0, 2.0 * m - 8.0))
    v = torch.where(n >= 8, -mag, mag).unflatten(-1, (-1, GROUP))
    b = scale.int()
    s = torch.where(b == 255, float("nan"), torch.where(b > 0, (b << 23).view(torch.float32), 2.0 ** -127))
    return (v * s[..., None]).flatten(-2)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _hidden(gen, T, cols):
    """Hidden states: normal, with a few columns that are far larger, as a model's residual stream has."""
    x = torch.randn(T, cols, generator=gen, device=DEV)
    loud = torch.rand(cols, generator=gen, device=DEV) < 0.004
    return x * torch.where(loud, 24.0, 1.0)


def _loads(T, experts, seed):
    """How many of T rows each expert has: uneven, none for some."""
    gen = torch.Generator().manual_seed(seed)
    p = torch.rand(experts, generator=gen) ** 2 + 1e-6
    picks = torch.multinomial(p, T, replacement=True, generator=gen)
    return torch.bincount(picks, minlength=experts).tolist()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, C = case["op"], case["cols"]
    st = {"op": op}

    def u8(*shape):
        return torch.empty(*shape, dtype=torch.uint8, device=DEV)

    if op == "form":
        act, R = getattr(torch, case["act"]), case["rows"]
        st["x"] = (torch.randn(R, C, generator=gen, device=DEV) / math.sqrt(C)).to(act)
        st["q"], st["scale"], st["back"] = u8(R, C // 2), u8(R, C // GROUP), torch.empty(R, C, dtype=act, device=DEV)
        return st
    T, E = case["T"], case["experts"]
    if op == "route":
        k = case["k"]
        # k different experts a token, where there are as many; loads uneven
        score = torch.rand(T, E, generator=gen, device=DEV) + 0.3 * torch.rand(E, generator=gen, device=DEV)
        expert = score.argsort(-1, descending=True)[:, torch.arange(k, device=DEV) % E].int()
        if case["padded"]:
            expert[T - T // 8:] = -1
        st["expert"] = expert.contiguous()
        st["weight"] = torch.rand(T, k, generator=gen, device=DEV).softmax(-1)
        st["x"] = _hidden(gen, T, C).bfloat16()
        st["ys"] = torch.randn(T * k, C, generator=gen, device=DEV).bfloat16()
        st["d_xs"] = torch.randn(T * k, C, generator=gen, device=DEV).bfloat16()
        st["dy"] = torch.randn(T, C, generator=gen, device=DEV).bfloat16()
        st["experts"] = E
        st["order"] = torch.empty(T * k, dtype=torch.int32, device=DEV)
        st["inverse"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
        st["offsets"] = torch.empty(E + 1, dtype=torch.int32, device=DEV)
        # rows behind the last expert's are left as they are
        st["xs"], st["d_ys"] = torch.zeros_like(st["ys"]), torch.zeros_like(st["ys"])
        st["y"], st["dx"], st["d_weight"] = torch.empty_like(st["x"]), torch.empty_like(st["x"]), torch.empty(T, k, device=DEV)
        return st
    out = case["out"]
    parts = []
    for _ in range(max(E, 1)):
        parts.append(_quantize(torch.randn(out, C, generator=gen, device=DEV) / math.sqrt(C)))
    wq, wscale = (torch.stack(p) for p in zip(*parts))
    st["wq"], st["wscale"] = (wq, wscale) if E else (wq[0], wscale[0])
    st["counts"] = _loads(T, E, seed) if E else [T]
    st["offsets"] = None
    if E:
        st["offsets"] = torch.tensor([0] + st["counts"], device=DEV).cumsum(0).int()
    wide = C if op == "matmul" else out
    st["x"] = (_hidden(gen, T, wide) if op == "matmul" else torch.randn(T, wide, generator=gen, device=DEV)).bfloat16()
    st["y"] = torch.empty(T, out if op == "matmul" else C, dtype=torch.bfloat16, device=DEV)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _plain_route(st):
    expert, E = st["expert"].flatten().long(), st["experts"]
    T, k = st["weight"].shape
    at = torch.where((expert >= 0) & (expert < E), expert, E)
    hot = at[:, None] == torch.arange(E + 1, device=DEV)
    count = hot.sum(0)
    start = count.cumsum(0) - count
    rank = hot.int().cumsum(0).gather(1, at[:, None]).squeeze(1) - 1
    inverse = start[at] + rank
    order = torch.empty_like(inverse)
    order[inverse] = torch.arange(T * k, device=DEV)
    sent = (at < E).view(T, k)
    p = inverse.view(T, k)
    live = (torch.arange(T * k, device=DEV) < start[E])[:, None]
    xs = torch.where(live, st["x"][order // k], 0.0)
    w = torch.where(sent, st["weight"], 0.0)
    y = torch.zeros(T, st["x"].shape[1], device=DEV)
    dx = torch.zeros_like(y)
    d_weight = torch.zeros_like(w)
    dy = st["dy"].float()
    for j in range(k):
        row = st["ys"][p[:, j]].float()
        y += w[:, j, None] * row
        dx += torch.where(sent[:, j, None], st["d_xs"][p[:, j]].float(), 0.0)
        d_weight[:, j] = torch.where(sent[:, j], (dy * row).sum(-1), 0.0)
    d_ys = torch.where(live, w.flatten()[order][:, None] * dy[order // k], 0.0)
    return {"order": order.int(), "inverse": p.int(), "offsets": start.int(), "xs": xs, "y": y.bfloat16(),
            "d_ys": d_ys.bfloat16(), "d_weight": d_weight, "dx": dx.bfloat16()}


def _plain(st):
    op = st["op"]
    if op == "form":
        return {"x": _dequantize(*_quantize(st["x"].float())).to(st["x"].dtype)}
    if op == "route":
        return _plain_route(st)
    x, wq, wscale = st["x"].float(), st["wq"], st["wscale"]
    if st["offsets"] is None:
        wq, wscale = wq[None], wscale[None]
    y = []
    for e, rows in enumerate(x.split(st["counts"])):
        if rows.shape[0]:
            W = _dequantize(wq[e], wscale[e])
            y.append(rows @ (W.t() if op == "matmul" else W))
    return {"y": torch.cat(y).bfloat16()}


def _library(st):
    import parameter_efficient_fine_gb300 as dora
    op = st["op"]
    if op == "form":
        dora.dora_q4_store(st["x"], st["q"], st["scale"])
        dora.dora_q4_load(st["q"], st["scale"], st["back"])
        return {"x": st["back"]}
    if op == "route":
        dora.dora_expert_sort(st["expert"], st["experts"], st["order"], st["inverse"], st["offsets"])
        dora.dora_expert_send(st["x"], st["inverse"], st["offsets"], st["xs"])
        dora.dora_expert_return(st["ys"], st["inverse"], st["offsets"], st["weight"], st["y"])
        dora.dora_expert_return_bwd(st["dy"], st["ys"], st["inverse"], st["offsets"], st["weight"], st["d_ys"],
                                    st["d_weight"])
        dora.dora_expert_return(st["d_xs"], st["inverse"], st["offsets"], None, st["dx"])
        return {n: st[n] for n in ("order", "inverse", "offsets", "xs", "y", "d_ys", "d_weight", "dx")}
    if "workspace" not in st:      # the call's scratch memory, kept beside its other buffers
        out, half = st["wq"].shape[-2:]
        E = 1 if st["offsets"] is None else st["wq"].shape[0]
        size = dora.dora_matmul_q4_workspace if op == "matmul" else dora.dora_matmul_q4_t_workspace
        st["workspace"] = torch.empty(max(size(st["x"].shape[0], out, 2 * half, E), 1), dtype=torch.uint8, device=DEV)
    call = dora.dora_matmul_q4 if op == "matmul" else dora.dora_matmul_q4_t
    call(st["x"], st["wq"], st["wscale"], st["y"], st["offsets"], st["workspace"])
    return {"y": st["y"]}


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, C = case["op"], case["cols"]
    form = lambda R, K: R * K // 2 + R * K // GROUP  # noqa: E731
    if op == "form":             # x in, the 4-bit form out and in again, x back out
        R, e = case["rows"], {"bfloat16": 2, "float32": 4}[case["act"]]
        return {"bytes": 2 * e * R * C + 2 * form(R, C), "flops": 3 * R * C}
    T, E = case["T"], case["experts"]
    if op == "route":
        N = T * case["k"]
        if case["padded"]:
            N -= (T // 8) * case["k"]
        # x, dy in, y, dx out; ys, d_xs in, xs, d_ys out; indexes and weights
        return {"bytes": 8 * T * C + 8 * N * C + 20 * T * case["k"], "flops": 6 * N * C}
    out = case["out"]
    k, n = (C, out) if op == "matmul" else (out, C)
    used = min(E, T) if E else 1                 # experts that have tokens, at most
    if E:
        used = min(used, sum(c > 0 for c in _loads(T, E, 0)))
    return {"bytes": 2 * T * k + used * form(out, C) + 2 * T * n, "flops": 2 * T * out * C}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _two_to(k):
    """2^k for an integer tensor, exactly (a normal float64)."""
    return ((k.long() + 1023) << 52).view(torch.float64)


_VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exact_values(q, scale):
    """What the bytes of one matrix stand for."""
    table = torch.tensor(_VALUES + [-v for v in _VALUES], dtype=torch.float64, device=DEV)
    out = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.float64, device=DEV)
    out[:, 0::2] = table[(q % 16).long()]
    out[:, 1::2] = table[torch.div(q, 16, rounding_mode="floor").long()]
    return out.mul_(_two_to(scale.long() - 127).repeat_interleave(GROUP, 1))


def _exact_form(x):
    """The nearest values of the form to a float64 matrix, ties to even; one scale per 32 columns."""
    v = torch.empty_like(x)
    for c in range(0, x.shape[1], GROUP):
        b = x[:, c:c + GROUP]
        top = b.abs().amax(1, keepdim=True)
        m, e = torch.frexp(top)                     # top = m 2^e, m in [0.5, 1); 6 = 0.75 * 2^3
        k = torch.where(m > 0.75, e - 2, e - 3)
        k = torch.where(top == 0, torch.full_like(k, -125), k).clamp(min=-125)
        u = b * _two_to(-k)
        step = _two_to((torch.frexp(u)[1] - 1).clamp(min=0) - 1)     # one mantissa bit
        v[:, c:c + GROUP] = torch.round(u / step) * step * _two_to(k)
    return v


def _exact_route(st):
    expert = st["expert"].flatten().tolist()
    E, (T, k) = st["experts"], st["weight"].shape
    bins = [[] for _ in range(E + 1)]
    for i, e in enumerate(expert):
        bins[e if 0 <= e < E else E].append(i)
    offsets = [0]
    for b in bins[:E]:
        offsets.append(offsets[-1] + len(b))
    order = torch.tensor([i for b in bins for i in b], dtype=torch.int64)
    inverse = torch.empty_like(order)
    inverse[order] = torch.arange(T * k)
    n = offsets[E]
    tok = order[:n].to(DEV) // k
    first = order[:n].to(DEV)
    w = st["weight"].double().flatten()[first]
    x, dy, ys, d_xs = (st[v].double() for v in ("x", "dy", "ys", "d_xs"))
    xs, d_ys = torch.zeros_like(ys), torch.zeros_like(ys)
    xs[:n] = x[tok]
    d_ys[:n] = w[:, None] * dy[tok]
    y = torch.zeros_like(x).index_add_(0, tok, w[:, None] * ys[:n])
    dx = torch.zeros_like(x).index_add_(0, tok, d_xs[:n])
    d_weight = torch.zeros(T * k, dtype=torch.float64, device=DEV)
    d_weight[first] = torch.einsum("nc,nc->n", dy[tok], ys[:n])
    return {"order": order.int().to(DEV), "inverse": inverse.view(T, k).int().to(DEV),
            "offsets": torch.tensor(offsets, dtype=torch.int32, device=DEV), "xs": xs, "y": y, "d_ys": d_ys,
            "d_weight": d_weight.view(T, k), "dx": dx}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "form":
        return {"x": _exact_form(st["x"].double())}
    if op == "route":
        return _exact_route(st)
    stack = case["experts"] > 0
    y = torch.zeros(st["y"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for e, n in enumerate(st["counts"]):
        if n:
            W = _exact_values(*(v[e] if stack else v for v in (st["wq"], st["wscale"])))
            rows = st["x"][at:at + n].double()
            y[at:at + n] = torch.einsum("tk,nk->tn" if op == "matmul" else "tk,kn->tn", rows, W)
            at += n
    return {"y": y}
