"""The 8-bit operators of a DoRA training step, as cases that can be timed and compared.

The 8-bit form of a matrix [rows, cols]: one E4M3 byte per element, and one
power-of-two scale 2^(byte - 127) per block of 128 columns of a row (an
activation) or of 128 rows x 128 columns (a frozen weight).

  store      an activation into the 8-bit form and back
  compose_fwd  y = base + (g-1) base + g s lora, and v = base + s lora kept in 8 bits
  compose_bwd  d_base = g dy, d_lora = s g dy, d_mag = sum_t dy v / n from that v
  lora_grad  dA = dxa^T x from the 8-bit x
  matmul     y = x W^T with x and W in 8 bits
  matmul_t   dx = dy W with dy and W in 8 bits

With ``own`` false, run() computes them in elementary torch operations in 32
bits; with ``own`` true it calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
MIN_SCALE = 10          # 2^-117, the smallest scale


def listed():
    return [
        # one token's hidden state going into a cache of activations: latency
        {"name": "store token", "op": "store", "act": "bfloat16", "T": 1, "cols": 4096},
        # a layer's input kept for the backward pass, batch 3 x 5120 tokens
        {"name": "store step", "op": "store", "act": "bfloat16", "T": 15360, "cols": 8192},
        # odd sizes in float32: a scale block that ends inside a row, rows that start unaligned
        {"name": "compose fwd ragged f32", "op": "compose_fwd", "act": "float32", "T": 333, "cols": 1003, "r": 16},
        # the MLP's gate/up projection, the widest layer of the training step
        {"name": "compose fwd mlp", "op": "compose_fwd", "act": "bfloat16", "T": 16384, "cols": 14336, "r": 512},
        # the high-rank module's backward
        {"name": "compose bwd high rank", "op": "compose_bwd", "act": "bfloat16", "T": 15360, "cols": 8192, "r": 384},
        # the smallest module: latency
        {"name": "lora grad tiny", "op": "lora_grad", "T": 256, "cols": 512, "r": 16},
        # an attention projection at low rank: bound by reading x
        {"name": "lora grad attention", "op": "lora_grad", "T": 8192, "cols": 4096, "r": 64},
        # the high-rank module: bound by the products
        {"name": "lora grad high rank", "op": "lora_grad", "T": 15360, "cols": 8192, "r": 384},
        # serving one token: bound by reading the weight
        {"name": "matmul token", "op": "matmul", "T": 1, "out": 8192, "cols": 8192},
        # serving an odd batch through the MLP's gate/up projection
        {"name": "matmul batch", "op": "matmul", "T": 37, "out": 14336, "cols": 4096},
        # an attention projection of a training step
        {"name": "matmul attention", "op": "matmul", "T": 8192, "out": 4096, "cols": 4096},
        # the gradient of the high-rank module's input
        {"name": "matmul_t high rank", "op": "matmul_t", "T": 15360, "out": 8192, "cols": 8192},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        case = _draw(rng)
        if 3072 not in case.values():    # a size that no layer here has
            return case


def _draw(rng):
    op = rng.choice(["store", "compose_fwd", "compose_bwd", "lora_grad", "lora_grad", "matmul", "matmul", "matmul_t"])
    T = _log(rng, 1, 16384)
    if op in ("store", "compose_fwd", "compose_bwd"):
        case = {"op": op, "act": rng.choice(["bfloat16", "bfloat16", "float32"]), "T": T, "cols": _log(rng, 100, 14336)}
        if rng.random() < 0.5:                       # rows of whole 16-byte pieces
            case["cols"] = -(-case["cols"] // 8) * 8
        if op != "store":
            case["r"] = 8 * rng.randint(1, 96)
        return case
    cols = 16 * _log(rng, 8, 896)
    if op == "lora_grad":
        return {"op": op, "T": T, "cols": cols, "r": 8 * _log(rng, 1, 96)}
    out = 16 * _log(rng, 8, 896)
    while T * out * cols > 15360 * 8192 * 8192:      # no more work than the largest listed case
        T = T // 2 + 1
    return {"op": op, "T": T, "out": out, "cols": cols}


# ---------------------------------------------------------------------------
# the 8-bit form, in elementary operations
# ---------------------------------------------------------------------------
def _blocks(v, rows):
    """[R, C] -> [ceil(R / rows), rows, ceil(C / 128), 128], zeros past the edges."""
    R, C = v.shape
    nr, nc = -(-R // rows), -(-C // BLOCK)
    if nr * rows != R or nc * BLOCK != C:
        v = torch.nn.functional.pad(v, (0, nc * BLOCK - C, 0, nr * rows - R))
    return v.view(nr, rows, nc, BLOCK)


def _quantize(v, rows=1):
    """float32 [R, C] -> (E4M3 bytes [R, C], scale bytes [ceil(R / rows), ceil(C / 128)])."""
    R, C = v.shape
    b = _blocks(v, rows)
    finite = torch.isfinite(b)
    amax = torch.where(finite, b.abs(), 0.0).amax(dim=(1, 3))
    # the smallest power of two that brings amax to at most 448 = 1.75 * 2^8
    byte = ((amax.view(torch.int32) + 0x1FFFFF) >> 23) - 8
    byte = byte.clamp(min=MIN_SCALE)
    inv = ((254 - byte) << 23).view(torch.float32)
    u = torch.where(finite, b * inv[:, None, :, None], float("nan"))
    q = u.to(torch.float8_e4m3fn).view(torch.uint8).view(b.shape[0] * rows, -1)[:R, :C]
    return q.contiguous(), byte.to(torch.uint8)


def _dequantize(q, scale, rows=1):
    """float32 [R, C] of an 8-bit form."""
    R, C = q.shape
    b = _blocks(q.view(torch.float8_e4m3fn).float(), rows)
    s = (scale.to(torch.int32) << 23).view(torch.float32)
    return (b * s[:, None, :, None]).view(b.shape[0] * rows, -1)[:R, :C]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _hidden(gen, T, cols):
    """Hidden states: normal, with a few columns that are far larger, as a model's residual stream has."""
    x = torch.randn(T, cols, generator=gen, device=DEV)
    loud = torch.rand(cols, generator=gen, device=DEV) < 0.004
    return x * torch.where(loud, 24.0, 1.0)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, T, cols = case["op"], case["T"], case["cols"]
    blocks = -(-cols // BLOCK)
    st = {"op": op}

    def u8(*shape):
        return torch.empty(*shape, dtype=torch.uint8, device=DEV)

    if op == "store":
        act = getattr(torch, case["act"])
        st["x"] = _hidden(gen, T, cols).to(act)
        st["q"], st["scale"], st["back"] = u8(T, cols), u8(T, blocks), torch.empty(T, cols, dtype=act, device=DEV)
    elif op in ("compose_fwd", "compose_bwd"):
        act, r = getattr(torch, case["act"]), case["r"]
        st["s"] = torch.tensor(32.0 / math.sqrt(r), dtype=torch.float32).item()
        st["g"] = 1.0 + 0.01 * torch.randn(cols, generator=gen, device=DEV)
        base = torch.randn(T, cols, generator=gen, device=DEV).to(act)
        lora = (0.01 * math.sqrt(r) * torch.randn(T, cols, generator=gen, device=DEV)).to(act)
        if op == "compose_fwd":
            st["base"], st["lora"] = base, lora
            st["q"], st["scale"] = u8(T, cols), u8(T, blocks)
            st["y"], st["v"] = torch.empty_like(base), torch.empty_like(base)
        else:
            st["q"], st["scale"] = _quantize(base.float() + st["s"] * lora.float())
            st["norm"] = 0.5 + torch.rand(cols, generator=gen, device=DEV)
            st["dy"] = torch.randn(T, cols, generator=gen, device=DEV).to(act)
            st["d_base"], st["d_lora"] = torch.empty_like(base), torch.empty_like(base)
            st["d_mag"] = torch.empty(cols, device=DEV)
    elif op == "lora_grad":
        r = case["r"]
        st["q"], st["scale"] = _quantize(_hidden(gen, T, cols))
        st["dxa"] = torch.randn(T, r, generator=gen, device=DEV).bfloat16()
        st["dA"] = torch.empty(r, cols, device=DEV)
    else:
        out = case["out"]
        W = torch.randn(out, cols, generator=gen, device=DEV) / math.sqrt(cols)
        st["wq"], st["wscale"] = _quantize(W, BLOCK)
        wide = cols if op == "matmul" else out
        x = _hidden(gen, T, wide) if op == "matmul" else torch.randn(T, wide, generator=gen, device=DEV)
        st["q"], st["scale"] = _quantize(x)
        st["y"] = torch.empty(T, out if op == "matmul" else cols, dtype=torch.bfloat16, device=DEV)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _plain(st):
    op = st["op"]
    if op == "store":
        return {"x": _dequantize(*_quantize(st["x"].float())).to(st["x"].dtype)}
    if op == "compose_fwd":
        act, s, g = st["base"].dtype, st["s"], st["g"]
        base, lora = st["base"].float(), st["lora"].float()
        y = base + ((g - 1.0) * base + g * s * lora)
        v = _dequantize(*_quantize(base + s * lora))
        return {"y": y.to(act), "v": v.to(act)}
    if op == "compose_bwd":
        dy, g, s = st["dy"].float(), st["g"], st["s"]
        d_mag = (dy * _dequantize(st["q"], st["scale"])).sum(0) / st["norm"]
        act = st["dy"].dtype
        return {"d_base": (g * dy).to(act), "d_lora": (g * s * dy).to(act), "d_mag": d_mag}
    x = _dequantize(st["q"], st["scale"])
    if op == "lora_grad":
        return {"dA": st["dxa"].float().t() @ x}
    W = _dequantize(st["wq"], st["wscale"], BLOCK)
    return {"y": (x @ (W.t() if op == "matmul" else W)).bfloat16()}


def _library(st):
    import parameter_efficient_fine_gb300 as dora
    op = st["op"]
    if op == "store":
        dora.dora_q8_store(st["x"], 1, st["q"], st["scale"])
        dora.dora_q8_load(st["q"], st["scale"], 1, st["back"])
        return {"x": st["back"]}
    if op == "compose_fwd":
        dora.dora_compose_fwd_q8(st["base"], st["lora"], st["g"], st["s"], st["y"], st["q"], st["scale"])
        dora.dora_q8_load(st["q"], st["scale"], 1, st["v"])
        return {"y": st["y"], "v": st["v"]}
    ws = st.get("workspace")
    if ws is None:      # the call's scratch memory, kept beside its other buffers
        T, cols = st["q"].shape
        if op == "compose_bwd":
            n = dora.dora_compose_bwd_q8_workspace(T, cols)
        elif op == "lora_grad":
            n = dora.dora_lora_grad_q8_workspace(T, cols, st["dxa"].shape[1])
        else:
            out, inp = st["wq"].shape
            n = dora.dora_matmul_q8_workspace(T, out, inp) if op == "matmul" else dora.dora_matmul_q8_t_workspace(T, out, inp)
        ws = st["workspace"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    if op == "compose_bwd":
        dora.dora_compose_bwd_q8(st["dy"], st["q"], st["scale"], st["g"], st["norm"], st["s"],
                                 st["d_base"], st["d_lora"], st["d_mag"], ws)
        return {"d_base": st["d_base"], "d_lora": st["d_lora"], "d_mag": st["d_mag"]}
    if op == "lora_grad":
        dora.dora_lora_grad_q8(st["dxa"], st["q"], st["scale"], st["dA"], ws)
        return {"dA": st["dA"]}
    call = dora.dora_matmul_q8 if op == "matmul" else dora.dora_matmul_q8_t
    call(st["q"], st["scale"], st["wq"], st["wscale"], st["y"], ws)
    return {"y": st["y"]}


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, T, C = case["op"], case["T"], case["cols"]
    form = lambda R, K, rows=1: R * K + -(-R // rows) * -(-K // BLOCK)  # noqa: E731
    e = {"bfloat16": 2, "float32": 4}.get(case.get("act"), 2)
    if op == "store":            # x in, the 8-bit form out and in again, x back out
        return {"bytes": 2 * e * T * C + 2 * form(T, C), "flops": 3 * T * C}
    if op == "compose_fwd":      # base, lora in; y and the 8-bit v out; v in again and out
        return {"bytes": 4 * e * T * C + 2 * form(T, C) + 4 * C, "flops": 9 * T * C}
    if op == "compose_bwd":      # dy and the 8-bit v in; d_base and d_lora out
        return {"bytes": 3 * e * T * C + form(T, C) + 12 * C, "flops": 5 * T * C}
    if op == "lora_grad":
        r = case["r"]
        return {"bytes": form(T, C) + 2 * T * r + 4 * r * C, "flops": 2 * T * C * r}
    out = case["out"]
    k, n = (C, out) if op == "matmul" else (out, C)
    return {"bytes": form(T, k) + form(out, C, BLOCK) + 2 * T * n, "flops": 2 * T * out * C}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _e4m3_table():
    """The value of each E4M3 byte: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f is NaN, no infinities."""
    t = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = math.nan if (b & 127) == 127 else (1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6
        t.append(-v if b & 128 else v)
    return torch.tensor(t, dtype=torch.float64, device=DEV)


def _two_to(k):
    """2^k for an integer tensor, exactly (a normal float64)."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _exact_values(q, scale, rows):
    """What an 8-bit form stands for."""
    v = _e4m3_table()[q.long()] if q.numel() < 1 << 26 else torch.cat([_e4m3_table()[p.long()] for p in q.split(512)])
    s = _two_to(scale.long() - 127).repeat_interleave(rows, 0).repeat_interleave(BLOCK, 1)
    return v.mul_(s[: q.shape[0], : q.shape[1]])


def _exact_store(x):
    """The nearest values of the 8-bit form to a float64 matrix, ties to even; one scale per 128 columns."""
    out = torch.empty_like(x)
    for c in range(0, x.shape[1], BLOCK):
        b = x[:, c:c + BLOCK]
        top = b.abs().amax(1, keepdim=True)
        m, e = torch.frexp(top)                     # top = m 2^e, m in [0.5, 1)
        k = torch.where(m > 0.875, e - 8, e - 9)    # 448 = 0.875 * 2^9
        k = torch.where(top == 0, torch.full_like(k, -117), k).clamp(min=-117)
        u = b * _two_to(-k)
        step = _two_to((torch.frexp(u)[1] - 1).clamp(min=-6) - 3)
        out[:, c:c + BLOCK] = torch.round(u / step) * step * _two_to(k)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "store":
        return {"x": _exact_store(st["x"].double())}
    if op == "compose_fwd":
        base, lora, g = st["base"].double(), st["lora"].double(), st["g"].double()
        v = base + st["s"] * lora
        return {"y": g * v, "v": _exact_store(v)}
    if op == "compose_bwd":
        dy, g = st["dy"].double(), st["g"].double()
        d_mag = torch.einsum("tc,tc->c", dy, _exact_values(st["q"], st["scale"], 1)) / st["norm"].double()
        return {"d_base": g * dy, "d_lora": g * st["s"] * dy, "d_mag": d_mag}
    x = _exact_values(st["q"], st["scale"], 1)
    if op == "lora_grad":
        return {"dA": torch.einsum("tr,tc->rc", st["dxa"].double(), x)}
    W = _exact_values(st["wq"], st["wscale"], BLOCK)
    return {"y": torch.einsum("tk,nk->tn" if op == "matmul" else "tk,kn->tn", x, W)}
