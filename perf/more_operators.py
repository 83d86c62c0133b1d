"""Measured cases of the 8-bit feed-forward path with scales for blocks of 128:
the quantiser, the product in its three forms (output, input gradient, weight
gradient), the gated projection pair and the gated backward pass from 8-bit
checkpoints.

``own`` false: the operators in plain torch, in 32 bits; ``own`` true: the
library's entry points.  Both take the state that ``prepare`` makes.

Codes are E4M3 or E5M2.  Scales are fp32: one for 128 consecutive values of a row
("row", laid out [blocks of the row, rows]), for 128 values of a column ("col",
[blocks of the column, columns]) or for a 128 x 128 tile ("tile", [blocks of rows,
blocks of columns]).  Blocks at an edge are cut short.
"""
import math

import torch

own = False

E4M3, E5M2 = 0, 1
TOP = (448.0, 57344.0)
TYPE = (torch.float8_e4m3fn, torch.float8_e5m2)
SILU, GELU, RELU = 0, 1, 2


def listed():
    return [
        # a decode step's one token before a projection: latency alone
        dict(name="quantize token", op="quantize", R=1, C=4096, source="bf16", fmt=E4M3, row=True, col=False),
        # a prompt's output gradient, for the input gradient and for the weight gradient in one
        # reading; an odd number of tokens
        dict(name="quantize gradient", op="quantize", R=4099, C=14336, source="bf16", fmt=E4M3, row=True, col=True),
        # the 8-bit input that the forward pass kept, turned for the weight gradient
        dict(name="quantize checkpoint", op="quantize", R=8192, C=4096, source="codes", fmt=E4M3, row=False, col=True),
        # one token through the down projection
        dict(name="product token", op="product", form="nt", M=1, N=4096, K=14336, a=E4M3, b=E4M3, f32=False, add=False),
        # a decode batch, no multiple of a tile
        dict(name="product batch", op="product", form="nt", M=77, N=14336, K=4096, a=E4M3, b=E4M3, f32=False, add=False),
        # a prompt through the down projection
        dict(name="product prompt", op="product", form="nt", M=4099, N=4096, K=14336, a=E4M3, b=E4M3, f32=False, add=False),
        # the gradient of a gated projection pair's input: wide-range codes against the weights as they lie
        dict(name="product input gradient", op="product", form="nn", M=4099, N=4096, K=28672, a=E5M2, b=E4M3, f32=False, add=False),
        # a weight gradient over an odd number of tokens, added to the sum so far
        dict(name="product weight gradient", op="product", form="tn", M=4096, N=14336, K=4099, a=E4M3, b=E4M3, f32=True, add=True),
        # one token through gate and up
        dict(name="gated token", op="gated", M=1, F=14336, K=4096, gate=SILU, keep=False),
        # a training step's prompt, gate and up kept in 8 bits for the backward pass
        dict(name="gated prompt", op="gated", M=4099, F=14336, K=4096, gate=SILU, keep=True),
        # a small layer's backward pass
        dict(name="backward small", op="backward", M=77, F=1408, gate=GELU, fmt=E4M3, f32=True),
        # a training step's
        dict(name="backward prompt", op="backward", M=4099, F=14336, gate=SILU, fmt=E4M3, f32=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _unit(rng, unit, lo, hi):
    return unit * max(1, _log(rng, lo, hi) // unit)


def draw(rng):
    op = rng.choice(("quantize", "product", "product", "gated", "backward"))
    if op == "quantize":
        row = rng.random() < 0.6
        source = rng.choice(("bf16", "bf16", "f32", "codes"))
        return dict(op=op, R=_log(rng, 1, 8192), C=_unit(rng, 16, 128, 7168), source=source,
                    fmt=rng.choice((E4M3, E4M3, E5M2)), row=row and source != "codes",
                    col=not row or source == "codes" or rng.random() < 0.5)
    if op == "product":
        form = rng.choice(("nt", "nt", "nn", "tn"))
        tokens, N, K = _log(rng, 1, 4099), _unit(rng, 16, 256, 7168), _unit(rng, 16, 256, 7168)
        a, b = rng.choice(((E4M3, E4M3), (E4M3, E4M3), (E5M2, E4M3), (E4M3, E5M2)))
        f32 = rng.random() < (0.8 if form == "tn" else 0.3)
        M, K = (K, tokens) if form == "tn" else (tokens, K)
        return dict(op=op, form=form, M=M, N=N, K=K, a=a, b=b, f32=f32, add=f32 and rng.random() < 0.5)
    if op == "gated":
        return dict(op=op, M=_log(rng, 1, 4099), F=_unit(rng, 128, 256, 7168), K=_unit(rng, 16, 256, 4096),
                    gate=rng.randint(0, 2), keep=rng.random() < 0.5)
    return dict(op=op, M=_log(rng, 1, 4099), F=_unit(rng, 128, 256, 14336), gate=rng.randint(0, 2),
                fmt=rng.choice((E4M3, E5M2)), f32=rng.random() < 0.3)


# ------------------------------------------------------------ the 8-bit format

def _blocks(x, block):
    """x [R, C] fp32, padded with zeros to whole blocks, as [R blocks, block rows, C blocks, block columns]."""
    h, w = {"row": (1, 128), "col": (128, 1), "tile": (128, 128)}[block]
    R, C = x.shape
    x = torch.nn.functional.pad(x, (0, -C % w, 0, -R % h))
    return x.view(x.shape[0] // h, h, x.shape[1] // w, w)


def _spread(s, block, R, C):
    """Scales as they are laid out -> one for each value [R, C]."""
    if block == "row":
        return s.t().repeat_interleave(128, 1)[:, :C]
    s = s.repeat_interleave(128, 0)[:R]
    return s if block == "col" else s.repeat_interleave(128, 1)[:, :C]


def _quant(x, block, fmt):
    """x [R, C] fp32 -> (codes uint8 [R, C], scales): scale = amax / largest value of the
    format (1 for a block of zeros), code = the nearest to x times the scale's reciprocal."""
    R, C = x.shape
    v = _blocks(x, block)
    s = v.abs().amax((1, 3)) / TOP[fmt]
    s = torch.where(s == 0, 1.0, s.clamp(min=2.0 ** -126))
    v = (v * (1 / s)[:, None, :, None]).view(v.shape[0] * v.shape[1], -1)[:R, :C]
    q = v.clamp(-TOP[fmt], TOP[fmt]).to(TYPE[fmt]).view(torch.uint8)
    return q.contiguous(), (s.t() if block == "row" else s).contiguous()


def _values(q, s, block, fmt):
    return q.view(TYPE[fmt]).float() * _spread(s, block, *q.shape)


# ------------------------------------------------------------------- inputs

def _activations(R, C, gen):
    """Rows of different size, a few large values among them, and a run of zeros (padding tokens)."""
    x = torch.randn((R, C), device="cuda", generator=gen)
    x *= torch.exp(torch.randn((R, 1), device="cuda", generator=gen))
    x *= 1 + 30 * (torch.rand((R, C), device="cuda", generator=gen) < 0.001)
    if R > 8:
        x[3:5] = 0
    return x


def _weights(N, K, gen):
    w = torch.randn((N, K), device="cuda", generator=gen) * K ** -0.5
    return w * torch.exp(0.5 * torch.randn((N, 1), device="cuda", generator=gen))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c, s = case, dict(case)
    if c["op"] == "quantize":
        x = _activations(c["R"], c["C"], gen)
        if c["source"] == "codes":
            s["q"], s["s"] = _quant(x, "row", E4M3)
        else:
            s["x"] = x.bfloat16() if c["source"] == "bf16" else x
    elif c["op"] == "product":
        M, N, K, form = c["M"], c["N"], c["K"], c["form"]
        if form == "tn":  # both [tokens, features], blocks along the tokens
            s["A"], s["sa"] = _quant(_activations(K, M, gen), "col", c["a"])
            s["B"], s["sb"] = _quant(_activations(K, N, gen), "col", c["b"])
        else:
            s["A"], s["sa"] = _quant(_activations(M, K, gen), "row", c["a"])
            s["B"], s["sb"] = _quant(_weights(*((N, K) if form == "nt" else (K, N)), gen), "tile", c["b"])
        if c["add"]:
            s["C"] = torch.randn((M, N), device="cuda", generator=gen) * K ** 0.5
    elif c["op"] == "gated":
        s["x"], s["sx"] = _quant(_activations(c["M"], c["K"], gen), "row", E4M3)
        s["W"], s["sw"] = _quant(_weights(2 * c["F"], c["K"], gen), "tile", E4M3)
    else:
        s["gu"], s["sgu"] = _quant(_activations(c["M"], 2 * c["F"], gen), "row", E4M3)
        dh = _activations(c["M"], c["F"], gen) * 1e-3
        s["dh"] = dh if c["f32"] else dh.bfloat16()
    return s


# --------------------------------------------------------------- plain forms

def _act(g, gate):
    """The gate's value and derivative."""
    if gate == SILU:
        y = 1 / (1 + torch.exp(-g))
        return g * y, y * (1 + g * (1 - y))
    if gate == GELU:
        y = 0.5 * (1 + torch.erf(g * 0.5 ** 0.5))
        return g * y, y + g * torch.exp(-0.5 * g * g) * (2 * math.pi) ** -0.5
    return g.clamp(min=0), (g > 0).to(g.dtype)


def _coded(pairs, fmt):
    """(codes, scales) pairs as what run() returns: the codes as the values they stand for, beside their scales."""
    return [t for q, s in pairs for t in (q.view(TYPE[fmt]), s)]


def _plain(s):
    if s["op"] == "quantize":
        x = _values(s["q"], s["s"], "row", E4M3) if s["source"] == "codes" else s["x"].float()
        return _coded([_quant(x, b, s["fmt"]) for b in ("row", "col") if s[b]], s["fmt"])
    if s["op"] == "product":
        form, f32 = s["form"], s["f32"]
        A = _values(s["A"], s["sa"], "col" if form == "tn" else "row", s["a"])
        B = _values(s["B"], s["sb"], "col" if form == "tn" else "tile", s["b"])
        C = (A.t() if form == "tn" else A) @ (B.t() if form == "nt" else B)
        if s["add"]:
            return s["C"].add_(C)
        return C if f32 else C.bfloat16()
    F = s["F"]
    if s["op"] == "gated":
        gu = _values(s["x"], s["sx"], "row", E4M3) @ _values(s["W"], s["sw"], "tile", E4M3).t()
        h = _act(gu[:, :F], s["gate"])[0] * gu[:, F:]
        return _coded([_quant(v, "row", E4M3) for v in ((h, gu) if s["keep"] else (h,))], E4M3)
    gu, dh = _values(s["gu"], s["sgu"], "row", E4M3), s["dh"].float()
    g, u = gu[:, :F], gu[:, F:]
    y, d = _act(g, s["gate"])
    dgu = torch.cat((dh * u * d, dh * y), 1)
    return (_coded([_quant(dgu, "row", s["fmt"]), _quant(dgu, "col", s["fmt"])], s["fmt"])
            + _coded([_quant(y * u, "col", E4M3)], E4M3))


def run(state):
    s = state
    if not own:
        return _plain(s)
    import fp8_block_scaled_06_gb300 as fp8g
    if s["op"] == "quantize":
        if s["source"] == "codes":
            return _coded([fp8g.requantize_block128(s["q"], s["s"], fmt=s["fmt"])], s["fmt"])
        got = fp8g.quantize_block128(s["x"], row=s["row"], col=s["col"], fmt=s["fmt"])
        return _coded([p for p in got if p is not None], s["fmt"])
    if s["op"] == "product":
        return fp8g.gemm_block128(s["A"], s["sa"], s["B"], s["sb"], form=s["form"], a_fmt=s["a"], b_fmt=s["b"],
                                  out="f32" if s["f32"] else "bf16", add_to=s.get("C"))
    if s["op"] == "gated":
        h, gu = fp8g.gated_block128(s["x"], s["sx"], s["W"], s["sw"], gate=s["gate"], keep=s["keep"])
        return _coded([h, gu] if s["keep"] else [h], E4M3)
    row, col, h = fp8g.gated_block128_backward(s["dh"], s["gu"], s["sgu"], gate=s["gate"], fmt=s["fmt"])
    return _coded([row, col], s["fmt"]) + _coded([h], E4M3)


def work(case):
    c = case

    def up(n):
        return -(-n // 128)

    if c["op"] == "quantize":
        R, C = c["R"], c["C"]
        there = {"bf16": 2 * R * C, "f32": 4 * R * C, "codes": R * C + 4 * R * up(C)}[c["source"]]
        back = c["row"] * (R * C + 4 * R * up(C)) + c["col"] * (R * C + 4 * up(R) * C)
        return {"bytes": there + back, "flops": 4 * R * C}
    if c["op"] == "product":
        M, N, K = c["M"], c["N"], c["K"]
        scales = 4 * up(K) * (M + (N if c["form"] == "tn" else up(N)))
        return {"bytes": K * (M + N) + scales + M * N * (8 if c["add"] else 4 if c["f32"] else 2), "flops": 2 * M * N * K}
    M, F = c["M"], c["F"]
    if c["op"] == "gated":
        K = c["K"]
        out = (3 if c["keep"] else 1) * M * (F + 4 * up(F))
        return {"bytes": K * (M + 2 * F) + 4 * up(K) * (M + 2 * up(F)) + out, "flops": 4 * M * F * K}
    reads = M * F * ((4 if c["f32"] else 2) + 2) + 8 * M * up(F)
    return {"bytes": reads + 5 * M * F + 8 * M * up(F) + 12 * up(M) * F, "flops": 30 * M * F}


# ------------------------------------------------------- definitions, 64 bits

def _table(fmt):
    """The value of each code."""
    bits, bias = ((3, 7), (2, 15))[fmt]
    out = []
    for code in range(256):
        e, m = (code & 127) >> bits, code & ((1 << bits) - 1)
        v = math.ldexp(m, 1 - bias - bits) if e == 0 else math.ldexp((1 << bits) + m, e - bias - bits)
        if fmt == E4M3 and code & 127 == 127 or fmt == E5M2 and e == 31:
            v = math.nan if fmt == E4M3 or m else math.inf
        out.append(-v if code & 128 else v)
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def _decode(q, s, kind, fmt):
    v = _table(fmt)[q.int()]
    R, C = q.shape
    i, j = torch.arange(R, device="cuda"), torch.arange(C, device="cuda")
    if kind == "row":
        return v * s.double()[j // 128][:, i].t()
    return v * s.double()[i // 128][:, j if kind == "col" else j // 128]


def _code64(x, kind, fmt):
    """x in 64 bits -> (the values of its codes, its scales)."""
    if kind == "col":
        v, s = _code64(x.t(), "row", fmt)
        return v.t().contiguous(), s
    R, C = x.shape
    n = -(-C // 128)
    wide = torch.zeros((R, n * 128), dtype=torch.float64, device="cuda")
    wide[:, :C] = x
    wide = wide.reshape(R, n, 128)
    s = wide.abs().amax(2) / TOP[fmt]
    s[s == 0] = 1.0
    v = wide / s[:, :, None]
    bits, least = ((3, -6), (2, -14))[fmt]
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=least) - bits)
    v = (torch.round(v / step) * step).clamp(-TOP[fmt], TOP[fmt])
    return v.reshape(R, -1)[:, :C].contiguous(), s.t().contiguous()


def _gate64(g, gate):
    if gate == SILU:
        y = torch.sigmoid(g)
        return g * y, y + g * y * torch.sigmoid(-g)
    if gate == GELU:
        y = torch.special.ndtr(g)
        return g * y, y + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    return torch.relu(g), torch.heaviside(g, torch.zeros_like(g))


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "quantize":
        x = _decode(s["q"], s["s"], "row", E4M3) if s["source"] == "codes" else s["x"].double()
        return [t for k in ("row", "col") if s[k] for t in _code64(x, k, s["fmt"])]
    if s["op"] == "product":
        if s["form"] == "tn":
            C = _decode(s["A"], s["sa"], "col", s["a"]).t() @ _decode(s["B"], s["sb"], "col", s["b"])
        else:
            B = _decode(s["B"], s["sb"], "tile", s["b"])
            C = _decode(s["A"], s["sa"], "row", s["a"]) @ (B.t() if s["form"] == "nt" else B)
        return C + s["C"].double() if s["add"] else C
    F = s["F"]
    if s["op"] == "gated":
        x, W = _decode(s["x"], s["sx"], "row", E4M3), _decode(s["W"], s["sw"], "tile", E4M3)
        g, u = x @ W[:F].t(), x @ W[F:].t()
        out = list(_code64(_gate64(g, s["gate"])[0] * u, "row", E4M3))
        return out + list(_code64(torch.cat((g, u), 1), "row", E4M3)) if s["keep"] else out
    gu, dh = _decode(s["gu"], s["sgu"], "row", E4M3), s["dh"].double()
    y, d = _gate64(gu[:, :F], s["gate"])
    dgu = torch.cat((dh * gu[:, F:] * d, dh * y), 1)
    out = list(_code64(dgu, "row", s["fmt"])) + list(_code64(dgu, "col", s["fmt"]))
    return out + list(_code64(y * gu[:, F:], "col", E4M3))
