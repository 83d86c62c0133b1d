"""Measured cases of the operators around the block-scaled GEMMs: the MoE
router, the MoE layer for a few tokens and the projection with low-rank
adapters.

``own`` false: the operators in plain torch, in 32 bits; ``own`` true: the
library's entry points.  Both take the state that ``prepare`` makes.
"""
import math

import torch

own = False

E4M3, E2M1 = 0, 2
F2 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

SOFTMAX, SOFTMAX_TOPK, SIGMOID, SIGMOID_NORM = 0, 1, 2, 3


def listed():
    return [
        # one token of a decode step chooses 2 of 8 experts: latency alone
        dict(name="route token", op="route", T=1, E=8, k=2, score=SOFTMAX_TOPK, bf16=False,
             ordered=False),
        # a decode batch over many experts, an odd number of tokens, bf16 logits
        dict(name="route batch", op="route", T=77, E=64, k=6, score=SIGMOID_NORM, bf16=True,
             ordered=True),
        # a long prompt's tokens, in the order the grouped GEMM takes
        dict(name="route prompt", op="route", T=32768, E=64, k=8, score=SOFTMAX, bf16=False,
             ordered=True),
        # one token through large experts: the weights of two of them
        dict(name="moe token", op="moe", T=1, E=8, k=2, H=4096, F=14336, fmt=E4M3),
        # a few tokens over many small experts, the sizes no multiple of a tile
        dict(name="moe small experts", op="moe", T=5, E=64, k=8, H=2080, F=1440, fmt=E4M3),
        # 4-bit weights
        dict(name="moe fp4", op="moe", T=16, E=32, k=4, H=4096, F=2048, fmt=E2M1),
        # a decode batch: every expert of the layer is used
        dict(name="moe batch", op="moe", T=64, E=8, k=2, H=4096, F=14336, fmt=E4M3),
        # one token with its adapter
        dict(name="lora token", op="lora", M=1, N=4096, K=4096, L=8, r=16, fmt=E4M3, runs=1),
        # a decode batch, each row its own request
        dict(name="lora batch", op="lora", M=33, N=4096, K=4096, L=16, r=16, fmt=E4M3, runs=33),
        # a full decode batch on a wide projection, higher rank
        dict(name="lora wide batch", op="lora", M=128, N=14336, K=4096, L=32, r=64, fmt=E4M3,
             runs=128),
        # the prompts of a few requests one after the other
        dict(name="lora prompt", op="lora", M=4099, N=14336, K=4096, L=8, r=16, fmt=E4M3, runs=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "moe", "lora"))
    if op == "route":
        E = rng.choice((8, 16, 33, 64))
        return dict(op=op, T=_log(rng, 1, 32768), E=E, k=rng.randint(1, 8), score=rng.randint(0, 3),
                    bf16=rng.random() < 0.5, ordered=rng.random() < 0.6)
    fmt = rng.choice((E4M3, E4M3, E2M1))
    unit = 128 if fmt == E2M1 else 32
    if op == "moe":
        E = rng.choice((4, 8, 16, 32, 64))
        H = unit * (_log(rng, 512, 4096) // unit)
        # experts of at most 1.4 G weights together, the largest listed layer's
        F = unit * max(1, min(_log(rng, 256, 14336), 1409286144 // (3 * E * H)) // unit)
        return dict(op=op, T=_log(rng, 1, 64), E=E, k=rng.randint(1, min(8, E)), H=H, F=F, fmt=fmt)
    M = _log(rng, 1, 4099)
    N = 8 * (_log(rng, 512, 14336) // 8)
    K = unit * (_log(rng, 512, 4096) // unit)
    runs = M if M <= 128 and rng.random() < 0.7 else min(M, rng.randint(1, 8))
    return dict(op=op, M=M, N=N, K=K, L=rng.choice((1, 4, 8, 32)), r=rng.choice((8, 16, 32, 64)),
                fmt=fmt, runs=runs)


# ------------------------------------------------------------------- inputs

def _codes(w, fmt):
    """Weights [rows, K] fp32 -> (uint8 codes, fp32 1x32 power-of-two scales)."""
    b = w.view(w.shape[0], -1, 32)
    top, emax = (1.75, 8) if fmt == E4M3 else (1.5, 2)
    m, e = torch.frexp(b.abs().amax(-1))
    e = torch.where(m == 0, 0, e - 1 - emax + (2 * m > top).int())
    s = torch.ldexp(torch.ones_like(m), e)
    v = (b / s[..., None]).view(w.shape)
    if fmt == E4M3:
        return v.to(torch.float8_e4m3fn).view(torch.uint8), s
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    q = torch.bucketize(v.abs(), edges, out_int32=True).to(torch.uint8) + (v < 0).to(torch.uint8) * 8
    return q[:, 0::2] | (q[:, 1::2] << 4), s


def _weights(n, rows, K, fmt, gen):
    """n matrices [rows, K]: codes and scales [n, rows, K/32]."""
    codes = torch.empty((n, rows, K if fmt == E4M3 else K // 2), dtype=torch.uint8, device="cuda")
    sf = torch.empty((n, rows, K // 32), device="cuda")
    for i in range(n):
        w = torch.randn((rows, K), device="cuda", generator=gen) * (K ** -0.5)
        codes[i], sf[i] = _codes(w, fmt)
    return codes, sf


def _pack(sf):
    """Scales laid out once for the weights' life (the library's pack_scales):
    fp32 scales [n, rows, K/32] -> uint8 [n, ceil(K/128), ceil(rows/128), 512]:
    byte 16 d + 4 w + j of a chunk is the exponent code of row 32 w + d, block j."""
    n, rows, kb = sf.shape
    nk, nr = -(-kb // 4), -(-rows // 128)
    c = torch.full((n, nr * 128, nk * 4), 127, dtype=torch.uint8, device=sf.device)
    c[:, :rows, :kb] = (sf.view(torch.int32) >> 23).to(torch.uint8)
    return c.view(n, nr, 4, 32, nk, 4).permute(0, 4, 1, 3, 2, 5).reshape(n, nk, nr, 512).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c, s = case, dict(case)
    if c["op"] == "route":
        x = torch.randn((c["T"], c["E"]), device="cuda", generator=gen) * 2
        if c["T"] > 8:  # masked experts, a token with fewer experts than k, one with none
            x[3, 1:] = -math.inf
            x[5] = -math.inf
            x[6, 0] = x[6, 1]
        s["logits"] = x.bfloat16() if c["bf16"] else x
        return s
    if c["op"] == "moe":
        T, E, k, H, F = c["T"], c["E"], c["k"], c["H"], c["F"]
        p = torch.randn((T, E), device="cuda", generator=gen) * 1.5
        v, i = torch.sort(p, dim=1, descending=True)
        s["ids"] = i[:, :k].int().contiguous()
        s["weights"] = torch.softmax(v[:, :k], 1).contiguous()
        if T > 8:  # padding tokens of the batch, and a choice that is not served here
            s["ids"][7] = -1
            s["ids"][2, 0] = -1
        s["x"] = torch.randn((T, H), device="cuda", generator=gen).bfloat16()
        s["W13"], s13 = _weights(E, 2 * F, H, c["fmt"], gen)
        s["W2"], s2 = _weights(E, H, F, c["fmt"], gen)
        s["s13"], s["s2"] = s13, s2
        # gate and up halves are packed as matrices of their own
        s["p13"], s["p2"] = _pack(s13.view(2 * E, F, H // 32)), _pack(s2)
        return s
    M, N, K, L, r = c["M"], c["N"], c["K"], c["L"], c["r"]
    s["x"] = torch.randn((M, K), device="cuda", generator=gen).bfloat16()
    W, sf = _weights(1, N, K, c["fmt"], gen)
    s["W"], s["sf"], s["pw"] = W[0], sf[0], _pack(sf)[0]
    s["A"] = (torch.randn((L, r, K), device="cuda", generator=gen) * K ** -0.5).bfloat16()
    s["B"] = (torch.randn((L, N, r), device="cuda", generator=gen) * 0.3).bfloat16()
    s["alpha"] = torch.rand((L,), device="cuda", generator=gen) + 0.5
    # requests one after the other, each with its adapter or none
    who = torch.randint(0, L + 1, (c["runs"],), device="cuda", generator=gen) - 1
    if c["runs"] == 1:
        who = who.clamp(min=0)
    at = torch.arange(M, device="cuda") * c["runs"] // M
    s["adapter"] = who[at].int()
    return s


# --------------------------------------------------------------- plain forms

def _fake_quant(x):
    """E4M3 with 1x32 power-of-two scales, back in fp32."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    m, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    e = torch.where(m == 0, 0, e - 1 - 8 + (2 * m > 1.75).int()).clamp(-126, 127)
    q = torch.ldexp(b, -e).to(torch.float8_e4m3fn).float()
    return torch.ldexp(q, e).reshape(x.shape)


def _dequant(codes, sf, fmt):
    if fmt == E4M3:
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        lut = torch.tensor(F2 + tuple(-f for f in F2), device=codes.device)
        v = lut[torch.stack((codes & 15, codes >> 4), -1).int()].flatten(-2)
    return (v.reshape(*sf.shape, 32) * sf[..., None]).reshape(v.shape)


def _plain_route(s):
    T, E, k = s["T"], s["E"], s["k"]
    x = s["logits"].float()
    x = torch.where(torch.isnan(x), -math.inf, x)
    v, i = torch.sort(x, dim=1, descending=True, stable=True)
    v, i = v[:, :k], i[:, :k]
    on = v > -math.inf
    top = torch.where(on[:, :1], v[:, :1], 0.0)
    if s["score"] in (SOFTMAX, SOFTMAX_TOPK):
        w = torch.exp(v - top)
        total = torch.exp(x - top) if s["score"] == SOFTMAX else w
        w = w / total.sum(1, keepdim=True)
    else:
        w = 1 / (1 + torch.exp(-v))
        if s["score"] == SIGMOID_NORM:
            w = w / w.sum(1, keepdim=True)
    ids = torch.where(on, i, -1).int()
    out = [ids, torch.where(on, w, 0.0) * 1.5]
    if s["ordered"]:
        flat = torch.where(on, i, E).reshape(-1)
        order = torch.argsort(flat, stable=True)
        live = flat[order] < E
        out.append((flat[:, None] == torch.arange(E, device=x.device)).sum(0).int())
        out.append(torch.where(live, order // k, -1).int())
        out.append(torch.where(live, order, -1).int())
    return out


def _plain_moe(s):
    T, E, k, F = s["T"], s["E"], s["k"], s["F"]
    x = _fake_quant(s["x"].float())
    ids = s["ids"].long()
    on = ids >= 0
    if T * k < E:  # the chosen experts, row by row
        pick = ids.clamp(min=0).reshape(-1)
        W13, W2 = (_dequant(s[a][pick], s[b][pick], s["fmt"]) for a, b in (("W13", "s13"), ("W2", "s2")))
        xe = x.repeat_interleave(k, 0)[:, None]                       # [T k, 1, H]
        wt = torch.where(on, s["weights"], 0.0).reshape(-1, 1, 1)
    else:  # every expert on every token, the unchosen ones weighted zero
        W13, W2 = _dequant(s["W13"], s["s13"], s["fmt"]), _dequant(s["W2"], s["s2"], s["fmt"])
        xe = x[None].expand(E, -1, -1)                                # [E, T, H]
        hot = (ids[..., None] == torch.arange(E, device=x.device)) * s["weights"][..., None]
        wt = hot.sum(1).t()[..., None]                                # [E, T, 1]
    gu = torch.bmm(xe, W13.transpose(1, 2))
    g, u = gu[..., :F], gu[..., F:]
    h = _fake_quant(g / (1 + torch.exp(-g)) * u)
    y = torch.bmm(h, W2.transpose(1, 2)) * wt
    y = y.reshape(T, k, -1).sum(1) if T * k < E else y.sum(0)
    return y.bfloat16()


def _plain_lora(s):
    M, L, r = s["M"], s["L"], s["r"]
    x = s["x"].float()
    y = _fake_quant(x) @ _dequant(s["W"], s["sf"], s["fmt"]).t()
    v = (x @ s["A"].float().reshape(L * r, -1).t()).view(M, L, r)
    hot = (s["adapter"].long()[:, None] == torch.arange(L, device=x.device)) * s["alpha"]
    v = (v * hot[..., None]).reshape(M, L * r)
    return (y + v @ s["B"].float().permute(0, 2, 1).reshape(L * r, -1)).bfloat16()


def run(state):
    s = state
    if not own:
        return {"route": _plain_route, "moe": _plain_moe, "lora": _plain_lora}[s["op"]](s)
    import fp8_block_scaled_06_gb300 as fp8g
    if s["op"] == "route":
        return fp8g.moe_route(s["logits"], s["k"], score=s["score"], scale=1.5, ordered=s["ordered"])
    if s["op"] == "moe":
        return fp8g.moe_layer(s["x"], s["ids"], s["weights"], s["W13"], s["p13"], s["W2"], s["p2"],
                              w_fmt=s["fmt"])
    return fp8g.gemm_lora(s["x"], s["W"], s["pw"], s["A"], s["B"], s["alpha"], s["adapter"],
                          w_fmt=s["fmt"])


def work(case):
    c = case
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        out = 8 * T * k + (8 * T * k + 4 * E if c["ordered"] else 0)
        return {"bytes": T * E * (2 if c["bf16"] else 4) + out, "flops": 2 * T * E}
    wb = (1 if c["fmt"] == E4M3 else 0.5) + 1 / 32
    if c["op"] == "moe":
        T, E, k, H, F = c["T"], c["E"], c["k"], c["H"], c["F"]
        used = E * (1 - (1 - k / E) ** T)  # experts that T independent choices of k use
        return {"bytes": used * 3 * F * H * wb + 4 * T * H + 8 * T * k,
                "flops": 6 * T * k * F * H}
    M, N, K, L, r = c["M"], c["N"], c["K"], c["L"], c["r"]
    used = L * (1 - (1 - 1 / L) ** (c["runs"] * L / (L + 1)))
    return {"bytes": N * K * wb + used * r * (N + K) * 2 + 2 * M * (K + N) + 4 * M,
            "flops": 2 * M * N * K + 2 * M * r * (N + K)}


# ------------------------------------------------------- definitions, 64 bits

def _round_e4m3(v):
    """Nearest E4M3 value (even ties) of |v| <= 448, in 64 bits."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), e.clamp(min=-5) - 4)  # 3 fraction bits, least exponent -6
    return torch.round(v / step) * step


def _quant64(x):
    rows = x.reshape(-1, 32)
    top = rows.abs().amax(1)
    e = torch.ceil(torch.log2(top / 448))
    e = torch.where(top == 0, 0.0, e).clamp(-126, 127)
    e = torch.where((torch.exp2(e - 1) * 448 >= top) & (top > 0), e - 1, e)
    s = torch.exp2(e)[:, None]
    return (_round_e4m3(rows / s) * s).reshape(x.shape)


def _matrix64(codes, sf, fmt):
    values = []
    for c in range(256 if fmt == E4M3 else 16):
        if fmt == E4M3:
            e, m = (c >> 3) & 15, c & 7
            v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
            values.append(-v if c & 128 else v)
        else:
            values.append(F2[c & 7] * (-1 if c & 8 else 1))
    table = torch.tensor(values, dtype=torch.float64, device=codes.device)
    if fmt != E4M3:
        codes = torch.stack((codes % 16, codes // 16), 2).reshape(codes.shape[0], -1)
    return table[codes.int()] * sf.double().repeat_interleave(32, 1)


def _exact_route(s):
    x = s["logits"].double().cpu()
    T, E = x.shape
    k, rows = s["k"], []
    x = torch.nan_to_num(x, nan=-math.inf, posinf=math.inf, neginf=-math.inf)
    order = torch.from_numpy((-x).numpy().argsort(axis=1, kind="stable"))[:, :k]
    v = torch.gather(x, 1, order)
    on = torch.isfinite(v)
    if s["score"] == SOFTMAX:
        w = torch.exp(v - torch.logsumexp(x, 1, keepdim=True))
    elif s["score"] == SOFTMAX_TOPK:
        w = torch.exp(v - torch.logsumexp(v, 1, keepdim=True))
    else:
        w = torch.sigmoid(v)
        if s["score"] == SIGMOID_NORM:
            w = w / w.sum(1, keepdim=True)
    out = [None, torch.where(on, w * 1.5, torch.zeros((), dtype=torch.float64))]
    return out + ([None] * 3 if s["ordered"] else [])


def _exact_moe(s):
    T, k, H, F = s["T"], s["k"], s["H"], s["F"]
    x = _quant64(s["x"].double())
    ids = s["ids"].cpu()
    out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in range(s["E"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not len(t):
            continue
        t, j = t.cuda(), j.cuda()
        gu = x[t] @ _matrix64(s["W13"][e], s["s13"][e], s["fmt"]).t()
        g = gu[:, :F]
        h = _quant64(g * torch.sigmoid(g) * gu[:, F:])
        y = h @ _matrix64(s["W2"][e], s["s2"][e], s["fmt"]).t()
        out.index_add_(0, t, y * s["weights"][t, j].double()[:, None])
    return out


def _exact_lora(s):
    x = s["x"].double()
    y = _quant64(x) @ _matrix64(s["W"], s["sf"], s["fmt"]).t()
    for n in range(s["L"]):
        i = torch.nonzero(s["adapter"] == n)[:, 0]
        y[i] += s["alpha"][n].double() * ((x[i] @ s["A"][n].double().t()) @ s["B"][n].double().t())
    return y


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "moe": _exact_moe, "lora": _exact_lora}[case["op"]](s)
