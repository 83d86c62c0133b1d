"""Plain references of the operators with scales for blocks of 128, in 64 bits
(the quantiser's in 32, bit for bit), and the tolerances that follow from them."""
import math

import torch

E4M3, E5M2 = 0, 1
TOP = (448.0, 57344.0)
DT = (torch.float8_e4m3fn, torch.float8_e5m2)
# a code is off by at most half a step: relative, and of the scale below the least normal
HALF = (2.0 ** -4, 2.0 ** -3)
SUB = (2.0 ** -10, 2.0 ** -17)


def up(n):
    return -(-n // 128)


def spread(s, kind, R, C):
    """Scales as laid out -> one for each value of [R, C]."""
    if kind == "row":
        return s.t().repeat_interleave(128, 1)[:, :C]
    s = s.repeat_interleave(128, 0)[:R]
    return s if kind == "col" else s.repeat_interleave(128, 1)[:, :C]


def decode(q, s, kind, fmt):
    """The values that codes and scales stand for, in 64 bits (exact)."""
    return q.view(DT[fmt]).double() * spread(s, kind, *q.shape).double()


def quant(x, kind, fmt):
    """The definition, operation by operation in fp32 (CPU): codes and scales bit for bit."""
    x = x.float()
    R, C = x.shape
    h, w = {"row": (1, 128), "col": (128, 1), "tile": (128, 128)}[kind]
    v = torch.nn.functional.pad(x, (0, -C % w, 0, -R % h))
    v = v.view(v.shape[0] // h, h, v.shape[1] // w, w)
    amax = torch.nan_to_num(v.abs(), nan=0.0, posinf=math.inf).amax((1, 3))
    s = amax / TOP[fmt]
    s = torch.where(amax == 0, torch.ones_like(s), s.clamp(min=2.0 ** -126))
    y = v * (1 / s)[:, None, :, None]
    y = y.reshape(v.shape[0] * h, -1)[:R, :C]
    q = y.clamp(-TOP[fmt], TOP[fmt]).to(DT[fmt]).view(torch.uint8).clone()
    q[y.isnan()] = 0x7F
    return q, (s.t() if kind == "row" else s).contiguous()


def product(A, B, form):
    """C and the sum of magnitudes, from operands in 64 bits."""
    f = {"nt": lambda a, b: a @ b.t(), "nn": lambda a, b: a @ b, "tn": lambda a, b: a.t() @ b}[form]
    return f(A, B), f(A.abs(), B.abs())


def sum_tol(K):
    """Relative to the sum of magnitudes: K products and as many additions in fp32 or better, the
    scales' product and each block's step into the sum, none off by more than 2^-23."""
    return (K + 3 * up(K) + 2) * 2.0 ** -23


def act(g, gate):
    """The gate's value and derivative."""
    if gate == 0:
        y = torch.sigmoid(g)
        return g * y, y * (1 + g * (1 - y))
    if gate == 1:
        c = torch.special.ndtr(g)
        return g * c, c + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    return g.clamp(min=0), (g > 0).double()


def assert_coded(q, s, kind, fmt, want, err):
    """Codes q with scales s stand for `want` (64 bits), each value of which may be off by err
    before it is coded: the scales by the largest err of their block, the values by half a step."""
    R, C = want.shape
    h, w = (1, 128) if kind == "row" else (128, 1)
    pad = lambda t: torch.nn.functional.pad(t, (0, -C % w, 0, -R % h)).view(up(R) if h > 1 else R, h, -1, w)
    amax, e = pad(want.abs()).amax((1, 3)), pad(err).amax((1, 3))
    if kind == "row":
        amax, e = amax.t(), e.t()
    assert s.shape == amax.shape
    # a block whose values are all no larger than their error may have come out as zeros
    zero = (amax <= e) & (s == 1)
    off = (s.double() - amax / TOP[fmt]).abs()
    ok = off <= e / TOP[fmt] + 2.0 ** -23 * amax / TOP[fmt] + 2.0 ** -126
    assert (ok | zero).all(), "scales"
    got = decode(q, s, kind, fmt)
    tol = err * (1 + HALF[fmt]) + HALF[fmt] * (1 + 2.0 ** -20) * want.abs() + SUB[fmt] * spread(s, kind, R, C).double()
    bad = (got - want).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} codes, worst at {bad.nonzero()[0].tolist()}"


def values(R, C, gen, zeros=True):
    """Rows of different size, a few outliers, a block of zeros."""
    x = torch.randn((R, C), generator=gen) * torch.exp(torch.randn((R, 1), generator=gen))
    x = x * (1 + 20 * (torch.rand((R, C), generator=gen) < 0.003))
    if zeros and R > 2:
        x[1, : min(C, 128)] = 0
    return x
