"""Values of the operators with scales for blocks of 128 where a loose bound would hide a fault:
short sums on many tiles, blocks in an activation's tail, long sums that are exact, each code
type."""
import importlib.util
import os

import pytest
import torch

import block128_ref as ref

pytestmark = pytest.mark.gpu
E4M3, E5M2 = 0, 1
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def settled(fp8g):
    st, detail = fp8g.fp8_gemm_status()
    assert st == 0, (st, detail)


# ------------------------------------------------ gated projections of one or two K blocks

@pytest.mark.parametrize("K", [16, 128, 144, 256])
@pytest.mark.parametrize("gate", [0, 1, 2])
def test_gated_short_sums_on_many_tiles(fp8g, K, gate):
    # both product buffers hold a tile's K blocks, so nothing but their own exchange keeps the two
    # warps of a row on the same tile; 240 tiles, three or four to a pair
    M, F = 3000, 2560
    r = torch.Generator(device="cuda").manual_seed(K + gate)
    x, _ = fp8g.quantize_block128(torch.randn((M, K), device="cuda", generator=r))
    W = fp8g.quantize_tile128(torch.randn((2 * F, K), device="cuda", generator=r) * K ** -0.5)
    h, gu = fp8g.gated_block128(*x, *W, gate=gate, keep=True)
    settled(fp8g)
    both, mags = ref.product(ref.decode(*x, "row", E4M3), ref.decode(*W, "tile", E4M3), "nt")
    err = ref.sum_tol(K) * mags
    g, u = both[:, :F], both[:, F:]
    y, _ = ref.act(g, gate)
    ref.assert_coded(*gu, "row", E4M3, both, err)
    # act' is at most 1.13 in magnitude; act itself within 2^-20 (2 + |g|) |g|; a product's rounding
    eh = (1.13 * err[:, :F] + 2.0 ** -20 * (2 + g.abs()) * g.abs()) * (u.abs() + err[:, F:]) + y.abs() * err[:, F:] \
        + 2.0 ** -23 * (y * u).abs()
    ref.assert_coded(*h, "row", E4M3, y * u, eh)
    for _ in range(20):
        again = fp8g.gated_block128(*x, *W, gate=gate, keep=True)
        assert all(torch.equal(a, b) for a, b in zip(again[0] + again[1], h + gu))
    settled(fp8g)


# ------------------------------------------- activations to a bound relative to their own value
# A block's scale goes by its own largest value, so a block of small values leaves no slack: M = 1
# and the last row of 129 make column blocks of one value each.

def act_errors(g, gate):
    """The activation and its derivative in 64 bits, and how far the kernels' may be off: every
    operation once, in units of 2^-24 (u), with up to two units in g itself and four more for the
    products that follow."""
    u, a = 2.0 ** -24, g.abs()
    if gate == 1:  # (the complement: torch's ndtr is 1 + erf, nothing is left of it at -9)
        c, phi = torch.special.erfc(-g / 2 ** 0.5) / 2, torch.exp(-g * g / 2) / (2 * torch.pi) ** 0.5
        y, d = g * c, c + g * phi
    else:
        y, d = ref.act(g, gate)
    if gate == 0:
        # e^-g: 2 + 2 units of its argument (the constant, the product) make 4 |g|, the exponential 4,
        # the sum 1, the reciprocal 2; the derivative s (1 + g (1 - s)) has that twice, of s (1 + |g|)
        r = (16 + 4 * a) * u
        size = torch.sigmoid(g) * (1 + a)
        ey, ed = r * y.abs(), 2 * r * size
    elif gate == 1:
        # Phi and |g| phi each relative to itself: e^(-g^2 / 2) has g^2 / 2 times 7 units (g twice, square,
        # constant, product) and its own 4; Phi's other factor, with slope at most 2.7 in what it is
        # a polynomial of, 15 for that (sum, reciprocal, g), the fit's 2 and 4 for its steps; the
        # products' 4 with it
        r = (4 * g * g + 28) * u
        ey, ed = r * y.abs(), r * (c + a * phi)
    else:
        ey, ed = 8 * u * y.abs(), 8 * u * d
    # below the normal numbers: one of them, of the sigmoid, of Phi or of phi
    floor = 0.0 if gate == 2 else (a + 1) * 2.0 ** -125
    return y, d, ey + floor, ed + floor


def gates(kind, M, F, gen):
    """Gates of one kind, in blocks of 128 columns that lie close together."""
    t = torch.rand((M, F), generator=gen)
    if kind == "tail":      # -9 .. -4
        return -4 - 5 * (torch.arange(F) // 128 + t) / (F // 128)
    if kind == "far":       # -40 .. -9
        return -9 - 31 * (torch.arange(F) // 128 + t) / (F // 128)
    return 16 * t - 8       # -8 .. 8


@pytest.mark.parametrize("M", [1, 129, 257])
@pytest.mark.parametrize("gate", [0, 1, 2])
@pytest.mark.parametrize("kind", ["tail", "far", "both"])
@pytest.mark.parametrize("fmt", [E4M3, E5M2])
def test_backward_in_the_tails(fp8g, M, gate, kind, fmt):
    F = 384
    r = torch.Generator().manual_seed(M + 10 * gate)
    gu, sgu = ref.quant(torch.cat((gates(kind, M, F, r), torch.randn((M, F), generator=r)), 1), "row", E4M3)
    dh = torch.randn((M, F), generator=r).bfloat16()
    row, col, h = fp8g.gated_block128_backward(dh.cuda(), gu.cuda(), sgu.cuda(), gate=gate, fmt=fmt)
    settled(fp8g)
    both = ref.decode(gu, sgu, "row", E4M3)
    g, u, x = both[:, :F], both[:, F:], dh.double()
    y, d, ey, ed = act_errors(g, gate)
    want, err = torch.cat((x * u * d, x * y), 1), torch.cat((x.abs() * u.abs() * ed, x.abs() * ey), 1)
    ref.assert_coded(row[0].cpu(), row[1].cpu(), "row", fmt, want, err)
    ref.assert_coded(col[0].cpu(), col[1].cpu(), "col", fmt, want, err)
    ref.assert_coded(h[0].cpu(), h[1].cpu(), "col", E4M3, y * u, ey * u.abs())


@pytest.mark.parametrize("M", [1, 3, 40, 300])
@pytest.mark.parametrize("gate", [0, 1, 2])
@pytest.mark.parametrize("kind", ["tail", "far", "both"])
def test_gated_in_the_tails(fp8g, M, gate, kind):
    # x has a one in its first column and zeros elsewhere: gate and up are one product each, with two
    # roundings (the scales' product, its product with the code's)
    F, K = 384, 16
    r = torch.Generator().manual_seed(M + 10 * gate)
    code = lambda t: t.to(torch.float8_e4m3fn).view(torch.uint8)
    x = torch.zeros((M, K))
    x[:, 0] = 1
    W = torch.zeros((2 * F, K))
    W[:F, 0] = gates(kind, 1, F, r)[0]
    W[F:, 0] = torch.randn(F, generator=r)
    sx, sw = torch.rand((1, M), generator=r) * 0.1 + 1, torch.rand((2 * F // 128, 1), generator=r) * 0.1 + 0.95
    qx, qw = code(x), code(W)
    h, gu = fp8g.gated_block128(qx.cuda(), sx.cuda(), qw.cuda(), sw.cuda(), gate=gate, keep=True)
    settled(fp8g)
    both, _ = ref.product(ref.decode(qx, sx, "row", E4M3), ref.decode(qw, sw, "tile", E4M3), "nt")
    ref.assert_coded(gu[0].cpu(), gu[1].cpu(), "row", E4M3, both, 2.0 ** -23 * both.abs())
    g, u = both[:, :F], both[:, F:]
    y, _, ey, _ = act_errors(g, gate)
    ref.assert_coded(h[0].cpu(), h[1].cpu(), "row", E4M3, y * u, ey * u.abs())


# ------------------------------------------------------------- sums that are exact in any order

def small(r, shape, fmt, most=2):
    """Codes of whole numbers -most .. most."""
    t = torch.randint(-most, most + 1, shape, device="cuda", generator=r)
    return t.float().to(ref.DT[fmt]).view(torch.uint8)


def halves(r, *shape):
    """Scales 1/2, 1 or 2."""
    return torch.exp2(torch.randint(-1, 2, shape, device="cuda", generator=r).float())


def exact_product(r, form, M, N, K, a_fmt=E4M3, b_fmt=E4M3):
    """Operands of whole numbers and powers of two: a sum is a multiple of 1/4 of at most 16 K, exact in
    fp32 in any order up to K = 2^18.  And the product in 64 bits."""
    mk, nk, kk = ref.up(M), ref.up(N), ref.up(K)
    A = small(r, (K, M) if form == "tn" else (M, K), a_fmt), halves(r, kk, M)
    B = small(r, (N, K) if form == "nt" else (K, N), b_fmt), halves(r, *((kk, N) if form == "tn" else (nk, kk) if form == "nt"
                                                                       else (kk, nk)))
    ka, kb = ("col", "col") if form == "tn" else ("row", "tile")
    return A, B, ref.product(ref.decode(*A, ka, a_fmt), ref.decode(*B, kb, b_fmt), form)[0]


SUMS = [
    # K blocks of tiles shared between CTA pairs: all tiles, the last ones behind whole ones
    ("tn", 272, 400, 12000), ("nn", 1500, 1040, 16000), ("tn", 16, 16, 12001), ("nt", 4100, 1288, 16384),
    ("tn", 2304, 2304, 16400), ("nt", 300, 264, 12304), ("nn", 4099, 4096, 12304),
    # several whole tiles to a pair
    ("nt", 4099, 5000, 2064), ("nn", 2100, 2592, 2000), ("tn", 4096, 2832, 2051),
    # few rows: K split over clusters of up to eight CTAs, one and two of them to an SM
    ("nt", 1, 4096, 14336), ("nt", 1, 128, 16384), ("nn", 16, 144, 16384), ("nt", 33, 520, 12304), ("nt", 64, 5120, 5120),
    ("nt", 77, 5120, 5120), ("nn", 128, 272, 16000), ("nt", 128, 2048, 4096), ("nt", 250, 256, 16384),
]


@pytest.mark.parametrize("form,M,N,K", SUMS)
def test_long_sums_exact(fp8g, form, M, N, K):
    r = torch.Generator(device="cuda").manual_seed(K + M)
    A, B, want = exact_product(r, form, M, N, K)
    start = torch.randint(-9, 10, (M, N), device="cuda", generator=r).float()
    assert torch.equal(fp8g.gemm_block128(*A, *B, form=form, out="f32").double(), want)
    assert torch.equal(fp8g.gemm_block128(*A, *B, form=form), want.float().bfloat16())
    assert torch.equal(fp8g.gemm_block128(*A, *B, form=form, add_to=start.clone()).double(), want + start)
    settled(fp8g)


@pytest.mark.parametrize("a_fmt,b_fmt", [(E4M3, E5M2), (E5M2, E4M3), (E5M2, E5M2)])
@pytest.mark.parametrize("form,M,N,K", [("nt", 5, 264, 12304), ("nt", 128, 1040, 4096), ("nn", 300, 272, 12304), ("tn", 272, 400, 12000),
                                        ("nt", 2100, 2600, 1040)])
def test_long_sums_exact_of_each_type(fp8g, form, M, N, K, a_fmt, b_fmt):
    r = torch.Generator(device="cuda").manual_seed(K + M + 2 * a_fmt + b_fmt)
    A, B, want = exact_product(r, form, M, N, K, a_fmt, b_fmt)
    C = fp8g.gemm_block128(*A, *B, form=form, a_fmt=a_fmt, b_fmt=b_fmt, out="f32")
    settled(fp8g)
    assert torch.equal(C.double(), want)


@pytest.mark.parametrize("x_fmt,w_fmt", [(E4M3, E4M3), (E5M2, E4M3), (E4M3, E5M2), (E5M2, E5M2)])
@pytest.mark.parametrize("M,F,K", [(1, 1408, 4112), (16, 256, 2064), (64, 384, 12304), (100, 256, 4096), (300, 384, 1040),
                                   (1500, 2048, 2064)])
def test_gated_bits(fp8g, M, F, K, x_fmt, w_fmt):
    # gate and up are exact, relu(g) u one rounding (of 32 bits here as there): codes and scales bit for bit
    r = torch.Generator(device="cuda").manual_seed(K + M)
    x, sx = small(r, (M, K), x_fmt), halves(r, ref.up(K), M)
    W, sw = small(r, (2 * F, K), w_fmt), halves(r, ref.up(2 * F), ref.up(K))
    h, gu = fp8g.gated_block128(x, sx, W, sw, gate=fp8g.FP8G_GATE_RELU, keep=True, x_fmt=x_fmt, w_fmt=w_fmt)
    only, none = fp8g.gated_block128(x, sx, W, sw, gate=fp8g.FP8G_GATE_RELU, x_fmt=x_fmt, w_fmt=w_fmt)
    settled(fp8g)
    both = ref.product(ref.decode(x, sx, "row", x_fmt), ref.decode(W, sw, "tile", w_fmt), "nt")[0].float().cpu()
    for got, v in ((h, both[:, :F].clamp(min=0) * both[:, F:]), (gu, both)):
        q, s = ref.quant(v, "row", E4M3)
        # (a zero that came from -0 keeps its sign in one and not in the other)
        assert torch.equal(got[1].cpu(), s) and torch.equal(got[0].cpu().view(ref.DT[0]).float(), q.view(ref.DT[0]).float())
    assert none is None and torch.equal(only[0], h[0]) and torch.equal(only[1], h[1])


# --------------------------------------- weights that the kernel in front writes

@pytest.mark.parametrize("M", [1, 40, 100, 300])
def test_weights_written_just_before(fp8g, M):
    # kernels for few rows fetch weights to L2 while the one in front still runs
    N, K = 2048, 4096
    r = torch.Generator(device="cuda").manual_seed(M)
    x, _ = fp8g.quantize_block128(torch.randn((M, K), device="cuda", generator=r))
    ws = [torch.randn((N, K), device="cuda", generator=r) for _ in range(3)]
    want = []
    for w in ws:
        t = fp8g.quantize_tile128(w)
        torch.cuda.synchronize()
        want.append((fp8g.gemm_block128(*x, *t), fp8g.gated_block128(*x, *t)[0]))
        torch.cuda.synchronize()
    q, s = (torch.empty_like(v) for v in fp8g.quantize_tile128(ws[0]))

    def turn():
        got = []
        for w in ws:
            fp8g.fp8g_quantize_tile128(w, fp8g.FP8G_IN_F32, K, N, K, E4M3, q, s)
            got.append(fp8g.gemm_block128(*x, q, s))
        for w in ws:
            fp8g.fp8g_quantize_tile128(w, fp8g.FP8G_IN_F32, K, N, K, E4M3, q, s)
            got.append(fp8g.gated_block128(*x, q, s)[0])
        return got

    def check(got):
        torch.cuda.synchronize()
        for i, (c, h) in enumerate(want):
            assert torch.equal(got[i], c) and all(torch.equal(a, b) for a, b in zip(got[3 + i], h))
    for _ in range(5):
        check(turn())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = turn()
    for _ in range(20):
        g.replay()
        check(got)
    settled(fp8g)


# ------------------------------------------------- the training step, its roundings in quadrature

@pytest.mark.parametrize("tokens", [1, 33, 1100])
@pytest.mark.parametrize("gate", [0, 1, 2])
def test_training_step_in_quadrature(fp8g, tokens, gate):
    spec = importlib.util.spec_from_file_location("ffn_step", os.path.join(ROOT, "examples", "ffn_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    layer = example.Layer(384, 256, gate, seed=tokens)
    r = torch.Generator(device="cuda").manual_seed(tokens)
    x, dy = (torch.randn((tokens, 384), device="cuda", generator=r).bfloat16() for _ in range(2))
    y, dx = layer.forward(x), layer.backward(dy)
    settled(fp8g)
    v = [t.detach().double().requires_grad_() for t in (x, layer.w13, layer.w2)]
    gu = v[0] @ v[1].t()
    h = ref.act(gu[:, :256], gate)[0] * gu[:, 256:]
    out = h @ v[2].t()
    wants = [out.detach()] + list(torch.autograd.grad(out, v, dy.double()))
    # roundings on the way, each independent of the others and of root mean square at most half a step
    # over sqrt 3: x, W13 (both in g and in u), h, W2; dy, W2, x and W13 in g and in u, the checkpoint, dgu,
    # W13; the same without the last weights and with x; dy, x and W13 in g and in u, the checkpoint, h
    for name, got, want, n in (("y", y, wants[0], 6), ("dx", dx, wants[1], 10), ("dw13", layer.dw13, wants[2], 10),
                               ("dw2", layer.dw2, wants[3], 8)):
        square = n / 3 * ref.HALF[E4M3] ** 2
        if gate == 2 and name in ("dx", "dw13"):
            # ReLU's derivative steps: a gate of unit variance, off by 0.051 (two roundings), changes sign in
            # 0.051 sqrt(2 / pi) phi(0) = 0.0163 of all places, 0.0325 of those that count, in the half of
            # the gradient's square that comes through the gate
            square += 0.0163
        got, most = got.double(), square ** 0.5
        assert (got - want).norm() <= most * want.norm(), name
        # along the wanted gradient: four standard deviations of what 256 independent values leave, and
        # the second order
        along = ((got * want).sum() / want.square().sum()).item() - 1
        assert abs(along) <= most / 4 + most ** 2, (name, along)
