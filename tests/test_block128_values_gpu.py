"""Values of the operators with scales for blocks of 128 where a loose bound would hide a fault:
short sums on many tiles, blocks in an activation's tail, long sums that are exact, each code
type."""
import pytest
import torch

import block128_ref as ref

pytestmark = pytest.mark.gpu
E4M3, E5M2 = 0, 1


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
