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
