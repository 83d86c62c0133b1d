"""Host-side checks of the operators with scales for blocks of 128: refused before
a device is touched (no GPU needed)."""
import pytest

import fp8_block_scaled_06_gb300 as m

P = 1 << 20  # an aligned fake address; never dereferenced
ARG, ALIGN, SHAPE = m.FP8G_ERR_INVALID_ARG, m.FP8G_ERR_ALIGNMENT, m.FP8G_ERR_UNSUPPORTED_SHAPE
BIG = 1 << 31

QUANT = ("x in_dtype ld rows cols fmt q_row s_row q_col s_col".split(), (P, 0, 64, 8, 64, 0, P, P, P, P))
TILE = ("x in_dtype ld rows cols fmt q s".split(), (P, 0, 64, 8, 64, 0, P, P))
TURN = ("q q_fmt s rows cols fmt q_col s_col".split(), (P, 0, P, 8, 64, 0, 2 * P, P))
GEMM = ("form A sfa a_fmt B sfb b_fmt C out add M N K".split(), (0, P, P, 0, P, P, 0, P, 0, 0, 32, 64, 128))
GATED = ("x sfx x_fmt W13 sf13 w_fmt gate h sh gu sgu M F K".split(), (P, P, 0, P, P, 0, 0, P, P, P, P, 4, 128, 64))
BACK = ("dh dh_dtype gu sgu gate fmt M F row s_row col s_col h sh".split(),
        (P, 0, P, P, 0, 0, 4, 128, P, P, P, P, P, P))


def nulls(*names):
    return [(ARG, {n: 0}) for n in names]


def odd(*names):
    return [(ALIGN, {n: P + 8}) for n in names]


CASES = [
    ("fp8g_quantize_block128", QUANT, nulls("x", "q_row", "s_row", "q_col", "s_col") + odd("x", "q_row", "s_row", "q_col", "s_col") + [
        (ARG, dict(q_row=0, s_row=0, q_col=0, s_col=0)), (ARG, dict(in_dtype=2)), (ARG, dict(fmt=2)), (ARG, dict(fmt=-1)),
        (ARG, dict(rows=-1)), (ARG, dict(cols=0)), (ARG, dict(ld=48)), (SHAPE, dict(cols=56, ld=64)),
        (SHAPE, dict(rows=65535 * 16 + 1)), (SHAPE, dict(cols=BIG, ld=BIG)), (ALIGN, dict(ld=66)), (ALIGN, dict(in_dtype=1, ld=68))]),
    ("fp8g_quantize_tile128", TILE, nulls("x", "q", "s") + odd("x", "q", "s") + [
        (ARG, dict(in_dtype=-1)), (ARG, dict(fmt=3)), (SHAPE, dict(cols=24)), (ALIGN, dict(ld=65))]),
    ("fp8g_requantize_block128", TURN, nulls("q", "s", "q_col", "s_col") + odd("q", "s", "q_col", "s_col") + [
        (ARG, dict(q_fmt=2)), (ARG, dict(fmt=2)), (ARG, dict(q_col=P)), (ARG, dict(rows=-1)), (ARG, dict(cols=0)),
        (SHAPE, dict(cols=40)), (SHAPE, dict(rows=65535 * 16 + 1))]),
    ("fp8_gemm_block128", GEMM, nulls("A", "sfa", "B", "sfb", "C") + odd("A", "sfa", "B", "sfb", "C") + [
        (ARG, dict(form=3)), (ARG, dict(form=-1)), (ARG, dict(a_fmt=2)), (ARG, dict(b_fmt=4)), (ARG, dict(out=2)),
        (ARG, dict(add=1)), (ARG, dict(out=1, add=2)), (ARG, dict(M=-1)), (ARG, dict(N=0)), (ARG, dict(K=0)),
        (ARG, dict(form=1, K=0)), (ARG, dict(form=2, M=0)), (ARG, dict(form=2, K=-1)),
        (SHAPE, dict(M=BIG)), (SHAPE, dict(N=BIG)), (SHAPE, dict(K=BIG)), (SHAPE, dict(M=BIG - 1, N=BIG - 8)),
        (ALIGN, dict(K=120)), (ALIGN, dict(N=60)), (ALIGN, dict(form=1, N=56)), (ALIGN, dict(form=1, K=24)),
        (ALIGN, dict(form=2, M=24)), (ALIGN, dict(form=2, N=40)), (ALIGN, dict(out=1, N=62))]),
    ("fp8_gated_block128", GATED, nulls("x", "sfx", "W13", "sf13", "h", "sh", "gu", "sgu") +
     odd("x", "sfx", "W13", "sf13", "h", "sh", "gu", "sgu") + [
        (ARG, dict(x_fmt=2)), (ARG, dict(w_fmt=-1)), (ARG, dict(gate=3)), (ARG, dict(gate=-1)), (ARG, dict(M=-1)),
        (ARG, dict(F=0)), (ARG, dict(K=0)), (SHAPE, dict(F=192)), (SHAPE, dict(M=BIG)), (SHAPE, dict(F=1 << 30)),
        (SHAPE, dict(K=BIG)), (ALIGN, dict(K=72))]),
    ("fp8g_gated_block128_backward", BACK, nulls("dh", "gu", "sgu", "row", "s_row", "col", "s_col", "h", "sh") +
     odd("dh", "gu", "sgu", "row", "s_row", "col", "s_col", "h", "sh") + [
        (ARG, dict(dh_dtype=2)), (ARG, dict(gate=3)), (ARG, dict(fmt=2)), (ARG, dict(M=-1)), (ARG, dict(F=0)),
        (SHAPE, dict(F=64)), (SHAPE, dict(M=65535 * 16 + 1)), (SHAPE, dict(F=1 << 30))]),
]


@pytest.mark.parametrize("name,call,want,change",
                         [(n, c, w, d) for n, c, l in CASES for w, d in l],
                         ids=[f"{n}-{'-'.join(map(str, sum(d.items(), ())))}" for n, _, l in CASES for _, d in l])
def test_refused(fp8g, name, call, want, change):
    names, args = call
    assert set(change) <= set(names)
    with pytest.raises(m.Fp8gError) as e:
        getattr(fp8g, name)(*[change.get(n, a) for n, a in zip(names, args)], 0)
    assert e.value.status == want


def test_tensors_on_the_host_are_refused(fp8g):
    import torch
    u = torch.zeros((16, 128), dtype=torch.uint8)
    s = torch.ones((1, 16))
    for call in (lambda: fp8g.quantize_block128(torch.zeros((16, 128))), lambda: fp8g.quantize_tile128(torch.zeros((16, 128))),
                 lambda: fp8g.requantize_block128(u, s), lambda: fp8g.gemm_block128(u, s, u, torch.ones((1, 1))),
                 lambda: fp8g.gated_block128(u, s, torch.zeros((256, 128), dtype=torch.uint8), torch.ones((2, 1))),
                 lambda: fp8g.gated_block128_backward(torch.zeros((16, 64)), u, s)):
        with pytest.raises((AssertionError, RuntimeError)):
            call()
