"""Host-side checks of the router, the MoE layer, the projection with adapters
and the scale packing: refused before a device is touched (no GPU needed)."""
import pytest

import fp8_block_scaled_06_gb300 as m

P = 1 << 20  # an aligned fake address; never dereferenced
ARG, ALIGN, SHAPE = m.FP8G_ERR_INVALID_ARG, m.FP8G_ERR_ALIGNMENT, m.FP8G_ERR_UNSUPPORTED_SHAPE


def status(fn, args, names, **change):
    assert set(change) <= set(names)
    with pytest.raises(m.Fp8gError) as e:
        fn(*[change.get(n, a) for n, a in zip(names, args)], 0)
    return e.value.status


ROUTE = ("logits in_dtype ld T E k score scale ids weights counts rows slots".split(),
         (P, 0, 8, 4, 8, 2, 0, 1.0, P, P, P, P, P))
MOE = ("x x_dtype ids weights W13 sf13 W2 sf2 out out_dtype w_fmt gate T k E H F".split(),
       (P, 0, P, P, P, P, P, P, P, 0, 0, 0, 4, 2, 8, 128, 64))
LORA = ("x x_dtype W sfw w_fmt a b alpha adapter L r bias C out M N K".split(),
        (P, 0, P, P, 0, P, P, P, P, 4, 16, P, P, 0, 4, 64, 64))
PACK = ("sf matrices rows K packed".split(), (P, 1, 8, 64, P))

CASES = [
    ("fp8g_moe_route", ROUTE, [
        (ARG, dict(in_dtype=2)), (ARG, dict(score=4)), (ARG, dict(score=-1)), (ARG, dict(T=-1)), (ARG, dict(E=0)),
        (ARG, dict(k=0)), (ARG, dict(k=9)), (ARG, dict(ld=7)), (ARG, dict(logits=0)), (ARG, dict(ids=0)),
        (ARG, dict(weights=0)), (ARG, dict(counts=0)), (ARG, dict(rows=0)), (ARG, dict(slots=0)),
        (SHAPE, dict(E=257, ld=257)), (SHAPE, dict(k=17, E=32, ld=32)), (SHAPE, dict(T=262145)),
        (ALIGN, dict(logits=P + 2)), (ALIGN, dict(in_dtype=1, logits=P + 1)), (ALIGN, dict(ids=P + 2)),
        (ALIGN, dict(weights=P + 1)), (ALIGN, dict(slots=P + 2))]),
    ("fp8_moe_layer", MOE, [
        (ARG, dict(x_dtype=2)), (ARG, dict(out_dtype=2)), (ARG, dict(w_fmt=5)), (ARG, dict(w_fmt=-1)),
        (ARG, dict(gate=3)), (ARG, dict(T=-1)), (ARG, dict(k=0)), (ARG, dict(E=0)), (ARG, dict(H=0)), (ARG, dict(F=0)),
        (ARG, dict(x=0)), (ARG, dict(ids=0)), (ARG, dict(weights=0)), (ARG, dict(W13=0)), (ARG, dict(sf13=0)),
        (ARG, dict(W2=0)), (ARG, dict(sf2=0)), (ARG, dict(out=0)),
        (SHAPE, dict(H=48)), (SHAPE, dict(F=48)), (SHAPE, dict(w_fmt=2, F=160)), (SHAPE, dict(w_fmt=3, H=160)),
        (SHAPE, dict(T=513)), (SHAPE, dict(k=17)), (SHAPE, dict(E=257)),
        (ALIGN, dict(x=P + 8)), (ALIGN, dict(out=P + 8)), (ALIGN, dict(W13=P + 8)), (ALIGN, dict(sf2=P + 8)),
        (ALIGN, dict(w_fmt=2, F=128, W2=P + 16))]),
    ("fp8_gemm_lora", LORA, [
        (ARG, dict(x_dtype=2)), (ARG, dict(out=2)), (ARG, dict(w_fmt=5)), (ARG, dict(M=-1)), (ARG, dict(N=0)),
        (ARG, dict(K=0)), (ARG, dict(L=-1)), (ARG, dict(r=0)), (ARG, dict(x=0)), (ARG, dict(W=0)), (ARG, dict(sfw=0)),
        (ARG, dict(C=0)), (ARG, dict(a=0)), (ARG, dict(b=0)), (ARG, dict(adapter=0)),
        (SHAPE, dict(K=48)), (SHAPE, dict(w_fmt=2)), (SHAPE, dict(r=12)), (SHAPE, dict(r=264)), (SHAPE, dict(L=1025)),
        (SHAPE, dict(M=1 << 24)), (SHAPE, dict(N=1 << 24)),
        (ALIGN, dict(x=P + 8)), (ALIGN, dict(C=P + 8)), (ALIGN, dict(W=P + 8)), (ALIGN, dict(w_fmt=2, K=128, W=P + 16)),
        (ALIGN, dict(sfw=P + 8)), (ALIGN, dict(a=P + 8)), (ALIGN, dict(b=P + 8)), (ALIGN, dict(alpha=P + 2)),
        (ALIGN, dict(bias=P + 2)), (ALIGN, dict(adapter=P + 2)), (ALIGN, dict(N=60))]),
    ("fp8g_pack_scales", PACK, [
        (ARG, dict(sf=0)), (ARG, dict(packed=0)), (ARG, dict(matrices=0)), (ARG, dict(rows=0)), (ARG, dict(K=0)),
        (SHAPE, dict(K=48)), (SHAPE, dict(matrices=65536)), (SHAPE, dict(rows=65536 * 128)),
        (ALIGN, dict(sf=P + 4)), (ALIGN, dict(packed=P + 8))]),
]


@pytest.mark.parametrize("name,call,want,change",
                         [(n, c, w, d) for n, c, l in CASES for w, d in l],
                         ids=[f"{n}-{'-'.join(map(str, sum(d.items(), ())))}" for n, _, l in CASES for _, d in l])
def test_refused(fp8g, name, call, want, change):
    names, args = call
    assert status(getattr(fp8g, name), args, names, **change) == want


def test_packed_scale_bytes(fp8g):
    f = fp8g.load().fp8g_packed_scale_bytes
    assert f(1, 1, 32) == 512 and f(3, 129, 160) == 3 * 2 * 2 * 512
    assert f(0, 8, 64) == 0 and f(1, 8, 48) == 0 and f(1, 0, 64) == 0 and f(-1, 8, 64) == 0
    assert f(65536, 8, 64) == 0 and f(65535, 128, 128) == 65535 * 512
