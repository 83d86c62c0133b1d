"""The operators with fp32 scales for blocks of 128: the quantisers bit for bit, the
products, the gated projections and their backward pass against 64 bits."""
import math
import zlib

import pytest
import torch

import block128_ref as ref

pytestmark = pytest.mark.gpu
E4M3, E5M2 = 0, 1


def gen(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def settled(fp8g):
    st, detail = fp8g.fp8_gemm_status()
    assert st == 0, (st, detail)


def same(got, want):
    (q, s), (qw, sw) = got, want
    assert torch.equal(s.cpu(), sw) or (torch.equal(s.cpu().isnan(), sw.isnan()) and torch.equal(s.cpu().nan_to_num(), sw.nan_to_num()))
    bad = q.cpu() != qw
    assert not bad.any(), f"{int(bad.sum())} codes, first at {bad.nonzero()[0].tolist()}"


# ------------------------------------------------------------------ quantisers

SHAPES = [(1, 16), (1, 4096), (3, 128), (7, 144), (128, 128), (129, 112), (257, 400), (300, 1024)]


@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", [E4M3, E5M2])
def test_quantise_bits(fp8g, R, C, dtype, fmt):
    x = ref.values(R, C, gen(1, R, C))
    x = x.bfloat16() if dtype == "bf16" else x
    row, col = fp8g.quantize_block128(x.cuda(), row=True, col=True, fmt=fmt)
    same(row, ref.quant(x, "row", fmt))
    same(col, ref.quant(x, "col", fmt))
    only, none = fp8g.quantize_block128(x.cuda(), fmt=fmt)
    assert none is None
    same(only, ref.quant(x, "row", fmt))
    same(fp8g.quantize_block128(x.cuda(), row=False, col=True, fmt=fmt)[1], ref.quant(x, "col", fmt))
    same(fp8g.quantize_tile128(x.cuda(), fmt=fmt), ref.quant(x, "tile", fmt))


def test_quantise_strides_and_edges(fp8g):
    x = ref.values(130, 320, gen(2))
    x[0, 0], x[5, 200], x[129, 319] = math.nan, math.inf, -math.inf
    x[7] = 0
    x[9] *= 1e-42   # scales at their least
    x[11] = 3e38
    row, col = fp8g.quantize_block128(x.cuda(), row=True, col=True)
    qr, sr = ref.quant(x, "row", E4M3)
    same(row, (qr, sr))
    same(col, ref.quant(x, "col", E4M3))
    assert (sr[:, 7] == 1).all() and sr[1, 5] == math.inf
    wide = torch.zeros((130, 512), device="cuda")
    wide[:, 64:384] = x.cuda()
    same(fp8g.quantize_block128(wide[:, 64:384])[0], (qr, sr))          # rows apart
    same(fp8g.quantize_block128(x.t().contiguous().cuda().t())[0], (qr, sr))  # columns apart
    odd = torch.zeros((130, 322), device="cuda")
    odd[:, 1:321] = x.cuda()
    same(fp8g.quantize_block128(odd[:, 1:321])[0], (qr, sr))            # neither aligned
    for R in (0, 1):
        (q, s), (qc, sc) = fp8g.quantize_block128(x[:R].cuda(), row=True, col=True)
        assert q.shape == (R, 320) and s.shape == (3, R) and qc.shape == (R, 320) and sc.shape == (R, 320)


@pytest.mark.parametrize("R,C", [(1, 16), (129, 272), (256, 512)])
@pytest.mark.parametrize("q_fmt,fmt", [(E4M3, E4M3), (E4M3, E5M2), (E5M2, E4M3)])
def test_requantise_bits(fp8g, R, C, q_fmt, fmt):
    q, s = ref.quant(ref.values(R, C, gen(3, R)), "row", q_fmt)
    if R > 100:
        q[100, 3] = 0x7F
    x = q.view(ref.DT[q_fmt]).float() * ref.spread(s, "row", R, C)  # one fp32 product, as defined
    same(fp8g.requantize_block128(q.cuda(), s.cuda(), fmt=fmt, q_fmt=q_fmt), ref.quant(x, "col", fmt))


def test_codes_feed_the_product_round_trip(fp8g):
    # identity weights in tiles: the product gives back what the codes stand for
    x = ref.values(300, 256, gen(4))
    (q, s), _ = fp8g.quantize_block128(x.cuda())
    w, sw = fp8g.quantize_tile128(torch.eye(256).cuda())
    C = fp8g.gemm_block128(q, s, w, sw, out="f32")
    settled(fp8g)
    want = ref.decode(q.cpu(), s.cpu(), "row", E4M3)
    # 448 * fl(1/448) and the scales' product: three roundings
    assert ((C.cpu().double() - want).abs() <= 2.0 ** -22 * want.abs()).all()


# -------------------------------------------------------------------- products

def operands(form, M, N, K, a_fmt, b_fmt, g):
    if form == "tn":
        A, B = ref.quant(ref.values(K, M, g), "col", a_fmt), ref.quant(ref.values(K, N, g), "col", b_fmt)
        return A, B, "col", "col"
    A = ref.quant(ref.values(M, K, g), "row", a_fmt)
    B = ref.quant(ref.values(*((N, K) if form == "nt" else (K, N)), g, zeros=False), "tile", b_fmt)
    return A, B, "row", "tile"


def check_product(fp8g, form, M, N, K, a_fmt=E4M3, b_fmt=E4M3, out="bf16", add=False):
    g = gen(5, form, M, N, K)
    A, B, ka, kb = operands(form, M, N, K, a_fmt, b_fmt, g)
    start = torch.randn((M, N), generator=g) if add else None
    dev = [t.cuda() for t in A + B]
    C = fp8g.gemm_block128(*dev, form=form, a_fmt=a_fmt, b_fmt=b_fmt, out=out,
                           add_to=start.cuda() if add else None)
    settled(fp8g)
    want, mags = ref.product(ref.decode(*A, ka, a_fmt), ref.decode(*B, kb, b_fmt), form)
    tol = ref.sum_tol(K) * mags
    if add:
        want = want + start.double()
        tol = tol + 2.0 ** -24 * want.abs()
    if out == "bf16":
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    bad = (C.cpu().double() - want).abs() > tol
    assert C.shape == (M, N) and not bad.any(), f"{int(bad.sum())} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}"
    return C


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 65, 128])
@pytest.mark.parametrize("N,K", [(8, 16), (136, 144), (1000, 1024), (128, 2064)])
def test_forward_few_rows(fp8g, M, N, K):
    check_product(fp8g, "nt", M, N, K)


@pytest.mark.parametrize("M,N,K", [(129, 128, 128), (256, 256, 16), (257, 264, 144), (300, 8, 400), (1030, 776, 640),
                                   (200, 2048, 4096)])
def test_forward(fp8g, M, N, K):
    check_product(fp8g, "nt", M, N, K)
    check_product(fp8g, "nt", M, N, K, out="f32", add=True)


@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (19, 144, 272), (64, 1040, 528), (129, 128, 128), (300, 272, 400),
                                   (513, 784, 1040)])
def test_input_gradient(fp8g, M, N, K):
    check_product(fp8g, "nn", M, N, K, a_fmt=E5M2)
    check_product(fp8g, "nn", M, N, K, out="f32")


@pytest.mark.parametrize("M,N,K", [(16, 16, 1), (128, 144, 3), (144, 128, 127), (256, 256, 128), (272, 400, 129),
                                   (528, 784, 700), (1040, 256, 2050)])
def test_weight_gradient(fp8g, M, N, K):
    check_product(fp8g, "tn", M, N, K, out="f32", add=True)
    check_product(fp8g, "tn", M, N, K, a_fmt=E5M2)


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
@pytest.mark.parametrize("a_fmt,b_fmt", [(E4M3, E5M2), (E5M2, E4M3), (E5M2, E5M2)])
@pytest.mark.parametrize("M", [32, 192])
def test_formats_and_outputs(fp8g, form, a_fmt, b_fmt, M):
    for out in ("bf16", "f32"):
        check_product(fp8g, form, M, 144, 272, a_fmt, b_fmt, out)


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
@pytest.mark.parametrize("M", [16, 48, 320])
def test_exact_on_small_integers(fp8g, form, M):
    # integers in codes, powers of two in scales: every sum is exact, in any order
    N, K = 272, 400
    g = gen(6, form, M)
    a = torch.randint(-3, 4, (K, M) if form == "tn" else (M, K), generator=g)
    b = torch.randint(-3, 4, (N, K) if form == "nt" else (K, N), generator=g)
    p2 = lambda *s: torch.exp2(torch.randint(-2, 3, s, generator=g).float())
    sa = p2(4, M)
    sb = p2(4, N) if form == "tn" else p2(3, 4) if form == "nt" else p2(4, 3)
    ka, kb = ("col", "col") if form == "tn" else ("row", "tile")
    code = lambda t: t.float().to(torch.float8_e4m3fn).view(torch.uint8)
    want, _ = ref.product(ref.decode(code(a), sa, ka, E4M3), ref.decode(code(b), sb, kb, E4M3), form)
    C = fp8g.gemm_block128(code(a).cuda(), sa.cuda(), code(b).cuda(), sb.cuda(), form=form, out="f32")
    settled(fp8g)
    assert torch.equal(C.cpu().double(), want)


@pytest.mark.parametrize("M", [24, 300])
def test_not_finite_stays_in_its_row_and_column(fp8g, M):
    N, K = 256, 512
    A, B, _, _ = operands("nt", M, N, K, E4M3, E4M3, gen(7, M))
    plain = fp8g.gemm_block128(*(t.cuda() for t in A + B), out="f32")
    qa, qb = A[0].clone(), B[0].clone()
    qa[5, 130] = 0x7F
    qb[77, 400] = 0xFF
    C = fp8g.gemm_block128(qa.cuda(), A[1].cuda(), qb.cuda(), B[1].cuda(), out="f32")
    settled(fp8g)
    nan = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    nan[5] = nan[:, 77] = True
    assert torch.equal(C.isnan(), nan) and torch.equal(C[~nan], plain[~nan])


def test_no_rows_and_no_sum(fp8g):
    A, B, _, _ = operands("nt", 3, 16, 32, E4M3, E4M3, gen(8))
    C = fp8g.gemm_block128(A[0][:0].cuda(), A[1][:, :0].contiguous().cuda(), *(t.cuda() for t in B))
    assert C.shape == (0, 16)
    e = lambda n: torch.empty((0, n), device="cuda")
    u = lambda n: torch.empty((0, n), dtype=torch.uint8, device="cuda")
    C = fp8g.gemm_block128(u(32), e(32), u(48), e(48), form="tn", out="f32")
    assert torch.equal(C, torch.zeros((32, 48), device="cuda"))
    kept = torch.randn((32, 48), device="cuda")
    want = kept.clone()
    assert torch.equal(fp8g.gemm_block128(u(32), e(32), u(48), e(48), form="tn", add_to=kept), want)


@pytest.mark.parametrize("form,M", [("nt", 40), ("nt", 200), ("nn", 130), ("tn", 144)])
def test_rows_behind_the_output_stay(fp8g, form, M):
    N, K = 144, 160
    A, B, _, _ = operands(form, M, N, K, E4M3, E4M3, gen(9, form))
    A, B = [t.cuda() for t in A], [t.cuda() for t in B]
    for out, dt in ((0, torch.bfloat16), (1, torch.float32)):
        C = torch.full((M + 70, N), 7.0, dtype=dt, device="cuda")
        fp8g.fp8_gemm_block128({"nt": 0, "nn": 1, "tn": 2}[form], A[0], A[1], 0, B[0], B[1], 0, C, out, 0, M, N, K)
        settled(fp8g)
        assert (C[M:] == 7).all()
        assert torch.equal(C[:M], fp8g.gemm_block128(*A, *B, form=form, out="f32" if out else "bf16"))


def test_unaligned_rows_of_the_output(fp8g):
    # C 16- but not 32-byte aligned, rows no multiple of 32 bytes
    M, N, K = 300, 136, 256
    A, B, _, _ = operands("nt", M, N, K, E4M3, E4M3, gen(10))
    A, B = [t.cuda() for t in A], [t.cuda() for t in B]
    room = torch.zeros(M * N + 8, dtype=torch.bfloat16, device="cuda")
    fp8g.fp8_gemm_block128(0, A[0], A[1], 0, B[0], B[1], 0, room[8:], 0, 0, M, N, K)
    settled(fp8g)
    assert torch.equal(room[8:].view(M, N), fp8g.gemm_block128(*A, *B))


def test_repeat_streams_and_graph(fp8g):
    cases = []
    for form, M in (("nt", 9), ("nt", 500), ("nn", 70), ("tn", 272)):
        A, B, _, _ = operands(form, M, 1040, 2048, E4M3, E4M3, gen(11, form, M))
        cases.append((form, [t.cuda() for t in A + B]))
    want = [fp8g.gemm_block128(*t, form=f, out="f32") for f, t in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s, (f, t) in zip(streams, cases):
            with torch.cuda.stream(s):
                got.append(fp8g.gemm_block128(*t, form=f, out="f32"))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    own = torch.cuda.Stream()
    with torch.cuda.stream(own):
        fp8g.gemm_block128(*cases[0][1], stream=own)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = [fp8g.gemm_block128(*t, form=f, out="f32") for f, t in cases]
    for _ in range(2):
        [c.zero_() for c in got]
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    settled(fp8g)


# ----------------------------------------------------------------------- gated

def check_gated(fp8g, M, F, K, gate, keep):
    g = gen(12, M, F, K, gate)
    x, sx = ref.quant(ref.values(M, K, g), "row", E4M3)
    W, sw = ref.quant(ref.values(2 * F, K, g, zeros=False) * K ** -0.5, "tile", E4M3)
    h, gu = fp8g.gated_block128(x.cuda(), sx.cuda(), W.cuda(), sw.cuda(), gate=gate, keep=keep)
    settled(fp8g)
    both, mags = ref.product(ref.decode(x, sx, "row", E4M3), ref.decode(W, sw, "tile", E4M3), "nt")
    err = ref.sum_tol(K) * mags
    gg, uu = both[:, :F], both[:, F:]
    y, d = ref.act(gg, gate)
    # act' is at most 1.13 in magnitude; act itself within 2^-20 (2 + |g|) |g|; a product's rounding
    eh = (1.13 * err[:, :F] + 2.0 ** -20 * (2 + gg.abs()) * gg.abs()) * (uu.abs() + err[:, F:]) + y.abs() * err[:, F:] \
        + 2.0 ** -23 * (y * uu).abs()
    ref.assert_coded(h[0].cpu(), h[1].cpu(), "row", E4M3, y * uu, eh)
    if keep:
        ref.assert_coded(gu[0].cpu(), gu[1].cpu(), "row", E4M3, both, err)
    else:
        assert gu is None


@pytest.mark.parametrize("M,F,K", [(1, 128, 16), (1, 1408, 1024), (7, 256, 144), (16, 128, 272), (31, 384, 640),
                                   (64, 256, 2064), (128, 256, 256)])
@pytest.mark.parametrize("gate", [0, 1, 2])
def test_gated_few_rows(fp8g, M, F, K, gate):
    check_gated(fp8g, M, F, K, gate, keep=gate != 1)
    check_gated(fp8g, M, F, K, gate, keep=gate == 1)


@pytest.mark.parametrize("M,F,K", [(129, 128, 128), (256, 256, 16), (300, 384, 400), (1030, 640, 272)])
@pytest.mark.parametrize("gate", [0, 1, 2])
def test_gated(fp8g, M, F, K, gate):
    check_gated(fp8g, M, F, K, gate, keep=True)
    check_gated(fp8g, M, F, K, gate, keep=False)


# -------------------------------------------------------------------- backward

@pytest.mark.parametrize("M,F", [(1, 128), (5, 256), (128, 128), (129, 384), (300, 1408)])
@pytest.mark.parametrize("gate", [0, 1, 2])
@pytest.mark.parametrize("dtype,fmt", [("bf16", E4M3), ("f32", E5M2)])
def test_backward(fp8g, M, F, gate, dtype, fmt):
    r = gen(13, M, F, gate)
    gu, sgu = ref.quant(ref.values(M, 2 * F, r), "row", E4M3)
    dh = ref.values(M, F, r) * 1e-3
    dh = dh.bfloat16() if dtype == "bf16" else dh
    row, col, h = fp8g.gated_block128_backward(dh.cuda(), gu.cuda(), sgu.cuda(), gate=gate, fmt=fmt)
    both = ref.decode(gu, sgu, "row", E4M3)
    g, u, x = both[:, :F], both[:, F:], dh.double()
    y, d = ref.act(g, gate)
    want = torch.cat((x * u * d, x * y), 1)
    # sigmoid and its like within 2^-22 (1 + |g| / 4), derivative and value from them with few roundings
    e = 2.0 ** -19 * (2 + g.abs())
    err = torch.cat((x.abs() * u.abs() * e, x.abs() * (g.abs() * e)), 1)
    ref.assert_coded(row[0].cpu(), row[1].cpu(), "row", fmt, want, err)
    ref.assert_coded(col[0].cpu(), col[1].cpu(), "col", fmt, want, err)
    ref.assert_coded(h[0].cpu(), h[1].cpu(), "col", E4M3, y * u, g.abs() * u.abs() * e)


@pytest.mark.parametrize("gate", [0, 1, 2])
def test_backward_against_differences(fp8g, gate):
    M, F = 40, 128
    r = gen(14, gate)
    gu, sgu = ref.quant(ref.values(M, 2 * F, r), "row", E4M3)
    dh = ref.values(M, F, r, zeros=False)
    row, _, _ = fp8g.gated_block128_backward(dh.cuda(), gu.cuda(), sgu.cuda(), gate=gate)
    both = ref.decode(gu, sgu, "row", E4M3)
    g, u, x = both[:, :F], both[:, F:], dh.double()
    step = 1e-5
    h = lambda a, b: ref.act(a, gate)[0] * b
    want = torch.cat((x * (h(g + step, u) - h(g - step, u)), x * (h(g, u + step) - h(g, u - step))), 1) / (2 * step)
    got = ref.decode(row[0].cpu(), row[1].cpu(), "row", E4M3)
    # a code's half step; differences: 64-bit rounding over the step (1e-10 of the terms) and the
    # third derivative, below 2, times step^2 / 6
    tol = 1.001 * ref.HALF[0] * want.abs() + ref.SUB[0] * ref.spread(row[1].cpu(), "row", M, 2 * F).double()
    tol = tol + (1e-9 + 2.0 ** -19 * (2 + g.abs())).repeat(1, 2) * (x.abs() * (1 + u.abs()) * (1 + g.abs())).repeat(1, 2)
    smooth = torch.ones_like(want, dtype=torch.bool)
    if gate == 2:  # the corner of ReLU has no derivative
        smooth[:, :F] = g.abs() > step
    assert (((got - want).abs() <= tol) | ~smooth).all()


def test_backward_not_finite_and_empty(fp8g):
    M, F = 140, 256
    gu, sgu = ref.quant(ref.values(M, 2 * F, gen(15)), "row", E4M3)
    dh = ref.values(M, F, gen(16))
    plain = fp8g.gated_block128_backward(dh.cuda(), gu.cuda(), sgu.cuda())
    dh[3, 17] = math.nan
    row, col, h = fp8g.gated_block128_backward(dh.cuda(), gu.cuda(), sgu.cuda())
    code = lambda p: p[0].view(torch.float8_e4m3fn).float()
    assert code(row)[3, 17].isnan() and code(row)[3, F + 17].isnan() and code(row).isnan().sum() == 2
    assert code(col).isnan().sum() == 2 and torch.equal(h[0], plain[2][0])
    others = [i for i in range(M) if i != 3]
    assert torch.equal(row[0][others], plain[0][0][others])
    row, col, h = fp8g.gated_block128_backward(dh[:0].cuda(), gu[:0].cuda(), sgu[:, :0].contiguous().cuda())
    assert row[0].shape == (0, 2 * F) and col[1].shape == (0, 2 * F) and h[0].shape == (0, F)


def test_backward_rows_behind_stay(fp8g):
    M, F = 30, 128
    gu, sgu = ref.quant(ref.values(M, 2 * F, gen(17)), "row", E4M3)
    dh = ref.values(M, F, gen(18)).cuda()
    a, b, c = (torch.full((M + 9, w), 0x55, dtype=torch.uint8, device="cuda") for w in (2 * F, 2 * F, F))
    s = [torch.empty(n, device="cuda") for n in (2 * M, 2 * F, F)]
    fp8g.fp8g_gated_block128_backward(dh, fp8g.FP8G_IN_F32, gu.cuda(), sgu.cuda(), 0, 0, M, F, a, s[0], b, s[1], c, s[2])
    settled(fp8g)
    assert all((t[M:] == 0x55).all() for t in (a, b, c))


# --------------------------------------- more tiles than the kernels' grids: several a CTA

@pytest.mark.parametrize("form,M,N,K", [("nt", 2100, 2600, 144), ("nn", 2100, 2592, 400), ("tn", 2064, 2832, 260),
                                        ("nt", 130, 5000, 1040), ("tn", 4096, 4096, 128),
                                        # K blocks of tiles shared between pairs: all tiles, the last ones
                                        ("nn", 1500, 1040, 16000), ("tn", 272, 400, 12000), ("tn", 16, 16, 12001),
                                        ("nt", 4100, 1288, 16384), ("tn", 2304, 2304, 16400)])
@pytest.mark.parametrize("out", ["bf16", "add"])
def test_many_tiles(fp8g, form, M, N, K, out):
    r = torch.Generator(device="cuda").manual_seed(19)

    def coded(R, C, kind, x):
        if kind == "tile":
            return fp8g.quantize_tile128(x)
        return fp8g.quantize_block128(x, row=kind == "row", col=kind == "col")[kind == "col"]
    rand = lambda *s: torch.randn(s, device="cuda", generator=r)
    if form == "tn":
        A, B, ka, kb = coded(K, M, "col", rand(K, M)), coded(K, N, "col", rand(K, N)), "col", "col"
    else:
        b = rand(N, K) if form == "nt" else rand(K, N)
        A, B, ka, kb = coded(M, K, "row", rand(M, K)), coded(*b.shape, "tile", b), "row", "tile"
    C = rand(M, N) if out == "add" else None
    start = C.clone() if out == "add" else None
    got = fp8g.gemm_block128(*A, *B, form=form, add_to=C)
    settled(fp8g)
    want, mags = ref.product(ref.decode(*A, ka, E4M3), ref.decode(*B, kb, E4M3), form)
    tol = ref.sum_tol(K) * mags
    if out == "add":
        want = want + start.double()
        tol = tol + 2.0 ** -24 * want.abs()
    else:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    assert ((got.double() - want).abs() <= tol).all()
    again = fp8g.gemm_block128(*A, *B, form=form, add_to=start)
    assert torch.equal(again, got)


@pytest.mark.parametrize("M,F,K", [(1500, 2048, 272), (1030, 384, 4112), (3000, 1024, 4096)])
def test_many_tiles_gated_and_back(fp8g, M, F, K):
    r = torch.Generator(device="cuda").manual_seed(20)
    x, _ = fp8g.quantize_block128(torch.randn((M, K), device="cuda", generator=r))
    W = fp8g.quantize_tile128(torch.randn((2 * F, K), device="cuda", generator=r) * K ** -0.5)
    h, gu = fp8g.gated_block128(*x, *W, keep=True)
    settled(fp8g)
    both, mags = ref.product(ref.decode(*x, "row", E4M3), ref.decode(*W, "tile", E4M3), "nt")
    err = ref.sum_tol(K) * mags
    g, u = both[:, :F], both[:, F:]
    y, _ = ref.act(g, 0)
    ref.assert_coded(*gu, "row", E4M3, both, err)
    eh = (1.13 * err[:, :F] + 2.0 ** -20 * (2 + g.abs()) * g.abs()) * (u.abs() + err[:, F:]) + y.abs() * err[:, F:] \
        + 2.0 ** -23 * (y * u).abs()
    ref.assert_coded(*h, "row", E4M3, y * u, eh)
    dh = torch.randn((M, F), device="cuda", generator=r).bfloat16()
    row, col, hc = fp8g.gated_block128_backward(dh, *gu)
    both = ref.decode(*gu, "row", E4M3)
    g, u, xx = both[:, :F], both[:, F:], dh.double()
    y, d = ref.act(g, 0)
    e = 2.0 ** -19 * (2 + g.abs())
    want = torch.cat((xx * u * d, xx * y), 1)
    err = torch.cat((xx.abs() * u.abs() * e, xx.abs() * (g.abs() * e)), 1)
    ref.assert_coded(*row, "row", E4M3, want, err)
    ref.assert_coded(*col, "col", E4M3, want, err)
    ref.assert_coded(*hc, "col", E4M3, y * u, g.abs() * u.abs() * e)


def test_quantise_bits_many_tiles(fp8g):
    x = ref.values(2500, 1200, gen(21))
    row, col = fp8g.quantize_block128(x.bfloat16().cuda(), row=True, col=True)
    same(row, ref.quant(x.bfloat16(), "row", E4M3))
    same(col, ref.quant(x.bfloat16(), "col", E4M3))
    same(fp8g.quantize_block128(x.cuda())[0], ref.quant(x, "row", E4M3))


@pytest.mark.parametrize("arg", ["A", "sfa", "B", "sfb", "add_to"])
def test_the_product_refuses_what_does_not_fit(fp8g, arg):
    u = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    f = lambda *s: torch.ones(s, device="cuda")
    good = dict(A=u(32, 256), sfa=f(2, 32), B=u(64, 256), sfb=f(1, 2), add_to=f(32, 64))
    fp8g.gemm_block128(**good)
    bad = {"A": [u(32, 240), u(256, 32).t(), torch.zeros((32, 256), device="cuda"), u(32, 256).cpu()],
           "sfa": [f(32, 2), f(2, 32).double(), f(4, 32)[::2]], "B": [u(64, 128), u(256, 64).t()],
           "sfb": [f(2, 1), f(1, 2).bfloat16()], "add_to": [f(64, 32), f(32, 64).bfloat16(), f(64, 32).t()]}[arg]
    for t in bad:
        with pytest.raises((AssertionError, fp8g.Fp8gError)):
            fp8g.gemm_block128(**dict(good, **{arg: t}))
    settled(fp8g)


def test_shared_tiles_at_once_and_replayed(fp8g):
    r = torch.Generator(device="cuda").manual_seed(22)
    rand = lambda *s: torch.randn(s, device="cuda", generator=r)
    cases = []
    for M, N in ((272, 400), (1040, 784), (16, 16)):
        A, B = (fp8g.quantize_block128(rand(12000, n), row=False, col=True)[1] for n in (M, N))
        cases.append((*A, *B))
    call = lambda t: fp8g.gemm_block128(*t, form="tn", out="f32")
    want = [call(t) for t in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s, t in zip(streams, cases):
            with torch.cuda.stream(s):
                got.append(call(t))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, got = [], []
    for t in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(call(t))
        graphs.append(g)
    [c.zero_() for c in got]
    torch.cuda.synchronize()
    for _ in range(3):  # two graphs at once, an eager call beside them
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        eager = call(cases[1])
        torch.cuda.synchronize()
        assert torch.equal(eager, want[1])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        [c.zero_() for c in got]
        torch.cuda.synchronize()
    settled(fp8g)


def test_codes_of_another_type_are_refused(fp8g):
    x = torch.randn((32, 256), device="cuda")
    W, sw = fp8g.quantize_tile128(torch.randn((256, 256), device="cuda"))
    q = {f: fp8g.quantize_block128(x, fmt=f)[0] for f in (E4M3, E5M2)}
    for f, typed in ((E4M3, torch.float8_e4m3fn), (E5M2, torch.float8_e5m2)):
        (a, s), other = q[f], 1 - f
        want = fp8g.gemm_block128(a, s, W, sw, a_fmt=f)
        assert torch.equal(fp8g.gemm_block128(a.view(typed), s, W, sw, a_fmt=f), want)
        for bad in (lambda: fp8g.gemm_block128(a.view(typed), s, W, sw, a_fmt=other),
                    lambda: fp8g.gemm_block128(a.view(torch.int8), s, W, sw, a_fmt=f),
                    lambda: fp8g.gated_block128(a.view(typed), s, W, sw, x_fmt=other),
                    lambda: fp8g.requantize_block128(a.view(typed), s, q_fmt=other)):
            with pytest.raises(AssertionError):
                bad()
    h, gu = fp8g.gated_block128(*q[E4M3], W, sw, keep=True)
    dh = torch.randn((32, 128), device="cuda")
    with pytest.raises(AssertionError):
        fp8g.gated_block128_backward(dh, gu[0].view(torch.float8_e5m2), gu[1])
    settled(fp8g)


@pytest.mark.parametrize("M", [5, 130, 300])
def test_gated_rows_behind_stay(fp8g, M):
    F, K = 256, 272
    x, _ = fp8g.quantize_block128(torch.randn((M, K), device="cuda"))
    W = fp8g.quantize_tile128(torch.randn((2 * F, K), device="cuda"))
    h = torch.full((M + 200, F), 0x55, dtype=torch.uint8, device="cuda")
    gu = torch.full((M + 200, 2 * F), 0x55, dtype=torch.uint8, device="cuda")
    sh, sgu = torch.zeros((F // 128, M), device="cuda"), torch.zeros((2 * F // 128, M), device="cuda")
    fp8g.fp8_gated_block128(x[0], x[1], E4M3, W[0], W[1], E4M3, 0, h, sh, gu, sgu, M, F, K)
    settled(fp8g)
    assert (h[M:] == 0x55).all() and (gu[M:] == 0x55).all()
    want = fp8g.gated_block128(*x, *W, keep=True)
    assert torch.equal(h[:M], want[0][0]) and torch.equal(sh, want[0][1])
    assert torch.equal(gu[:M], want[1][0]) and torch.equal(sgu, want[1][1])
