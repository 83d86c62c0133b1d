"""The projection with low-rank adapters against its definition in 64 bits.

Most cases are exact: small integers, so that every fp32 sum is exact in any
order and V = alpha A x fits the 16 bits it is held to; outputs have to be equal."""
import pytest
import torch

import fp8_block_scaled_06_gb300 as fp8g

pytestmark = pytest.mark.gpu
FORMATS = (fp8g.FP8G_E4M3, fp8g.FP8G_E5M2, fp8g.FP8G_E2M1, fp8g.FP8G_E2M3, fp8g.FP8G_E3M2)


class Projection:
    def __init__(self, M, N, K, L, r, fmt=fp8g.FP8G_E4M3, seed=0, runs=None):
        gen = torch.Generator().manual_seed(seed * 7919 + M * 31 + N + K)
        self.fmt, self.L = fmt, L

        def ints(shape, density, top):
            v = torch.randint(-top, top + 1, shape, generator=gen).double()
            return v * (torch.rand(shape, generator=gen) < density)
        self.x = ints((M, K), min(1.0, 64 / K), 8)
        self.w = ints((N, K), 1.0, 2)
        self.a = ints((L, r, K), 1.0, 3)
        self.b = ints((L, N, r), 1.0, 3)
        self.alpha = 2.0 ** torch.randint(-2, 3, (L,), generator=gen)
        self.bias = torch.randint(-50, 51, (N,), generator=gen).float()
        runs = runs or M
        who = torch.randint(-1, max(L, 1), (runs,), generator=gen)
        self.adapter = who[torch.arange(M) * runs // max(M, 1)].int() if M else who[:0].int()
        if L == 0:
            self.adapter[:] = -1
        self.W, sf = fp8g.quantize(self.w.float().cuda(), 32, fmt=fmt)
        self.pw = fp8g.pack_scales(sf)

    def reference(self, bias, alpha):
        out = self.x @ self.w.T
        room = self.x.abs() @ self.w.abs().T
        if bias:
            out = out + self.bias
            room = room + self.bias.abs()
        for l in range(self.L):
            at = self.adapter == l
            v = self.x[at] @ self.a[l].T * (self.alpha[l].double() if alpha else 1)
            out[at] += v @ self.b[l].T
            room[at] += v.abs() @ self.b[l].abs().T
        return out, room

    def run(self, out="f32", bf16=True, bias=True, alpha=True):
        x = self.x.bfloat16() if bf16 else self.x.float()
        return fp8g.gemm_lora(x.cuda(), self.W, self.pw, self.a.bfloat16().cuda(), self.b.bfloat16().cuda(),
                              self.alpha.float().cuda() if alpha else None, self.adapter.cuda(),
                              bias=self.bias.cuda() if bias else None, w_fmt=self.fmt, out=out)

    def check_exact(self):
        ref, room = self.reference(True, True)
        assert float(room.max()) * 4 < 2 ** 24  # alpha is a multiple of 1/4: exact in fp32
        got = self.run()
        assert fp8g.fp8_gemm_status()[0] == 0
        assert torch.equal(got.cpu().double(), ref)
        ref, _ = self.reference(False, False)
        got = self.run("bf16", bf16=False, bias=False, alpha=False)
        assert fp8g.fp8_gemm_status()[0] == 0
        assert torch.equal(got.cpu(), ref.float().bfloat16())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K,L,r", [(1, 128, 128, 1, 8), (20, 264, 384, 5, 16), (600, 136, 256, 4, 24)])
def test_formats(M, N, K, L, r, fmt):
    Projection(M, N, K, L, r, fmt).check_exact()


# single tokens, each boundary of the token columns and of the two paths, odd
# tiles, splits of a long K, ranks that end inside a block
@pytest.mark.parametrize("M,N,K,L,r", [
    (1, 8, 32, 1, 8), (2, 136, 2080, 3, 16), (16, 520, 96, 16, 40), (17, 128, 1024, 40, 64),
    (33, 1000, 416, 8, 72), (64, 256, 160, 1024, 8), (65, 256, 160, 7, 256), (80, 264, 128, 3, 16),
    (96, 128, 64, 2, 8), (112, 392, 288, 9, 32), (128, 640, 512, 32, 64), (129, 128, 128, 5, 136),
    (400, 136, 96, 300, 8), (512, 264, 160, 4, 64), (513, 264, 160, 4, 64), (700, 520, 96, 3, 200),
    (1500, 128, 64, 20, 16)])
def test_sizes(M, N, K, L, r):
    Projection(M, N, K, L, r).check_exact()


@pytest.mark.parametrize("M", [48, 128, 300, 900])
def test_runs_of_rows_of_one_adapter(M):
    Projection(M, 264, 160, 3, 16, runs=3).check_exact()
    Projection(M, 136, 96, 1, 88, runs=1, seed=1).check_exact()


@pytest.mark.parametrize("M", [1, 40, 200, 600])
def test_no_adapters(M):
    Projection(M, 136, 160, 0, 8).check_exact()
    p = Projection(M, 136, 160, 4, 8)
    p.adapter[:] = -1
    p.check_exact()


def test_no_rows():
    assert Projection(0, 64, 64, 2, 8).run().shape == (0, 64)


@pytest.mark.parametrize("M", [3, 40, 600])
def test_adapter_out_of_range(M):
    p = Projection(M, 136, 160, 4, 8)
    p.adapter[2] = 4
    ref, _ = p.reference(True, True)  # the row gets no adapter
    got = p.run()
    assert fp8g.fp8_gemm_status() == (fp8g.FP8G_ERR_INVALID_ARG, 2)
    assert torch.equal(got.cpu().double(), ref)


@pytest.mark.parametrize("M", [5, 100, 600])
def test_non_finite_rows_stay_where_they_are(M):
    p = Projection(M, 136, 160, 2, 8)
    want = p.run()
    p.x[1, 3] = float("nan")
    p.x[3, 0] = float("inf")
    got = p.run()
    keep = torch.ones(M, dtype=torch.bool)
    keep[[1, 3]] = False
    assert torch.equal(got[keep.cuda()], want[keep.cuda()]) and torch.isnan(got[1]).all()


@pytest.mark.parametrize("M,N,K,L,r", [(1, 512, 1024, 4, 16), (50, 264, 768, 8, 48), (128, 136, 1024, 16, 64),
                                       (700, 264, 512, 4, 16)])
def test_random_values(M, N, K, L, r):
    """x rounded by Q, V to 16 bits (2^-16), K + r fp32 additions, the output's bf16."""
    p = Projection(M, N, K, L, r)
    gen = torch.Generator().manual_seed(3)
    x32 = torch.randn((M, K), generator=gen)
    p.x = x32.double()
    p.a = (torch.randn((L, r, K), generator=gen) / K ** 0.5).bfloat16().double()
    p.b = torch.randn((L, N, r), generator=gen).bfloat16().double()
    q, s = fp8g.quantize(x32.cuda(), 32)
    qx = (q.cpu().view(torch.float8_e4m3fn).double().view(M, -1, 32) * s.cpu().double()[..., None]).view(M, K)
    ref, room = qx @ p.w.T, qx.abs() @ p.w.abs().T
    low = torch.zeros_like(ref)
    for l in range(L):
        at = p.adapter == l
        v = p.x[at] @ p.a[l].T * p.alpha[l].double()
        ref[at] += v @ p.b[l].T
        low[at] += (p.x[at].abs() @ p.a[l].abs().T * p.alpha[l].double()) @ p.b[l].abs().T
    tol = (K + r + 2) * 2.0 ** -22 * (room + low) + 3 * 2.0 ** -16 * low
    got = p.run(bf16=False, bias=False).cpu().double()
    assert ((got - ref).abs() <= tol).all()
    got = p.run("bf16", bf16=False, bias=False).cpu().double()
    assert ((got - ref).abs() <= tol + 2.0 ** -8 * ref.abs() + 2.0 ** -130).all()


@pytest.mark.parametrize("M", [30, 600])
def test_repeats_streams_and_graph(M):
    p = Projection(M, 392, 1024, 6, 16)
    gen = torch.Generator().manual_seed(9)
    p.x = torch.randn((M, 1024), generator=gen).bfloat16().double()
    want = p.run()
    for _ in range(5):
        assert torch.equal(p.run(), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [p.run() for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(g, want) for g in got)
    args = (p.x.bfloat16().cuda(), p.W, p.pw, p.a.bfloat16().cuda(), p.b.bfloat16().cuda(),
            p.alpha.float().cuda(), p.adapter.cuda())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fp8g.gemm_lora(*args, bias=None, out="f32")
    graph.replay()
    assert torch.equal(out, p.run(bias=False))


def test_same_projection_as_the_plain_gemm():
    """Without adapters: the block-scaled GEMM of the quantised rows, where sums are exact."""
    p = Projection(70, 264, 160, 0, 8)
    q, s = fp8g.quantize(p.x.float().cuda(), 32)
    _, sw = fp8g.quantize(p.w.float().cuda(), 32)
    assert torch.equal(p.run(bias=False), fp8g.gemm(q, p.W, s, sw, out="f32"))


@pytest.mark.parametrize("n,rows,K", [(1, 1, 32), (1, 128, 128), (3, 200, 160), (2, 1440, 2080)])
def test_pack_scales(n, rows, K):
    gen = torch.Generator().manual_seed(rows)
    sf = 2.0 ** torch.randint(-126, 128, (n, rows, K // 32), generator=gen).float()
    nk, nr = -(-K // 128), -(-rows // 128)
    c = torch.full((n, nr * 128, nk * 4), 127, dtype=torch.uint8)
    c[:, :rows, :K // 32] = (sf.view(torch.int32) >> 23).to(torch.uint8)
    want = c.view(n, nr, 4, 32, nk, 4).permute(0, 4, 1, 3, 2, 5).reshape(n, nk, nr, 512)
    got = fp8g.pack_scales(sf.cuda())
    assert fp8g.fp8_gemm_status()[0] == 0
    assert torch.equal(got.cpu(), want)
    assert fp8g._packed_bytes(n, rows, K) == got.numel()
    sf[0, 0, 0] = 3.0
    fp8g.pack_scales(sf.cuda())
    assert fp8g.fp8_gemm_status()[0] == fp8g.FP8G_ERR_SCALE_FORMAT


@pytest.mark.parametrize("M,N,K,L,r", [(129, 136, 1024, 1, 8), (200, 264, 1056, 2, 32), (300, 520, 2048, 1, 72),
                                       (512, 128, 1024, 4, 16)])
def test_few_adapters_of_many_rows(M, N, K, L, r):
    """From 129 rows on a call with few adapters beside its K takes the path of the prompts."""
    Projection(M, N, K, L, r).check_exact()


def test_calls_on_several_streams():
    ps = [Projection(m, 520, 1056, 5, 16, seed=m) for m in (1, 40, 128, 700)]
    want = [p.run() for p in ps]
    args = [(p.x.bfloat16().cuda(), p.W, p.pw, p.a.bfloat16().cuda(), p.b.bfloat16().cuda(),
             p.alpha.float().cuda(), p.adapter.cuda(), p.bias.cuda()) for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    got = [[] for _ in ps]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(fp8g.gemm_lora(*args[i], out="f32"))
    torch.cuda.synchronize()
    assert fp8g.fp8_gemm_status()[0] == 0
    assert all(torch.equal(g, w) for w, gs in zip(want, got) for g in gs)


@pytest.mark.parametrize("M", [5, 100, 600])
def test_non_finite_adapter_values_stay_with_its_rows(M):
    """A and alpha of one adapter, a value of W: NaN in its rows, its column."""
    p = Projection(M, 136, 160, 3, 8)
    want = p.run()
    p.a[1, 2, 7] = float("nan")
    p.alpha[2] = float("inf")
    got = p.run()
    others = ((p.adapter != 1) & (p.adapter != 2)).cuda()
    assert torch.equal(got[others], want[others])
    hit = (p.adapter == 1) & (p.x[:, 7] != 0)
    assert torch.isnan(got[hit.cuda()]).any(1).all()
    p = Projection(M, 136, 160, 3, 8)
    p.W[40, 3] = 0x7F  # NaN
    got = p.run()
    keep = torch.arange(136) != 40
    assert torch.equal(got[:, keep.cuda()], want[:, keep.cuda()]) and torch.isnan(got[:, 40]).all()


@pytest.mark.parametrize("r", [0, 8, 16, 256, 300, -1])
@pytest.mark.parametrize("M", [1, 40, 128, 129, 600])
def test_no_adapters_null_pointers(M, r):
    """With L = 0 lora_a, lora_b and adapter may be null, and r says nothing."""
    p = Projection(M, 136, 160, 0, 8)
    x, bias = p.x.bfloat16().cuda(), p.bias.cuda()
    C = torch.full((M, 136), float("nan"), device="cuda")
    fp8g.fp8_gemm_lora(x, fp8g.FP8G_IN_BF16, p.W, p.pw, p.fmt, None, None, None, None, 0, r, bias, C,
                       fp8g.FP8G_OUT_F32, M, 136, 160)
    assert fp8g.fp8_gemm_status()[0] == 0
    ref, _ = p.reference(True, False)
    assert torch.equal(C.cpu().double(), ref)


def poisoned(M, N, K, L, r, at, fmt=fp8g.FP8G_E4M3, runs=None):
    p = Projection(M, N, K, L, r, fmt, runs=runs)
    nan, inf = float("nan"), float("inf")
    if at == "all":
        p.b[1] = inf
    elif at == "some":
        p.b[1, 3, 0], p.b[1, N - 1, r - 1], p.b[0, 5, 2], p.b[0, N // 2] = nan, -inf, inf, nan
    else:  # a column of NaN in every adapter but the last
        p.b[:-1, :, r // 2] = nan
    return p


def check_poisoned(p):
    ref, _ = p.reference(True, True)
    clean = torch.isfinite(p.b).all(2)  # [L, N]
    own = torch.ones_like(ref, dtype=torch.bool)  # outputs whose own row of B is finite
    for l in range(p.L):
        own[p.adapter == l] = clean[l]
    assert torch.isfinite(ref[own]).all()
    for out, bf16 in (("f32", True), ("bf16", False)):
        got = p.run(out, bf16=bf16).cpu()
        assert fp8g.fp8_gemm_status()[0] == 0
        want = ref if out == "f32" else ref.float().bfloat16()
        torch.testing.assert_close(got.to(want.dtype), want, rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("at", ["all", "some", "column"])
@pytest.mark.parametrize("M,N,K,L,r,runs", [
    (5, 136, 160, 3, 8, None), (33, 264, 416, 16, 16, None), (100, 136, 96, 4, 72, None),
    (128, 520, 160, 32, 64, None), (300, 136, 1056, 2, 8, None), (400, 136, 96, 40, 40, None),
    (600, 264, 160, 3, 8, None), (700, 136, 96, 5, 136, 9), (1, 128, 6144, 2, 8, None),
    (20, 136, 5120, 5, 136, None)])
def test_non_finite_b_stays_with_its_rows(M, N, K, L, r, runs, at):
    """Every output is that of the definition: other adapters' rows, rows without an
    adapter and features whose row of B is finite have their values, the others the
    infinity or NaN that they sum to."""
    p = poisoned(M, N, K, L, r, at, runs=runs)
    p.adapter[0] = 1  # some row has a poisoned adapter
    check_poisoned(p)


@pytest.mark.parametrize("M", [20, 600])
@pytest.mark.parametrize("fmt", FORMATS)
def test_non_finite_b_formats(M, fmt):
    p = poisoned(M, 264, 256, 3, 16, "all", fmt)
    p.adapter[:3] = torch.tensor([0, 1, -1], dtype=torch.int32)
    check_poisoned(p)


@pytest.mark.parametrize("M", [24, 600])
def test_non_finite_b_beside_other_nan(M):
    """A NaN of x, of W or of its scales is left where it is."""
    p = poisoned(M, 136, 160, 3, 8, "all")
    p.adapter[:4] = torch.tensor([1, 0, 2, -1], dtype=torch.int32)
    ref, _ = p.reference(True, True)
    p.x[1, 3] = float("nan")
    p.x[3, 8] = float("nan")
    p.W[40, 3] = 0x7F
    p.pw.view(2, 2, 512)[0, 0, 16 * 9] = 255  # the scale of feature 9, first block
    got = p.run().cpu().double()
    assert torch.isnan(got[[1, 3]]).all() and torch.isnan(got[:, [9, 40]]).all()
    rows, cols = torch.ones(M, dtype=torch.bool), torch.ones(136, dtype=torch.bool)
    rows[[1, 3]] = False
    cols[[9, 40]] = False
    torch.testing.assert_close(got[rows][:, cols], ref[rows][:, cols], rtol=0, atol=0, equal_nan=True)


class LowRank(Projection):
    """Only the low-rank term: W is zero, alpha 1, a row's V the sums of `terms`
    products, B one rank in each feature, so that the fp32 output is V itself."""

    def __init__(self, M, N, K, L, r, top_x, top_a, terms, runs=None):
        super().__init__(M, N, K, L, r, runs=runs)
        gen = torch.Generator().manual_seed(M + r)
        self.W.zero_()
        self.pw = fp8g.pack_scales(torch.ones((N, K // 32), device="cuda"))
        self.w.zero_()
        self.alpha[:] = 1
        self.adapter[0] = 0  # one row at least has an adapter
        where = torch.rand((M, K), generator=gen).argsort(1) < terms
        self.x = torch.randint(-top_x, top_x + 1, (M, K), generator=gen).double() * where
        self.a = torch.randint(-top_a, top_a + 1, (L, r, K), generator=gen).double()
        self.b = torch.zeros((L, N, r), dtype=torch.double)
        at = torch.randint(0, r, (L, N), generator=gen)
        self.b.scatter_(2, at[..., None], torch.randint(0, 2, (L, N, 1), generator=gen).double() * 2 - 1)


SHAPES = [(1, 128, 512, 1, 8), (20, 264, 96, 3, 16), (33, 136, 160, 2, 24), (40, 136, 2080, 5, 32), (64, 136, 96, 2, 40),
          (128, 264, 160, 9, 64), (100, 136, 96, 2, 72), (300, 136, 1056, 2, 16), (300, 136, 96, 50, 24),
          (600, 136, 160, 3, 8), (600, 264, 96, 4, 24), (700, 136, 160, 5, 136)]


@pytest.mark.parametrize("runs", [None, 2])
@pytest.mark.parametrize("M,N,K,L,r", SHAPES)
def test_v_keeps_24_bits(M, N, K, L, r, runs):
    """bf16 x and A of eight bits, V of up to 23."""
    p = LowRank(M, N, K, L, r, 255, 255, 64, runs)
    ref, room = p.reference(False, False)
    assert float(room.max()) < 2 ** 24 and float(room.max()) > 2 ** 17
    got = p.run(bias=False)
    assert fp8g.fp8_gemm_status()[0] == 0
    assert torch.equal(got.cpu().double(), ref)


@pytest.mark.parametrize("M,N,K,L,r", SHAPES)
def test_fp32_x_keeps_24_bits(M, N, K, L, r):
    """One product a sum, of an x of 24 bits and an A of one."""
    p = LowRank(M, N, K, L, r, 2 ** 24 - 1, 1, 1)
    ref, room = p.reference(False, False)
    got = p.run(bf16=False, bias=False)
    assert fp8g.fp8_gemm_status()[0] == 0
    assert torch.equal(got.cpu().double(), ref)


@pytest.mark.parametrize("M", [3, 600])
def test_largest_finite_x_and_v(M):
    """Finite values stay finite: the pieces of the largest floats are."""
    p = LowRank(M, 136, 96, 2, 8, 1, 1, 1)
    p.x *= torch.finfo(torch.float32).max
    ref, _ = p.reference(False, False)
    got = p.run(bf16=False, bias=False)
    assert torch.equal(got.cpu().double(), ref)


@pytest.mark.parametrize("M,r,L", [(3000, 256, 1024), (4200, 200, 256), (5300, 136, 300)])
def test_rows_in_shares(M, r, L):
    """Many rows of many adapters are taken in shares, which bounds V's temporary."""
    p = Projection(M, 136, 96, L, r)
    p.check_exact()
    p.adapter[M - 100] = L
    ref, _ = p.reference(True, True)
    got = p.run()
    assert fp8g.fp8_gemm_status() == (fp8g.FP8G_ERR_INVALID_ARG, M - 100)
    assert torch.equal(got.cpu().double(), ref)
