"""The MoE layer of a few tokens against its definition in 64 bits.

Most cases are exact: small integers, so that every fp32 sum is exact in any
order and the quantisation of h has one answer; outputs have to be equal.  The
gates with an exponential get a tolerance."""
import pytest
import torch

import fp8_block_scaled_06_gb300 as fp8g

pytestmark = pytest.mark.gpu
FORMATS = (fp8g.FP8G_E4M3, fp8g.FP8G_E5M2, fp8g.FP8G_E2M1, fp8g.FP8G_E2M3, fp8g.FP8G_E3M2)


def sparse_ints(shape, density, gen, top=1):
    v = torch.randint(-top, top + 1, shape, generator=gen).double()
    return v * (torch.rand(shape, generator=gen) < density)


def encode(w, fmt):
    """Integers [n, rows, K] -> codes, packed scales; exact in every format."""
    n, rows, K = w.shape
    q, s = fp8g.quantize(w.view(-1, K).float().cuda(), 32, fmt=fmt)
    return q.view(n, rows, -1), fp8g.pack_scales(s.view(n, rows, K // 32))


def quantised(h):
    """E4M3 with 1x32 power-of-two scales of fp32 values, as values."""
    b = h.float().reshape(*h.shape[:-1], -1, 32)
    m, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    e = torch.where(m == 0, 0, e - 9 + (m > 0.875).int()).clamp(-126, 127)
    q = torch.ldexp(b, -e).to(torch.float8_e4m3fn).float()
    return torch.ldexp(q, e).reshape(h.shape).double()


def act(g, gate):
    if gate == fp8g.FP8G_GATE_SILU:
        return g / (1 + torch.exp(-g))
    if gate == fp8g.FP8G_GATE_GELU:
        return 0.5 * g * (1 + torch.erf(g / 2 ** 0.5))
    return torch.relu(g)


class Layer:
    def __init__(self, T, E, k, H, F, fmt=fp8g.FP8G_E4M3, seed=0, gate=fp8g.FP8G_GATE_RELU):
        gen = torch.Generator().manual_seed(seed * 7919 + T * 31 + H + F)
        self.k, self.gate, self.fmt = k, gate, fmt
        self.x = sparse_ints((T, H), min(1.0, 48 / H), gen, 2)
        self.w13 = sparse_ints((E, 2 * F, H), 0.5, gen)
        self.w2 = sparse_ints((E, H, F), 0.5, gen)
        self.ids = torch.stack([torch.randperm(E, generator=gen)[:k] for _ in range(T)]).int() if T else \
            torch.empty((0, k), dtype=torch.int32)
        self.w = 2.0 ** torch.randint(-2, 2, (T, k), generator=gen)
        self.W13, s13 = encode(self.w13, fmt)
        self.p13 = fp8g.pack_scales(fp8g.quantize(self.w13.view(-1, H).float().cuda(), 32, fmt=fmt)[1]
                                    .view(2 * E, F, H // 32))
        self.W2, self.p2 = encode(self.w2, fmt)

    def reference(self):
        out = torch.zeros_like(self.x)
        room = torch.zeros_like(self.x)  # sum of magnitudes
        near = torch.zeros_like(self.x)  # what codes next to a rounding boundary can change
        F = self.w2.shape[2]
        for t in range(self.x.shape[0]):
            for j in range(self.k):
                e = int(self.ids[t, j])
                if e < 0 or e >= self.w2.shape[0]:
                    continue
                gu = self.w13[e] @ self.x[t]
                h = act(gu[:F], self.gate) * gu[F:]
                q = quantised(h)
                w = float(self.w[t, j])
                out[t] += w * (self.w2[e] @ q)
                room[t] += w * (self.w2[e].abs() @ q.abs())
                d = 2.0 ** -20 * (gu[:F] * gu[F:]).abs()
                spread = (quantised(h + d) - quantised(h - d)).abs()
                near[t] += w * (self.w2[e].abs() @ spread)
        return out, room, near

    def run(self, out="f32", bf16=True):
        x = self.x.bfloat16() if bf16 else self.x.float()
        o = fp8g.moe_layer(x.cuda(), self.ids.cuda(), self.w.cuda(), self.W13, self.p13, self.W2, self.p2,
                           w_fmt=self.fmt, gate=self.gate, out=out)
        return o

    def check_exact(self, status=0):
        ref, room, _ = self.reference()
        assert float(room.max()) < 2 ** 22 if room.numel() else True  # the sums are exact in fp32
        got = self.run()
        assert fp8g.fp8_gemm_status()[0] == status
        assert torch.equal(got.cpu().double(), ref)
        assert torch.equal(self.run("bf16", bf16=False).cpu(), ref.float().bfloat16())
        fp8g.fp8_gemm_status()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,E,k,H,F", [(1, 4, 2, 128, 128), (7, 8, 3, 384, 256), (40, 4, 4, 256, 640)])
def test_formats(T, E, k, H, F, fmt):
    Layer(T, E, k, H, F, fmt).check_exact()


# one token; odd tiles; a group of 64, 65 and 128 tokens and more; more experts than
# tokens; k = 16; a single step of K; the largest call
@pytest.mark.parametrize("T,E,k,H,F", [
    (1, 1, 1, 32, 32), (1, 8, 2, 2080, 1440), (5, 64, 8, 160, 96), (17, 2, 2, 416, 352),
    (33, 32, 16, 128, 64), (64, 1, 1, 288, 160), (65, 1, 1, 288, 160), (130, 2, 1, 96, 32),
    (300, 3, 2, 64, 96), (512, 2, 2, 128, 128), (2, 256, 2, 64, 32)])
def test_sizes(T, E, k, H, F):
    Layer(T, E, k, H, F).check_exact()


def test_skipped_choices_and_tokens_without_expert():
    l = Layer(12, 4, 2, 160, 96)
    l.ids[3] = -1
    l.ids[5, 0] = -1
    l.ids[7, 1] = -2 ** 31
    l.check_exact()
    l.ids[:] = -1
    l.check_exact()
    assert (l.run() == 0).all()


@pytest.mark.parametrize("T", [2, 60])
def test_expert_out_of_range(T):
    l = Layer(T, 4, 2, 160, 96)
    l.ids[1, 1] = 4
    ref, _, _ = l.reference()
    got = l.run()
    assert fp8g.fp8_gemm_status() == (fp8g.FP8G_ERR_INVALID_ARG, 3)
    assert torch.equal(got.cpu().double(), ref)


def test_repeated_expert_of_a_token():
    l = Layer(9, 4, 3, 128, 64)
    l.ids[:, 1] = l.ids[:, 0]
    l.check_exact()


def test_no_tokens():
    assert Layer(0, 4, 2, 64, 64).run().shape == (0, 64)


def test_experts_without_tokens_are_not_read():
    l = Layer(3, 8, 1, 128, 64)
    l.ids[:] = 2
    want = l.run()
    l.p13.view(16, -1)[6:] = 255  # NaN scales of the others
    l.p2.view(8, -1)[3:] = 255
    assert torch.equal(l.run(), want)


def test_non_finite_token_stays_in_its_row():
    l = Layer(6, 1, 1, 128, 64)
    want = l.run()
    l.x[2, 5] = float("nan")
    got = l.run()
    keep = torch.arange(6) != 2
    assert torch.equal(got[keep.cuda()], want[keep.cuda()]) and torch.isnan(got[2]).any()


@pytest.mark.parametrize("gate", [fp8g.FP8G_GATE_SILU, fp8g.FP8G_GATE_GELU])
@pytest.mark.parametrize("T,E,k,H,F", [(1, 4, 2, 256, 160), (21, 4, 2, 160, 416)])
def test_gates(T, E, k, H, F, gate):
    """g and u are exact; act(g) u is within 2^-20 |g u| (a few ulps of an exponential
    or of 1 + erf), which changes a code only next to a rounding boundary (near);
    then F + k fp32 additions."""
    l = Layer(T, E, k, H, F, gate=gate)
    ref, room, near = l.reference()
    got = l.run().cpu().double()
    assert fp8g.fp8_gemm_status()[0] == 0
    assert ((got - ref).abs() <= near + (F + k + 2) * 2.0 ** -21 * room).all()


def test_repeats_streams_and_graph():
    l = Layer(48, 4, 2, 544, 1120)
    l.w = torch.rand((48, 2)) + 0.1
    l.gate = fp8g.FP8G_GATE_SILU
    want = l.run()
    for _ in range(5):
        assert torch.equal(l.run(), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [l.run() for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(g, want) for g in got)
    x, ids, w = l.x.bfloat16().cuda(), l.ids.cuda(), l.w.cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fp8g.moe_layer(x, ids, w, l.W13, l.p13, l.W2, l.p2, gate=l.gate, out="f32")
    for _ in range(2):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)


def test_route_then_layer():
    """The router's choices as they come, one with an expert masked for all."""
    l = Layer(24, 8, 2, 160, 96)
    logits = torch.randn((24, 8), generator=torch.Generator().manual_seed(5))
    logits[:, 3] = -float("inf")
    logits[4] = -float("inf")
    ids, w = fp8g.moe_route(logits.cuda(), 2)
    l.ids, l.w = ids.cpu(), w.cpu()
    ref, room, _ = l.reference()
    got = l.run().cpu().double()
    assert ((got - ref).abs() <= (96 + 4) * 2.0 ** -21 * room).all()
    assert (got[4] == 0).all()


@pytest.mark.parametrize("T,E,k,H,F", [(512, 16, 16, 64, 64), (33, 256, 16, 64, 32), (127, 20, 7, 96, 160)])
def test_many_pairs(T, E, k, H, F):
    Layer(T, E, k, H, F, seed=2).check_exact()


def test_calls_on_several_streams():
    """Calls in flight together: no CTA waits for one that has not started."""
    layers = [Layer(t, 4, 2, 1056, 1120, seed=t) for t in (1, 20, 64)]
    want = [l.run() for l in layers]
    args = [(l.x.bfloat16().cuda(), l.ids.cuda(), l.w.cuda(), l.W13, l.p13, l.W2, l.p2) for l in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    got = [[] for _ in layers]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(fp8g.moe_layer(*args[i], gate=layers[i].gate, out="f32"))
    torch.cuda.synchronize()
    assert fp8g.fp8_gemm_status()[0] == 0
    assert all(torch.equal(g, w) for w, gs in zip(want, got) for g in gs)
