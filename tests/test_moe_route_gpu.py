"""The MoE router against its definition in 64 bits: choices and order equal,
weights within the error of their fp32 formula."""
import pytest
import torch

import fp8_block_scaled_06_gb300 as fp8g

pytestmark = pytest.mark.gpu
INF = float("inf")
SCORES = (0, 1, 2, 3)  # softmax, softmax of the chosen, sigmoid, normalised sigmoid


def reference(logits, k, score, scale):
    x = logits.cpu().double()
    x = torch.where(torch.isnan(x), -INF, x)
    v, i = torch.sort(x, dim=1, descending=True, stable=True)
    v, i = v[:, :k], i[:, :k]
    on = v > -INF

    def softmax(of, over):
        top = x.max(1, keepdim=True).values
        top = torch.where(top == -INF, 0.0, top)
        one = torch.where(torch.isinf(top), 1.0, 0.0)  # +inf: shared equally

        def e(a):
            return torch.where(one > 0, (a == INF).double(), torch.exp(a - torch.where(one > 0, 0.0, top)))
        return e(of) / e(over).sum(1, keepdim=True)

    if score == 0:
        w = softmax(v, x)
    elif score == 1:
        w = softmax(v, v)
    else:
        w = 1 / (1 + torch.exp(-v))
        if score == 3:
            w = w / w.sum(1, keepdim=True)
    w = torch.where(on, w * scale, 0.0)
    return torch.where(on, i, -1).int(), w


def check(logits, k, score, scale=1.5, ordered=False):
    E = logits.shape[1]
    got = fp8g.moe_route(logits, k, score, scale, ordered)
    assert fp8g.fp8_gemm_status()[0] == 0
    ids, w = reference(logits, k, score, scale)
    assert torch.equal(got[0].cpu(), ids)
    # exp, a sum of at most E terms, a division, a product, each of a few ulps;
    # values whose exponential underflows: the smallest normal number
    tol = (E + 16) * 2.0 ** -23 * w.abs() + 2.0 ** -126 * scale
    assert ((got[1].cpu().double() - w).abs() <= tol).all()
    if ordered:
        order_of(ids, E, k, *(t.cpu() for t in got[2:]))
    return got


def order_of(ids, E, k, counts, rows, slots):
    flat = ids.reshape(-1).long()
    pairs = [p for e in range(E) for p in torch.nonzero(flat == e).view(-1).tolist()]
    assert counts.tolist() == [int((flat == e).sum()) for e in range(E)]
    n = len(pairs)
    assert slots[:n].tolist() == pairs and rows[:n].tolist() == [p // k for p in pairs]
    assert (slots[n:] == -1).all() and (rows[n:] == -1).all()


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (2, 256, 16), (31, 3, 3), (32, 64, 8),
                                   (33, 64, 6), (33, 65, 5), (257, 33, 4), (1000, 128, 8), (4099, 8, 2)])
def test_matches_definition(T, E, k, score):
    g = torch.Generator().manual_seed(T * 1000 + E)
    x = torch.randn((T, E), generator=g) * 3
    check(x.cuda(), k, score, ordered=True)
    check(x.bfloat16().cuda(), k, score)


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("T", [5, 40])  # both ways of choosing
@pytest.mark.parametrize("E", [24, 100])
def test_masks_ties_and_non_finite(T, E, score):
    x = torch.randn((T, E), generator=torch.Generator().manual_seed(E)) * 2
    x[0] = -INF                      # no expert at all
    x[1, 3:] = -INF                  # fewer than k
    x[2] = 0.25                      # all equal: lower index first
    x[3, ::2] = float("nan")         # never chosen
    x[4, 1] = x[4, 7] = INF          # share the softmax
    # finite, so chosen: the lowest value (whose sigmoid is 0), a low one
    x[T - 1] = torch.finfo(torch.float32).min if score < 2 else -60.0
    check(x.cuda(), 6, score, ordered=True)


def test_zero_tokens():
    got = fp8g.moe_route(torch.empty((0, 8), device="cuda"), 2, ordered=True)
    assert got[0].shape == (0, 2) and got[2].tolist() == [0] * 8


def test_row_stride_and_offset():
    wide = torch.randn((50, 40), device="cuda")
    check(wide[:, 3:20], 4, 1, ordered=True)


def test_long_prompt_order_is_stable():
    x = torch.randn((20000, 64), device="cuda")
    a = fp8g.moe_route(x, 8, ordered=True)
    b = fp8g.moe_route(x, 8, ordered=True)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    ids, counts, rows, slots = a[0], a[2], a[3], a[4]
    flat = ids.reshape(-1)
    assert torch.equal(slots.long(), torch.argsort(flat, stable=True))
    assert torch.equal(rows, slots // 8) and torch.equal(counts.long(), torch.bincount(flat, minlength=64))


def test_other_stream_and_graph():
    x = torch.randn((300, 64), device="cuda")
    want = fp8g.moe_route(x, 4, ordered=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = fp8g.moe_route(x, 4, ordered=True)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    buf = torch.zeros_like(x)
    with torch.cuda.graph(graph):
        got = fp8g.moe_route(buf, 4, ordered=True)
    buf.copy_(x)
    graph.replay()
    assert all(torch.equal(p, q) for p, q in zip(want, got))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(8, 2), (24, 6), (64, 16), (100, 6), (256, 16)])  # both ways of choosing
def test_normalised_sigmoid_of_low_logits(E, k, dtype):
    """Logits whose sigmoid is 0 in fp32: the quotient of the sigmoids stays that of
    the definition, in 64 bits and in logarithms."""
    gen = torch.Generator().manual_seed(E)
    spread = torch.rand((10, E), generator=gen) * 6
    spread[9] *= 15  # some chosen ones have a sigmoid, some none
    low = torch.tensor([-80.0, -88.7, -89.0, -100.0, -1e4, -1e9, 0.0, 60.0, -3.0, -30.0])[:, None]
    x = low - spread
    x = torch.cat([x, torch.full((1, E), torch.finfo(dtype).min), torch.full((1, E), -1e4), x[:1], x[3:4]])
    x[-2, 1:] = -120.0  # one that has a sigmoid, the others none
    x[-1, 2] = INF      # and +inf
    x = x.to(dtype)
    ids, w = fp8g.moe_route(x.cuda(), k, 3, 1.5)
    assert fp8g.fp8_gemm_status()[0] == 0
    v, i = torch.sort(x.double(), dim=1, descending=True, stable=True)
    v, i = v[:, :k], i[:, :k]
    want = 1.5 * torch.softmax(torch.nn.functional.logsigmoid(v), 1)
    assert torch.equal(ids.cpu(), i.int())
    # two exponentials, a difference of logits (exact where the quotient is not
    # small; else within 2^-24 of it, which the exponential turns into that much
    # of itself), two divisions, k additions, a product
    tol = (k + 16 + 256) * 2.0 ** -23 * want + 2.0 ** -126
    assert ((w.cpu().double() - want).abs() <= tol).all()
    assert ((w.sum(1) - 1.5).abs() <= (2 * k + 16) * 2.0 ** -23 * 1.5).all()
