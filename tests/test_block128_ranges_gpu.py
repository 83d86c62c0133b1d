"""The operators with scales for blocks of 128 at the ends of what they take: offsets past 32 bits,
the most rows, tiles with values that are not finite, a first call under capture, calls from two
threads, other streams."""
import math
import os
import subprocess
import sys
import threading

import pytest
import torch

import block128_ref as ref

pytestmark = pytest.mark.gpu
E4M3, E5M2 = 0, 1
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def settled(fp8g):
    st, detail = fp8g.fp8_gemm_status()
    assert st == 0, (st, detail)


def same(got, want):
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_quantisers_past_32_bits(fp8g):
    R, C, last = 262147, 8208, 131 + 128  # 2.15e9 values; the last rows are a block of columns and a bit
    x = torch.zeros((R, C), device="cuda", dtype=torch.bfloat16)
    x[-last:] = torch.randn((last, C), device="cuda")
    tail = x[-last:].contiguous()
    first = (R - last) // 128  # (whole blocks of zeros)
    assert (R - last) % 128 == 0
    row, col = fp8g.quantize_block128(x, row=True, col=True)
    wr, wc = fp8g.quantize_block128(tail, row=True, col=True)
    same((row[0][-last:], row[1][:, -last:]), wr)
    same((col[0][-last:], col[1][first:]), wc)
    assert (row[1][:, :-last] == 1).all() and (col[1][:first] == 1).all() and not row[0][:-last].any()
    del col
    turned = fp8g.requantize_block128(*row)
    same((turned[0][-last:], turned[1][first:]), fp8g.requantize_block128(wr[0], wr[1]))
    del turned
    only, _ = fp8g.quantize_block128(x)
    same((only[0][-last:], only[1][:, -last:]), wr)
    del only
    tile = fp8g.quantize_tile128(x)
    same((tile[0][-last:], tile[1][first:]), fp8g.quantize_tile128(tail))
    del tile, x
    # an operand past 32 bits: the last rows of the product (of other kernels than those rows alone
    # would have, so sums in another order)
    W = fp8g.quantize_tile128(torch.randn((144, C), device="cuda"))
    C1 = fp8g.gemm_block128(*row, *W, out="f32")
    want, mags = ref.product(ref.decode(*wr, "row", E4M3), ref.decode(*W, "tile", E4M3), "nt")
    assert ((C1[-last:].double() - want).abs() <= ref.sum_tol(C) * mags).all() and not C1[:-last].any()
    settled(fp8g)


def test_outputs_past_32_bits(fp8g):
    M, N, K = 70000, 32768, 128
    r = torch.Generator(device="cuda").manual_seed(1)
    x, _ = fp8g.quantize_block128(torch.randn((M, K), device="cuda", generator=r))
    W = fp8g.quantize_tile128(torch.randn((N, K), device="cuda", generator=r))
    part = lambda t, k: (t[0][-k:].contiguous(), t[1][:, -k:].contiguous())
    C = fp8g.gemm_block128(*x, *W)
    assert torch.equal(C[-300:], fp8g.gemm_block128(*part(x, 300), *W))
    del C
    h, gu = fp8g.gated_block128(*x, *W, keep=True)
    wh, wgu = fp8g.gated_block128(*part(x, 300), *W, keep=True)
    same(part(h, 300) + part(gu, 300), wh + wgu)
    last = M % 128 + 128
    dh = torch.randn((M, N // 2), device="cuda", generator=r).bfloat16()
    row, col, hc = fp8g.gated_block128_backward(dh, *gu)
    wrow, wcol, whc = fp8g.gated_block128_backward(dh[-last:].contiguous(), *part(gu, last))
    same(part(row, last), wrow)
    same((col[0][-last:], col[1][-2:], hc[0][-last:], hc[1][-2:]), wcol + whc)
    settled(fp8g)


def test_the_most_rows(fp8g):
    R, C = 65535 * 16, 16
    r = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((R, C), device="cuda", generator=r)
    row, col = fp8g.quantize_block128(x, row=True, col=True)
    same(fp8g.quantize_block128(x)[0], row)
    k = 1000
    q, s = ref.quant(x[-k:].cpu(), "row", E4M3)
    same((row[0][-k:].cpu(), row[1][:, -k:].cpu()), (q, s))
    k = R % 128 + 128 * 3
    q, s = ref.quant(x[-k:].cpu(), "col", E4M3)
    same((col[0][-k:].cpu(), col[1][-len(s):].cpu()), (q, s))
    W = fp8g.quantize_tile128(torch.randn((16, C), device="cuda", generator=r))
    for n in (R, R + 1):  # both sides of what one grid's second axis takes
        a = torch.cat((row[0], row[0][:1]))[:n].contiguous()
        sa = torch.cat((row[1], row[1][:, :1]), 1)[:, :n].contiguous()
        C1 = fp8g.gemm_block128(a, sa, *W, out="f32")
        want, mags = ref.product(ref.decode(a, sa, "row", E4M3), ref.decode(*W, "tile", E4M3), "nt")
        assert ((C1.double() - want).abs() <= ref.sum_tol(C) * mags).all()
    gu, sgu = fp8g.quantize_block128(torch.randn((R, 256), device="cuda", generator=r))[0]
    dh = torch.randn((R, 128), device="cuda", generator=r)
    row, col, h = fp8g.gated_block128_backward(dh, gu, sgu)
    wrow, wcol, wh = fp8g.gated_block128_backward(dh[-k:].contiguous(), gu[-k:].contiguous(), sgu[:, -k:].contiguous())
    same((row[0][-k:], row[1][:, -k:]), wrow)
    same((col[0][-k:], col[1][-4:], h[0][-k:], h[1][-4:]), wcol + wh)
    settled(fp8g)


@pytest.mark.parametrize("fmt", [E4M3, E5M2])
def test_tiles_not_finite_and_strided(fp8g, fmt):
    x = ref.values(300, 400, torch.Generator().manual_seed(3))
    x[0, 0], x[130, 5], x[140, 300] = math.nan, math.inf, -math.inf
    x[:128, 128:256] = 0
    x[256:, 256:384] *= 1e-42
    q, s = ref.quant(x, "tile", fmt)
    assert s[0, 1] == 1 and s[1, 0] == math.inf and s[2, 2] == 2.0 ** -126
    for t in (x.cuda(), x.t().contiguous().cuda().t(), torch.nn.functional.pad(x, (64, 48)).cuda()[:, 64:464],
              torch.nn.functional.pad(x, (1, 1)).cuda()[:, 1:401]):
        same([v.cpu() for v in fp8g.quantize_tile128(t, fmt=fmt)], (q, s))


def test_two_threads_at_once(fp8g):
    r = torch.Generator(device="cuda").manual_seed(4)
    rand = lambda *s: torch.randn(s, device="cuda", generator=r)
    work = []
    for M in (3, 260):
        x, dy, W13, W2 = rand(M, 512), rand(M, 512), rand(768, 512), rand(512, 384)

        def step(x=x, dy=dy, W13=W13, W2=W2):
            q13, q2 = fp8g.quantize_tile128(W13), fp8g.quantize_tile128(W2)
            row, _ = fp8g.quantize_block128(x)
            h, gu = fp8g.gated_block128(*row, *q13, keep=True)
            y = fp8g.gemm_block128(*h, *q2)
            drow, dcol = fp8g.quantize_block128(dy, row=True, col=True)
            dh = fp8g.gemm_block128(*drow, *q2, form="nn")
            a, b, c = fp8g.gated_block128_backward(dh, *gu)
            return [y, fp8g.gemm_block128(*dcol, *c, form="tn"), fp8g.gemm_block128(*b, *fp8g.requantize_block128(*row), form="tn"),
                    fp8g.gemm_block128(*a, *q13, form="nn")]
        work.append(step)
    want = [w() for w in work]
    torch.cuda.synchronize()
    bad = []

    def loop(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got = work[i]()
                s.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    bad.append(i)
    threads = [threading.Thread(target=loop, args=(i % 2,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad
    settled(fp8g)


def test_every_call_on_a_stream_of_its_own(fp8g):
    r = torch.Generator(device="cuda").manual_seed(5)
    x, W, dh = (torch.randn(s, device="cuda", generator=r) for s in ((140, 512), (512, 512), (140, 256)))

    def step(**at):
        row, col = fp8g.quantize_block128(x, row=True, col=True, **at)
        t = fp8g.quantize_tile128(W, **at)
        turned = fp8g.requantize_block128(*row, **at)
        h, gu = fp8g.gated_block128(*row, *t, keep=True, **at)
        a, b, c = fp8g.gated_block128_backward(dh, *gu, **at)
        return [*row, *col, *t, *turned, *h, *gu, *a, *b, *c, fp8g.gemm_block128(*row, *t, **at),
                fp8g.gemm_block128(*col, *b, form="tn", **at)]
    want = step()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for at in (s, s.cuda_stream):
        got = step(stream=at)
        s.synchronize()
        same(got, want)
    for call in (lambda: fp8g.quantize_block128(x.t(), stream=s), lambda: fp8g.quantize_tile128(W[:, 1:], stream=s),
                 lambda: fp8g.gated_block128_backward(dh.t().contiguous().t(), *want[10:12], stream=s)):
        with pytest.raises(AssertionError):  # (a copy would be another stream's)
            call()
    settled(fp8g)


FIRST = """
import sys
sys.path.insert(0, {root!r})
import torch
import fp8_block_scaled_06_gb300 as f
u = lambda *s: torch.randint(0, 0x70, s, dtype=torch.uint8, device="cuda")
one = lambda *s: torch.ones(s, device="cuda")
A, B = (u(12000, 272), one(94, 272)), (u(12000, 400), one(94, 400))
x, W, gu, dh = (u(3, 512), one(4, 3)), (u(512, 512), one(4, 4)), (u(3, 512), one(4, 3)), torch.randn((3, 256), device="cuda")
def step():
    return [f.gemm_block128(*A, *B, form="tn", out="f32"), f.gemm_block128(*x, *W), *f.gated_block128(*x, *W)[0],
            *f.gated_block128_backward(dh, *gu)[2]]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = step()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, step()))
assert f.fp8_gemm_status()[0] == 0
print("right")
"""


def test_a_first_call_under_capture(fp8g):
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "right", r.stderr[-2000:]
