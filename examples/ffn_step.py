"""A training step of a gated feed-forward layer in 8 bits, with fp32 scales for
blocks of 128.

    python examples/ffn_step.py [--tokens 4096] [--hidden 4096] [--ffn 14336]

Forward:  x in 8 bits along rows; gate, up and the activation in one kernel, whose
output h is in 8 bits and which keeps gate and up in 8 bits; the down projection.
Backward: dy in 8 bits along rows and along columns in one reading; dh from the down
weights as they lie; the gradient of gate and up from the 8-bit checkpoint, both ways,
and h again along columns; dx; both weight gradients, added to fp32 sums.  Weights are
random; prints the time of a step.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_06_gb300 as fp8g  # noqa: E402


class Layer:
    def __init__(self, hidden, ffn, gate=fp8g.FP8G_GATE_SILU, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.gate = gate
        self.w13 = torch.randn((2 * ffn, hidden), device="cuda", generator=gen) * hidden ** -0.5
        self.w2 = torch.randn((hidden, ffn), device="cuda", generator=gen) * ffn ** -0.5
        self.dw13, self.dw2 = torch.zeros_like(self.w13), torch.zeros_like(self.w2)
        self.quantise()

    def quantise(self):
        self.q13, self.s13 = fp8g.quantize_tile128(self.w13)
        self.q2, self.s2 = fp8g.quantize_tile128(self.w2)

    def forward(self, x):
        self.x, _ = fp8g.quantize_block128(x)
        h, self.gu = fp8g.gated_block128(*self.x, self.q13, self.s13, gate=self.gate, keep=True)
        return fp8g.gemm_block128(*h, self.q2, self.s2)

    def backward(self, dy):
        row, col = fp8g.quantize_block128(dy, row=True, col=True)
        dh = fp8g.gemm_block128(*row, self.q2, self.s2, form="nn")
        drow, dcol, h = fp8g.gated_block128_backward(dh, *self.gu, gate=self.gate)
        fp8g.gemm_block128(*col, *h, form="tn", add_to=self.dw2)
        fp8g.gemm_block128(*dcol, *fp8g.requantize_block128(*self.x), form="tn", add_to=self.dw13)
        return fp8g.gemm_block128(*drow, self.q13, self.s13, form="nn")

    def update(self, rate):
        for w, d in ((self.w13, self.dw13), (self.w2, self.dw2)):
            w.sub_(d, alpha=rate)
            d.zero_()
        self.quantise()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--ffn", type=int, default=14336)
    a = ap.parse_args()
    fp8g.build()
    layer = Layer(a.hidden, a.ffn)
    x = torch.randn((a.tokens, a.hidden), device="cuda").bfloat16()
    dy = torch.randn((a.tokens, a.hidden), device="cuda").bfloat16()
    times = []
    for _ in range(8):
        start, mid, end = (torch.cuda.Event(enable_timing=True) for _ in range(3))
        start.record()
        layer.forward(x)
        mid.record()
        layer.backward(dy)
        end.record()
        torch.cuda.synchronize()
        times.append((start.elapsed_time(mid), mid.elapsed_time(end)))
    f, b = (sorted(t)[len(t) // 2] for t in zip(*times))
    flops = 6 * a.tokens * a.hidden * a.ffn
    print(f"forward {f:.3f} ms ({flops / f / 1e9:.0f} TFLOPS), backward {b:.3f} ms ({2 * flops / b / 1e9:.0f} TFLOPS)")
    st, detail = fp8g.fp8_gemm_status()
    assert st == 0, (st, detail)


if __name__ == "__main__":
    main()
