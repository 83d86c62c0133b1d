"""A block of a served mixture-of-experts model: a projection whose rows carry
their requests' low-rank adapters, the router, the experts.

    python examples/moe_block.py [--tokens 8] [--hidden 1024] [--ffn 512] [--experts 16]

Few tokens (a decode step) take fp8_moe_layer, many (a prompt) the router's row
order and the grouped GEMMs.  Weights are random; prints the time of a step and
how far the two ways are apart on the same tokens.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_06_gb300 as fp8g  # noqa: E402


def quantised(w):
    """fp32 [matrices, rows, K] -> E4M3 codes, 1x32 scales of the same leading sizes."""
    n, rows, K = w.shape
    q, s = fp8g.quantize(w.view(-1, K), 32)
    return q.view(n, rows, K), s.view(n, rows, K // 32)


class Block:
    def __init__(self, hidden, ffn, experts, top_k, adapters, rank, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def rand(*shape):
            return torch.randn(shape, device="cuda", generator=gen) * shape[-1] ** -0.5
        self.H, self.F, self.E, self.k = hidden, ffn, experts, top_k
        W, sf = quantised(rand(1, hidden, hidden))
        self.W, self.sfw = W[0], fp8g.pack_scales(sf[0])
        self.lora_a, self.lora_b = rand(adapters, rank, hidden).bfloat16(), rand(adapters, hidden, rank).bfloat16()
        self.alpha = torch.full((adapters,), 2.0, device="cuda")
        self.router = rand(experts, hidden).bfloat16()
        self.W13, self.s13 = quantised(rand(experts, 2 * ffn, hidden))
        self.W2, self.s2 = quantised(rand(experts, hidden, ffn))
        # the scales as fp8_moe_layer takes them, once for the weights' life
        self.p13 = fp8g.pack_scales(self.s13.view(2 * experts, ffn, hidden // 32))
        self.p2 = fp8g.pack_scales(self.s2)

    def project(self, x, adapter):
        return x + fp8g.gemm_lora(x, self.W, self.sfw, self.lora_a, self.lora_b, self.alpha, adapter)

    def experts_of_few(self, x):
        ids, w = fp8g.moe_route(x @ self.router.T, self.k)
        return fp8g.moe_layer(x, ids, w, self.W13, self.p13, self.W2, self.p2)

    def experts_of_many(self, x):
        T, n = x.shape[0], x.shape[0] * self.k
        _, w, counts, rows, slots = fp8g.moe_route(x @ self.router.T, self.k, ordered=True)
        gu = torch.empty((n, 2 * self.F), device="cuda")
        fp8g.fp8_grouped_gemm_quant(x, fp8g.FP8G_IN_BF16, T, rows, self.W13, self.s13, gu, fp8g.FP8G_OUT_F32,
                                    fp8g.FP8G_E4M3, None, fp8g.FP8G_ACT_NONE, counts, self.E, 2 * self.F,
                                    self.H, n)
        h = torch.nn.functional.silu(gu[:, :self.F]) * gu[:, self.F:]
        y = torch.empty((T, self.k, self.H), device="cuda")
        each = torch.arange(n, dtype=torch.int32, device="cuda")
        fp8g.fp8_grouped_gemm_quant(h, fp8g.FP8G_IN_F32, n, each, self.W2, self.s2, y, fp8g.FP8G_OUT_F32,
                                    fp8g.FP8G_E4M3, None, fp8g.FP8G_ACT_NONE, counts, self.E, self.H,
                                    self.F, n, c_row_of=slots, c_rows=n)
        return (w[:, :, None] * y).sum(1).bfloat16()

    def __call__(self, x, adapter):
        x = self.project(x, adapter)
        # the layer is faster up to about 150 tokens at 64 experts of 2048 x 1024, k = 8, up to 400
        # at 32 of 4096 x 2048, k = 4, and up to its limit of 512 at 8 of 4096 x 14336, k = 2
        few = x.shape[0] <= 128
        return x + (self.experts_of_few(x) if few else self.experts_of_many(x))


def apart(block, tokens, adapters, seed=1):
    """Relative distance of the two ways through the experts for the same tokens."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((tokens, block.H), device="cuda", generator=gen).bfloat16()
    x = block.project(x, torch.randint(-1, adapters, (tokens,), device="cuda", generator=gen).int())
    a, b = block.experts_of_few(x).float(), block.experts_of_many(x).float()
    return float((a - b).norm() / b.norm())


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("tokens", 8), ("hidden", 1024), ("ffn", 512), ("experts", 16), ("top-k", 2),
                        ("adapters", 4), ("rank", 16)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    fp8g.build()
    block = Block(a.hidden, a.ffn, a.experts, a.top_k, a.adapters, a.rank)
    x = torch.randn((a.tokens, a.hidden), device="cuda").bfloat16()
    adapter = torch.arange(a.tokens, device="cuda").int() % (a.adapters + 1) - 1
    for _ in range(3):
        block(x, adapter)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(20):
        out = block(x, adapter)
    end.record()
    torch.cuda.synchronize()
    status, detail = fp8g.fp8_gemm_status()
    assert status == fp8g.FP8G_OK, (fp8g.fp8g_status_string(status), detail)
    print(f"{a.tokens} tokens: {begin.elapsed_time(end) / 20 * 1e3:.1f} us a step, "
          f"output {tuple(out.shape)}, the two ways {apart(block, min(a.tokens, 64), a.adapters):.1e} apart")


if __name__ == "__main__":
    main()
