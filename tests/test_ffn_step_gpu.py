"""The 8-bit feed-forward operators together: examples/ffn_step.py, its gradients
against the layer in 64 bits, eager and captured."""
import importlib.util
import os

import pytest
import torch

import block128_ref as ref
import fp8_block_scaled_06_gb300 as fp8g

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("ffn_step", os.path.join(ROOT, "examples", "ffn_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def wanted(layer, x, dy):
    """The layer without quantisation, in 64 bits: y and its gradients by differentiation."""
    v = [t.detach().double().requires_grad_() for t in (x, layer.w13, layer.w2)]
    gu = v[0] @ v[1].t()
    F = gu.shape[1] // 2
    h = ref.act(gu[:, :F], layer.gate)[0] * gu[:, F:]
    y = h @ v[2].t()
    return [y.detach()] + list(torch.autograd.grad(y, v, dy.double()))


def near(got, want, roundings):
    """To first order the relative errors of a path's roundings add up, half a step of E4M3 each."""
    off = ((got.double() - want).norm() / want.norm()).item()
    assert off <= roundings * ref.HALF[0], off


@pytest.mark.parametrize("tokens", [1, 33, 300, 1100])
@pytest.mark.parametrize("gate", [0, 1, 2])
def test_gradients(example, tokens, gate):
    layer = example.Layer(384, 256, gate, seed=tokens)
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    x = torch.randn((tokens, 384), device="cuda", generator=gen).bfloat16()
    dy = torch.randn((tokens, 384), device="cuda", generator=gen).bfloat16()
    y, dx = layer.forward(x), layer.backward(dy)
    assert fp8g.fp8_gemm_status()[0] == 0
    wy, wdx, wd13, wd2 = wanted(layer, x, dy)
    near(y, wy, 6)               # x, W13 (both in g and in u), h, W2
    near(dx, wdx, 9)             # dy, W2, g, u from x and W13, the checkpoint, dgu, W13
    near(layer.dw2, wd2, 7)      # dy, h from x, W13 and the checkpoint
    near(layer.dw13, wd13, 9)    # as dx, and x twice in the place of W13
    # a second backward pass adds the same again
    once = layer.dw2.clone()
    layer.forward(x)
    layer.backward(dy)
    assert torch.equal(layer.dw2, 2 * once)


def test_step_captured_and_on_another_stream(example):
    layer = example.Layer(256, 384, seed=3)
    x, dy = (torch.randn((200, 256), device="cuda").bfloat16() for _ in range(2))
    y, dx = layer.forward(x), layer.backward(dy)
    dw = layer.dw13.clone(), layer.dw2.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        for _ in range(2):
            layer.forward(x), layer.backward(dy)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            got = layer.forward(x), layer.backward(dy)
    layer.dw13.zero_(), layer.dw2.zero_()
    other = torch.randn_like(x)
    kept = x.clone()
    for inputs in (other, kept):
        x.copy_(inputs)
        layer.dw13.zero_(), layer.dw2.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], y) and torch.equal(got[1], dx)
    assert torch.equal(layer.dw13, dw[0]) and torch.equal(layer.dw2, dw[1])
    assert fp8g.fp8_gemm_status()[0] == 0


def test_update(example):
    layer = example.Layer(256, 128, seed=4)
    x = torch.randn((64, 256), device="cuda").bfloat16()
    before = layer.q13.clone()
    layer.forward(x), layer.backward(x)
    layer.update(1.0)
    assert not torch.equal(layer.q13, before) and (layer.dw13 == 0).all()
    assert torch.isfinite(layer.forward(x).float()).all()
