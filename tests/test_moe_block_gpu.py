"""The operators together: examples/moe_block.py, both ways through the experts."""
import importlib.util
import os

import pytest
import torch

import fp8_block_scaled_06_gb300 as fp8g

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_block", os.path.join(ROOT, "examples", "moe_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens", [1, 13, 64])
def test_both_ways_agree(example, tokens):
    """h's codes differ where the two ways' fp32 sums round to different sides
    (one code, 2^-3, of few); the bf16 outputs by a rounding (2^-8)."""
    block = example.Block(512, 256, 8, 2, 3, 16)
    assert example.apart(block, tokens, 3) < 2.0 ** -8
    assert fp8g.fp8_gemm_status()[0] == 0


def test_steps(example):
    block = example.Block(256, 128, 4, 2, 2, 8)
    for tokens in (5, 200):
        x = torch.randn((tokens, 256), device="cuda").bfloat16()
        out = block(x, torch.full((tokens,), -1, dtype=torch.int32, device="cuda"))
        assert out.shape == x.shape and torch.isfinite(out.float()).all()
    assert fp8g.fp8_gemm_status()[0] == 0
