"""Tiles whose K steps are split over several CTAs: the layer's down product
(whose parts the weighted sum reads), gate/up tiles of three and more parts,
adapters whose low-rank steps begin inside a slot.  Exact integers throughout;
a product is split when its tiles are fewer than half the SMs, into parts of
eight 128-wide steps at least."""
import pytest
import torch

import fp8_block_scaled_06_gb300 as fp8g
from test_gemm_lora_gpu import Projection
from test_moe_layer_gpu import Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k,H,F", [
    (1, 4, 2, 256, 4096),    # down: 2 tiles of 32 steps, four parts each
    (20, 4, 2, 256, 4096),   # and several tokens in a tile
    (3, 64, 8, 96, 2080),    # a row's part found among many groups
    (1, 2, 1, 5120, 96),     # gate/up: one tile of 40 steps, five parts
    (17, 3, 2, 4992, 160),   # 39 steps: parts of seven and eight; the last tile partly past F
    (5, 2, 2, 3104, 3104),   # both products, the last steps and tiles partly past the matrix
])
def test_layer(T, E, k, H, F):
    Layer(T, E, k, H, F).check_exact()


def test_layer_groups_of_one_expert():
    """More than 128 rows of an expert: two groups, each with a split down product."""
    l = Layer(70, 3, 2, 160, 2048)
    l.ids[:] = 1
    l.ids[60:, 1] = 2
    l.check_exact()


def test_layer_fp4():
    Layer(4, 4, 2, 256, 4096, fp8g.FP8G_E2M1).check_exact()


def test_layer_many_pairs():
    """More pairs than a table of the weighted sum holds."""
    Layer(40, 16, 8, 128, 2176, seed=1).check_exact()


@pytest.mark.parametrize("M,N,K,L,r", [
    (1, 128, 6144, 1, 8),      # one tile of 48 steps, six parts: joined in two rounds
    (33, 264, 5120, 16, 136),  # slots of three rank blocks, parts begin inside them
    (20, 136, 2080, 5, 40)])
def test_adapters(M, N, K, L, r):
    Projection(M, N, K, L, r).check_exact()


@pytest.mark.parametrize("first", [90, 33, 99])
def test_adapters_parts_begin_inside_a_slots_windows(first):
    """A slot of more than 64 columns takes two windows a rank block."""
    p = Projection(100, 136, 4096, 2, 72)
    p.adapter[:first] = 0
    p.adapter[first:] = 1
    p.check_exact()
    p.adapter = p.adapter[torch.randperm(100, generator=torch.Generator().manual_seed(first))]
    p.check_exact()
