"""What the conveniences of the router, the MoE layer and the projection with
adapters refuse before anything is launched: tensors on the host, scales that
are not packed, weights that are not codes."""
import pytest
import torch

import fp8_block_scaled_06_gb300 as fp8g

pytestmark = pytest.mark.gpu


def scales(*shape):
    return torch.ones(shape, device="cuda")


def layer_args():
    # sizes at which fp32 scales have as many elements as packed ones have bytes
    T, E, k, H, F = 3, 2, 2, 128, 128
    return dict(x=torch.zeros((T, H), device="cuda"), ids=torch.zeros((T, k), dtype=torch.int32, device="cuda"),
                weights=torch.zeros((T, k), device="cuda"),
                W13=torch.zeros((E, 2 * F, H), dtype=torch.uint8, device="cuda"),
                sf13=fp8g.pack_scales(scales(2 * E, F, H // 32)),
                W2=torch.zeros((E, H, F), dtype=torch.uint8, device="cuda"),
                sf2=fp8g.pack_scales(scales(E, H, F // 32)))


def projection_args():
    M, N, K, L, r = 3, 128, 128, 2, 8
    return dict(x=torch.zeros((M, K), device="cuda"), W=torch.zeros((N, K), dtype=torch.uint8, device="cuda"),
                sfw=fp8g.pack_scales(scales(N, K // 32)),
                lora_a=torch.zeros((L, r, K), dtype=torch.bfloat16, device="cuda"),
                lora_b=torch.zeros((L, N, r), dtype=torch.bfloat16, device="cuda"),
                alpha=torch.ones(L, device="cuda"), adapter=torch.zeros(M, dtype=torch.int32, device="cuda"),
                bias=torch.zeros(N, device="cuda"))


CALLS = {"moe_layer": layer_args, "gemm_lora": projection_args}


@pytest.mark.parametrize("name,arg", [(n, a) for n, names in (
    ("moe_layer", "x ids weights W13 sf13 W2 sf2"), ("gemm_lora", "x W sfw lora_a lora_b alpha adapter bias"))
    for a in names.split()])
def test_host_tensors(name, arg):
    args = CALLS[name]()
    assert (getattr(fp8g, name)(**args) == 0).all()
    args[arg] = args[arg].cpu()
    with pytest.raises(AssertionError):
        getattr(fp8g, name)(**args)


@pytest.mark.parametrize("name,arg,shape", [("moe_layer", "sf13", (4, 128, 4)), ("moe_layer", "sf2", (2, 128, 4)),
                                            ("gemm_lora", "sfw", (128, 4))])
def test_scales_that_are_not_packed(name, arg, shape):
    args = CALLS[name]()
    assert args[arg].numel() == scales(*shape).numel()
    args[arg] = scales(*shape)
    with pytest.raises(AssertionError, match="pack_scales"):
        getattr(fp8g, name)(**args)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.int32])
@pytest.mark.parametrize("name,arg", [("moe_layer", "W13"), ("moe_layer", "W2"), ("gemm_lora", "W")])
def test_weights_that_are_not_codes(name, arg, dtype):
    args = CALLS[name]()
    args[arg] = args[arg].to(dtype)
    with pytest.raises(AssertionError):
        getattr(fp8g, name)(**args)


@pytest.mark.parametrize("name,arg", [("moe_layer", "W13"), ("moe_layer", "W2"), ("gemm_lora", "W")])
def test_codes_of_other_one_byte_types(name, arg):
    args = CALLS[name]()
    args[arg] = args[arg].view(torch.float8_e4m3fn)
    assert (getattr(fp8g, name)(**args) == 0).all()


@pytest.mark.parametrize("name,arg", [("moe_layer", "ids"), ("moe_layer", "weights"), ("gemm_lora", "adapter"),
                                      ("gemm_lora", "lora_a"), ("gemm_lora", "alpha")])
def test_other_element_types(name, arg):
    args = CALLS[name]()
    args[arg] = args[arg].double()
    with pytest.raises(AssertionError):
        getattr(fp8g, name)(**args)


def test_router_host_logits():
    with pytest.raises(AssertionError):
        fp8g.moe_route(torch.zeros((4, 8)), 2)


def test_tensors_that_are_not_packed():
    """Copied on the current stream; refused by a call on a stream of its own,
    which would neither wait for the copy nor keep its memory."""
    sf = 2.0 ** torch.arange(160 * 8, device="cuda").remainder(9).float().view(160, 8)
    want = fp8g.pack_scales(sf)
    turned = sf.t().contiguous().t()
    assert not turned.is_contiguous() and torch.equal(fp8g.pack_scales(turned), want)
    x = torch.zeros((128, 3), device="cuda").t()
    calls = [lambda s: fp8g.pack_scales(turned, stream=s), lambda s: fp8g.moe_route(x[:, ::2], 2, stream=s),
             lambda s: fp8g.moe_layer(**{**layer_args(), "x": x}, stream=s),
             lambda s: fp8g.gemm_lora(**{**projection_args(), "x": x}, stream=s)]
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call in calls:
        call(None)
        with pytest.raises(AssertionError, match="packed"):
            call(other)
    got = fp8g.pack_scales(sf, stream=other)
    other.synchronize()
    assert torch.equal(got, want)
