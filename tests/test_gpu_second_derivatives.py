"""The backward passes have no derivative of their own: asking for one is an error, not a constant."""
import pytest
import torch

import exact_sum_gemm_gb300 as dg

pytestmark = pytest.mark.gpu


def new(*shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(len(shape))
    return torch.randn(*shape, generator=g, device="cuda")


def operator(name):
    """(function of one tensor, that tensor's value)"""
    if name == "layer_norm":
        return lambda x: dg.det_layer_norm(x, new(32), new(32)), new(4, 32)
    if name == "attention":
        return lambda x: dg.det_attention(x, x, x, causal=True), new(1, 6, 2, 32)
    if name == "token_logprobs":
        tokens = torch.arange(5, device="cuda")
        return lambda x: sum(dg.det_token_logprobs(x, tokens)), new(5, 40)
    layer = dg.DetLinear(32, 16, device="cuda", weight=new(16, 32), k_shards=2 if name == "linear_sharded" else 1)
    return layer, new(6, 32)


@pytest.mark.parametrize("name", ["layer_norm", "attention", "token_logprobs", "linear", "linear_sharded"])
def test_second_derivative_is_refused(name):
    f, x = operator(name)
    x.requires_grad_(True)
    (first,) = torch.autograd.grad(f(x).square().sum(), x)
    (kept,) = torch.autograd.grad(f(x).square().sum(), x, create_graph=True)
    assert torch.equal(first, kept.detach())                # the first derivative as ever
    # the penalty has another path to x besides the gradient
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (kept.square().sum() + x.square().sum()).backward()
