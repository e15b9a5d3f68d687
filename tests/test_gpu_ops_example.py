"""The feed-forward block example: its gradients against autograd in fp32, and
a sharded run that learns."""

import importlib.util
import os

import pytest
import torch

import fsdp_layout_aware_gb300 as tide

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("ffn_block", os.path.join(ROOT, "examples", "ffn_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("tokens,width,inner", [(96, 256, 640), (61, 203, 517)])
def test_block_against_autograd(tokens, width, inner):
    ex = example()
    bf = torch.bfloat16
    g = torch.Generator("cuda")
    g.manual_seed(3)

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda")

    params = [(1 + 0.1 * randn(width)).to(bf), (randn(inner, width) / width ** 0.5).to(bf), (0.1 * randn(inner)).to(bf),
              (randn(width, inner) / inner ** 0.5).to(bf), (0.1 * randn(width)).to(bf)]
    x, dy = randn(tokens, width).to(bf), randn(tokens, width).to(bf)
    grads = [torch.empty_like(p) for p in params]
    block = ex.Block(tokens, width, inner)
    y = block.forward(x, params)
    dx = block.backward(dy, params, grads)
    tide.tide_ops_check()

    ref = [p.double().requires_grad_() for p in params]
    xr = x.double().requires_grad_()
    n = xr * torch.rsqrt(xr.square().mean(1, keepdim=True) + ex.EPS) * ref[0]
    z = n @ ref[1].t() + ref[2]
    yr = xr + torch.nn.functional.gelu(z, approximate="tanh") @ ref[3].t() + ref[4]
    yr.backward(dy.double())
    # Relative, in the 2-norm: a bf16 value is off by up to 2^-9, a kept one by up to 2^-4 (2^-5 on average); the
    # gradients sum hundreds of such terms, whose errors do not add up but average.
    for got, want, tol in [(y, yr, 2 ** -7), (dx, xr.grad, 2 ** -5)] + [(a, b.grad, 2 ** -4) for a, b in zip(grads, ref)]:
        off = (got.double() - want).norm() / want.norm()
        assert off < tol, (tuple(got.shape), off.item())


def test_sharded_training_learns():
    losses = example().train(tokens=96, width=128, inner=256, nodes=2, gpus=2, steps=12, say=lambda s: None)
    assert losses[-1] < 0.8 * losses[0], losses
