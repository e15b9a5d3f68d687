"""The operators at both ends of a training step run together, as the language
model example runs them: gradients against autograd in fp64, and the sharded steps."""

import importlib.util
import math
import os

import pytest
import torch

import fsdp_layout_aware_gb300 as tide

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("language_model", os.path.join(ROOT, "examples", "language_model.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("tokens,vocab,width,inner", [(96, 200, 256, 640), (61, 333, 203, 517)])
def test_model_against_autograd(tokens, vocab, width, inner):
    ex = example()
    bf = torch.bfloat16
    g = torch.Generator("cuda")
    g.manual_seed(3)

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda")

    params = [(randn(*s) / s[-1] ** 0.5).to(bf) if len(s) == 2 else (0.1 * randn(*s)).to(bf)
              for s in ex.shapes_of(vocab, width, inner)]
    params[1], params[6] = (1 + params[1].float()).to(bf), (1 + params[6].float()).to(bf)
    ids = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    targets = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    ids[-7:] = targets[-7:] = ex.PADDING
    ids[:20] = 5
    grads = [torch.full_like(p, math.nan) for p in params]
    model = ex.Model(tokens, vocab, width, inner)
    loss = model.loss(ids, targets, params)
    model.backward(ids, targets, params, grads)
    tide.tide_ops_check()

    ref = [p.double().cpu().requires_grad_() for p in params]
    ids, targets = ids.cpu(), targets.cpu()
    here = ids >= 0
    x = torch.where(here[:, None], ref[0][ids.clamp(min=0)] * width ** 0.5, 0.0)

    def rms(x, w):
        return x * torch.rsqrt(x.square().mean(1, keepdim=True) + ex.EPS) * w

    z = rms(x, ref[1]) @ ref[2].t() + ref[3]
    y = x + torch.nn.functional.gelu(z, approximate="tanh") @ ref[4].t() + ref[5]
    logs = torch.log_softmax(rms(y, ref[6]) @ ref[7].t(), 1)
    want = -logs[here].gather(1, targets[here][:, None]).mean()
    want.backward()
    # The logits, of a few units, are bf16 (2^-8 of each, averaged over the tokens) and so are the activations before them.
    assert abs(loss.item() - want.item()) < 2 ** -6
    # Relative, in the 2-norm, as for the block alone: bf16 values are off by up to 2^-8 each, those kept in 8 bits by up
    # to 2^-4 (2^-5 on average).
    for got, p in zip(grads, ref):
        off = (got.double().cpu() - p.grad).norm() / p.grad.norm()
        assert off < 2 ** -4, (tuple(got.shape), off.item())
    absent = torch.ones(vocab, dtype=torch.bool)
    absent[ids[here]] = False
    assert (grads[0].cpu()[absent] == 0).all()


@pytest.mark.parametrize("nodes,gpus", [(1, 1), (2, 2)])
def test_sharded_steps_run(nodes, gpus):
    """Every step's loss is finite, and the norm is that of the averaged gradients of the ranks' batches."""
    history = example().train(tokens=64, vocab=101, width=72, inner=136, nodes=nodes, gpus=gpus, steps=3, say=lambda s: None)
    assert len(history) == 3 and all(math.isfinite(v) and v > 0 for step in history for v in step)
