"""What the language model example's sharded steps hand on: the reduced shards, their norm, the clipped shards and the
update, against the ranks' gradients in fp64."""

import math

import pytest
import torch

import fsdp_layout_aware_gb300 as tide
import lm_reference as R
from test_gpu_lm_example import example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nodes,gpus,max_norm", [(1, 1, 0.25), (1, 4, 0.05), (2, 2, 1e6)])
def test_norm_clipping_and_update_of_sharded_steps(nodes, gpus, max_norm, monkeypatch):
    ex = example()
    ranks, lr, steps = nodes * gpus, 0.5, 3
    seen = []  # a step: dict of what each call took and gave
    params = []  # what ag_place was given, a step

    def reduce(plan, grads, shards, inner=tide.TidePlan.rs_reduce):
        inner(plan, grads, shards)
        seen.append({"plan": plan, "grads": [g.double() for g in grads], "reduced": [s.clone() for s in shards]})

    def norm_of(shards, norm, inner=tide.tide_grad_norm):
        inner(shards, norm)
        seen[-1]["norm"] = norm.item()

    def clip(shards, norm, most, inner=tide.tide_grad_clip):
        inner(shards, norm, most)
        seen[-1]["clipped"] = [s.clone() for s in shards.tensors]

    def place(plan, shards, outs, elem_bytes, inner=tide.TidePlan.ag_place):
        params.append(torch.stack(list(shards)).double())
        inner(plan, shards, outs, elem_bytes)

    monkeypatch.setattr(tide.TidePlan, "rs_reduce", reduce)
    monkeypatch.setattr(tide.TidePlan, "ag_place", place)
    monkeypatch.setattr(tide, "tide_grad_norm", norm_of)
    monkeypatch.setattr(tide, "tide_grad_clip", clip)
    # pack reads the plan's offsets: kept, since the plan is gone when the steps are through.
    packed = {}

    def pack(plan, tensors, inner=ex.pack):
        packed["e"], packed["o"], packed["S"], packed["N"] = list(plan.e), list(plan.o), plan.S, plan.N
        return inner(plan, tensors)

    monkeypatch.setattr(ex, "pack", pack)
    history = ex.train(tokens=64, vocab=101, width=72, inner=136, nodes=nodes, gpus=gpus, steps=steps, lr=lr, max_norm=max_norm,
                       say=lambda s: None)
    assert len(seen) == len(params) == len(history) == steps
    count = len(seen[0]["grads"]) // ranks
    for step, (got, (loss, norm)) in enumerate(zip(seen, history)):
        assert math.isfinite(loss) and loss > 0 and norm == got["norm"]
        want = torch.zeros(packed["N"], packed["S"], dtype=torch.float64, device="cuda")
        size = torch.zeros_like(want)  # of the magnitudes added
        for p in range(count):
            mine = [got["grads"][r * count + p] for r in range(ranks)]
            for to, v in ((want, sum(mine) / ranks), (size, sum(g.abs() for g in mine) / ranks)):
                flat = torch.zeros(packed["N"] * packed["e"][p], dtype=torch.float64, device="cuda")
                flat[:v.numel()] = v.reshape(-1)
                to[:, packed["o"][p]:packed["o"][p] + packed["e"][p]] = flat.view(packed["N"], packed["e"][p])
        # Averages of `ranks` numbers in fp32: as many roundings of the magnitudes added.
        off = (ranks + 1) * R.U * size
        reduced = torch.stack(got["reduced"]).double()
        assert ((reduced - want).abs() <= off).all()
        exact = want.square().sum().sqrt().item()
        assert exact > 0 and abs(norm - exact) <= off.square().sum().sqrt().item() + 12 * R.U * exact
        by = min(1.0, max_norm / (norm + 1e-6))
        assert (by < 1) == (max_norm < 1e6)  # two of the three do clip
        clipped = torch.stack(got["clipped"]).double()
        assert ((clipped - reduced * by).abs() <= 5 * R.U * reduced.abs() * by + 1e-44).all()
        if by < 1:
            assert abs(clipped.square().sum().sqrt().item() / max_norm - 1) <= 1e-4  # norm + 1e-6, and roundings
        if step + 1 < steps:
            # The master parameters are rounded to bf16 (2^-8 of each) before they are placed, here and a step later.
            moved = params[step + 1] - params[step]
            assert ((moved + lr * clipped).abs() <= 2.0 ** -8 * (params[step].abs() + params[step + 1].abs()) * 1.01 + 1e-7).all()
