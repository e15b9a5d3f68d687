"""8-bit checkpoints of more elements than 31 bits count."""

import pytest
import torch

import fsdp_layout_aware_gb300 as tide

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def randn(*shape, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(BF)


# More than 2^31 elements in rows of any alignment and in aligned ones, and more rows than one launch takes.
@pytest.mark.parametrize("rows,cols", [(70001, 32771), (70001, 32776), ((1 << 31) + 1001, 1)])
@pytest.mark.parametrize("act,with_grad", [("none", False), ("silu", False), ("gelu_erf", True)])
def test_rows_at_both_ends_come_out_as_when_called_alone(rows, cols, act, with_grad):
    n = 2 if cols > 1 else 70000  # for one column: on both sides of the place where the second launch begins
    ends = [slice(0, n), slice(rows - n, rows)]
    x = torch.zeros(rows, cols, dtype=BF, device=DEV)
    for seed, at in enumerate(ends):
        x[at] = randn(n, cols, seed=seed)
    ck = tide.Checkpoint8.empty(rows, cols)
    tide.tide_checkpoint_store(x, ck)
    assert not ck.codes[n:-n].any() and not ck.scales[n:-n].any()
    wants = []
    for at in ends:
        alone = tide.Checkpoint8.empty(n, cols)
        tide.tide_checkpoint_store(x[at].clone(), alone)
        assert torch.equal(ck.codes[at], alone.codes) and torch.equal(ck.scales[at], alone.scales)
        want = torch.empty(n, cols, dtype=BF, device=DEV)
        tide.tide_checkpoint_load(alone, want, act=act, grad=x[at].clone() if with_grad else None)
        assert want.any()
        wants.append(want)
    tide.tide_checkpoint_load(ck, x, act=act, grad=x if with_grad else None)
    for at, want in zip(ends, wants):
        assert torch.equal(x[at], want)
    assert not x[n:-n].any()
