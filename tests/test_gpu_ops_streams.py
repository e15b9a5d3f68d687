"""The training-block operators called on streams beside the current one, and
from several threads."""

import pytest
import torch

import fsdp_layout_aware_gb300 as tide

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def randn(*shape, seed, dtype=BF):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def empty(*shape, dtype=BF):
    return torch.empty(*shape, dtype=dtype, device=DEV)


def split_product(seed):
    """Partial sums in the workspace."""
    x, w, y = randn(64, 8192, seed=seed), randn(256, 8192, seed=seed + 1), empty(64, 256)
    return (y,), lambda stream: tide.tide_linear(x, w, y, stream=stream)


def odd_operands(seed):
    """Both operands laid out anew in the workspace."""
    dy, w, dx = randn(1021, 2047, seed=seed), randn(2047, 1023, seed=seed + 1), empty(1021, 1023)
    return (dx,), lambda stream: tide.tide_linear_grad_input(dy, w, dx, stream=stream)


def kept_operand(seed):
    """A checkpoint's values and the bias gradient's partial sums in the workspace."""
    dy, x = randn(2048, 768, seed=seed), randn(2048, 1024, seed=seed + 1)
    ck, dw, db = tide.Checkpoint8.empty(2048, 1024), empty(768, 1024), empty(768)
    tide.tide_checkpoint_store(x, ck)
    return (dw, db), lambda stream: tide.tide_linear_grad_weight(dy, ck, dw, db=db, act="silu", stream=stream)


def norm_gradient(seed):
    """The weight gradient's partial sums in the workspace."""
    dy, h, w = randn(4096, 2048, seed=seed), randn(4096, 2048, seed=seed + 1), randn(2048, seed=seed + 2)
    rstd, dx, dw = torch.ones(4096, device=DEV), empty(4096, 2048), empty(2048)
    return (dx, dw), lambda stream: tide.tide_rms_norm_backward(dy, h, w, rstd, dx, dweight=dw, stream=stream)


@pytest.mark.parametrize("make", [split_product, odd_operands, kept_operand, norm_gradient])
@pytest.mark.parametrize("as_handle", [False, True])
def test_a_call_on_another_stream_leaves_the_current_ones_memory_alone(make, as_handle):
    """A call on the current stream, waiting behind a long kernel, has let its workspace go when the same call with other
    inputs is made on a side stream, as has a tensor of the current stream: neither may be the second call's workspace."""
    side = torch.cuda.Stream()
    here, run_here = make(1)
    there, run_there = make(11)
    run_here(None)
    run_there(None)
    want = [t.clone() for t in here + there]
    for t in here + there:
        t.zero_()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms
    held = [torch.full((n << 20,), n, dtype=torch.uint8, device=DEV) for n in (1, 4, 8)]
    copies = [t.clone() for t in held]
    del held
    run_here(None)
    run_there(side.cuda_stream if as_handle else side)
    torch.cuda.synchronize()
    tide.tide_ops_check()
    assert all(torch.equal(t, w) for t, w in zip(here + there, want))
    assert all((t == n).all() for t, n in zip(copies, (1, 4, 8)))
