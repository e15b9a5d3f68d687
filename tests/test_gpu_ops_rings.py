"""The RMS norm's gradient at every row length where the shape of its ring of rows
changes (its depth, the threads of a row, whether dres has room in it)."""

import pytest
import torch

import fsdp_layout_aware_gb300 as tide
import ops_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float32

LENGTHS = [1, 8, 160, 161, 168, 176, 204, 205, 224, 232, 512, 513, 544, 552, 648, 649, 720, 728, 1000, 1001, 2048, 2049, 2208,
           2216, 2640, 2641, 2928, 2936, 4072, 4073, 4416, 4424, 4784, 4785, 5120, 5121, 5128, 5292, 5293, 5880, 5888, 7596,
           7597, 8168, 8169, 8192, 8193, 8200, 8864, 8872, 9640, 9641, 10640, 10641, 11776, 11784, 13296, 13304, 15128, 15129,
           15192, 15193, 15360, 15361, 15368, 16383, 16384]


def randn(*shape, seed, dtype):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("odd", [False, True])
def test_lengths_on_both_sides_of_every_change(dtype, kept, odd):
    rows = 5
    for cols in LENGTHS:
        ld = cols + 3 if odd else -(-cols // 16) * 16  # rows on 16-byte boundaries, or not

        def put(x):
            v = torch.empty(rows * ld, dtype=x.dtype, device=DEV).as_strided((rows, cols), (ld, 1))
            v.copy_(x)
            return v

        h, dy, dres = (put(randn(rows, cols, seed=k, dtype=dtype)) for k in range(3))
        w = randn(cols, seed=3, dtype=dtype)
        rstd = 1 / torch.sqrt(h.float().square().mean(1) + 1e-5)
        hv, given = h.double(), h
        if kept:
            given = tide.Checkpoint8(put(torch.zeros(rows, cols, dtype=torch.uint8)),
                                     torch.zeros(rows, -(-cols // 32), dtype=torch.uint8, device=DEV))
            tide.tide_checkpoint_store(h, given)
            back = torch.empty(rows, cols, device=DEV)
            tide.tide_checkpoint_load(given, back)
            hv = back.double()
        n, g = hv * rstd.double()[:, None], dy.double() * w.double()
        mean = (g * n).mean(1, keepdim=True)
        base = rstd.double()[:, None] * (g - n * mean)
        size = rstd.double()[:, None] * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
        dw = (dy.double() * n).sum(0)
        # The bounds of the gradient's other tests: the output's rounding, and 96 units of the terms' magnitudes.
        for res in (None, dres):
            dx, got_dw = put(torch.zeros(rows, cols, dtype=dtype)), torch.empty(cols, dtype=dtype, device=DEV)
            tide.tide_rms_norm_backward(dy, given, w, rstd, dx, dweight=got_dw, dres=res)
            want = base if res is None else base + res.double()
            mag = size if res is None else size + res.double().abs()
            over = (dx.double() - want).abs() - R.rounding(dtype) * want.abs() - 96 * R.FP32 * mag
            assert over.max().item() <= 0, (cols, res is not None)
            over = (got_dw.double() - dw).abs() - R.rounding(dtype) * dw.abs() - 98 * R.FP32 * (dy.double() * n).abs().sum(0)
            assert over.max().item() <= 0, (cols, "dweight")
    tide.tide_ops_check()
