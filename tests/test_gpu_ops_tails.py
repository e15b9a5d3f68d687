"""Activations and their derivatives over their whole range, the negative tails
included, through every call that applies one: relative to the value, so that a
tail that is lost shows."""

import math

import numpy as np
import pytest
import torch

import fsdp_layout_aware_gb300 as tide
import ops_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float32
A, B = R.A, R.B


def exact(name, z):
    """(f, f', error of f, error of f') of fp64 values z: the last two are what fp32 arithmetic may be off by.

    p, the factor of z in f, is off by E of itself: for the sigmoids |t| times the 6 units of 2^-23 by which their argument
    may be off (its factors, the change of base) and 16 for exponential, sum and quotient; for the normal distribution
    twice z^2 units, the same for its argument, and 16.  Near p = 1 the sigmoids' difference 1 - p is off by 2^-24.  Below
    2^-119 everything may come out as 0: 2^-126, where exponentials end, times |z| up to 88 where they do."""
    with np.errstate(over="ignore", under="ignore"):
        if name == "relu":
            return np.maximum(z, 0.0), (z > 0).astype(float), 0 * z, 0 * z
        if name == "gelu_erf":
            p = 0.5 * torch.erfc(torch.from_numpy(-z / math.sqrt(2))).numpy()
            slope = np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
            unit = 2 * z * z + 16
            one = 0.0
        else:
            t = z if name == "silu" else 2 * A * (z + B * z ** 3)
            dt = np.ones_like(z) if name == "silu" else 2 * A * (1 + 3 * B * z * z)
            p, q = 1 / (1 + np.exp(-t)), 1 / (1 + np.exp(t))
            slope = p * q * dt
            unit = 6 * np.abs(t) + 16
            one = np.abs(z) * dt * p
        e = unit * R.FP32
        zs = np.abs(z) * slope
        return z * p, p + z * slope, e * np.abs(z) * p + 2.0 ** -119, 2 * e * (p + zs) + one * R.FP32 + 2.0 ** -119


def sweep():
    """Values of every size and both signs, dense where the tails run out."""
    z = torch.cat([torch.linspace(-100, 12, 400), torch.linspace(-14, -2, 500), torch.linspace(-1.5, 1.5, 60),
                   -torch.logspace(-6, 2, 64), torch.logspace(-6, 2, 64)])
    return z.to(BF)


def check(got, name, z, grad, what):
    z = z.double().cpu().numpy()
    f, df, ef, edf = exact(name, z)
    want, err = (df, edf) if grad else (f, ef)
    R.check(got, want, R.rounding(got.dtype) * np.abs(want) + 1.01 * err, f"{name} {what}")


NAMES = R.ACTS[1:]


def test_the_errors_allowed_are_relative():
    """What the tolerances leave to a value in the tail is a small part of it."""
    for name, ends in (("gelu_erf", -11.0), ("gelu", -9.0), ("silu", -75.0)):
        z = np.linspace(ends, -3.0, 200)
        f, df, ef, edf = exact(name, z)
        assert (ef < 2.0 ** -9 * np.abs(f)).all() and (edf < 2.0 ** -8 * np.abs(df)).all(), name


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("cols,lead", [(256, 0), (253, 1)])
@pytest.mark.parametrize("grad", [False, True])
def test_checkpoint_load(name, dtype, cols, lead, grad):
    """Every code at scales from 2^-17 to 1/4: magnitudes from 2^-26 to 112."""
    codes = torch.arange(256, dtype=torch.uint8).roll(-3).repeat(16, 1)[:, :cols]
    scales = (torch.arange(16, dtype=torch.uint8) + 110)[:, None].repeat(1, 8)
    fine = (codes & 127) != 127
    codes = torch.where(fine, codes, torch.zeros_like(codes))
    buf = torch.empty(16 * cols + lead, dtype=torch.uint8, device=DEV)
    c = buf[lead:].view(16, cols)
    c.copy_(codes)
    out = torch.empty(16 * cols + lead, dtype=dtype, device=DEV)[lead:].view(16, cols)
    ones = torch.ones_like(out) if grad else None
    tide.tide_checkpoint_load(tide.Checkpoint8(c, scales.to(DEV)), out, act=name, grad=ones)
    v = torch.from_numpy(R.values(codes.numpy(), scales.numpy()))
    check(out, name, v, grad, "of a checkpoint")


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("rows,inner", [(1, 1), (700, 8), (64, 8192)])
def test_linear(name, rows, inner):
    """z is the weight's first column in every row: one token, many, and a sum in splits."""
    z = sweep()
    x, w = torch.zeros(rows, inner, dtype=BF, device=DEV), torch.zeros(len(z), inner, dtype=BF, device=DEV)
    x[:, 0], w[:, 0] = 1, z.to(DEV)
    y = torch.empty(rows, len(z), dtype=BF, device=DEV)
    tide.tide_linear(x, w, y, act=name)
    check(y, name, z.expand(rows, len(z)), False, "of a product")


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("rows,outer", [(1, 1), (700, 8), (64, 8192)])
@pytest.mark.parametrize("kept", [False, True])
def test_linear_grad_input(name, rows, outer, kept):
    """dy W is 1 everywhere: dx is f'(z)."""
    z = sweep().expand(rows, -1).contiguous()
    cols = z.shape[1]
    dy, w = torch.zeros(rows, outer, dtype=BF, device=DEV), torch.zeros(outer, cols, dtype=BF, device=DEV)
    dy[:, 0], w[0] = 1, 1
    zin = z.to(DEV)
    if kept:
        ck = tide.Checkpoint8.empty(rows, cols)
        tide.tide_checkpoint_store(zin, ck)
        v = torch.empty(rows, cols, device=DEV)
        tide.tide_checkpoint_load(ck, v)
        zin, z = ck, v
    dx = torch.empty(rows, cols, dtype=BF, device=DEV)
    tide.tide_linear_grad_input(dy, w, dx, act=name, z=zin)
    check(dx, name, z, True, "behind a product")
