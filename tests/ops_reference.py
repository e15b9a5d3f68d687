"""The training-block operators in 64 bits on the CPU, written from their
formulas (include/tide_ops.h), and the tolerances the GPU tests use.

bf16 and e4m3 values, sums of them and their products are exact or nearly so in
fp64, so a reference value's own error is far below any tolerance here.
"""

import math

import numpy as np
import torch

BLOCK = 32
ACTS = ("none", "relu", "gelu", "gelu_erf", "silu")
A, B = math.sqrt(2.0 / math.pi), 0.044715


def e4m3_table():
    """Value of each of the 256 codes."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = math.nan if c & 127 == 127 else -v if c & 128 else v
    return out


TABLE = e4m3_table()
_POS = TABLE[:127]  # ascending; entry i is code i, so even entries have even mantissas


def nearest_codes(q):
    """Codes of scaled values |q| <= 448: nearest, ties to the even code; NaN for NaN."""
    a = np.abs(np.nan_to_num(q, nan=0.0))
    hi = np.clip(np.searchsorted(_POS, a, side="left"), 1, 126)
    lo = hi - 1
    dl, dh = a - _POS[lo], _POS[hi] - a
    c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    c = np.where(a == 0, 0, c) | np.where(np.signbit(q), 128, 0)
    return np.where(np.isnan(q), 127, c).astype(np.uint8)


def quantise(v):
    """(codes, scales) of fp64 values (rows, cols), block by block."""
    rows, cols = v.shape
    blocks = -(-cols // BLOCK)
    codes = np.zeros((rows, cols), np.uint8)
    scales = np.zeros((rows, blocks), np.uint8)
    for r in range(rows):
        for b in range(blocks):
            x = v[r, b * BLOCK:(b + 1) * BLOCK]
            fin = np.abs(x[np.isfinite(x)])
            a = fin.max() if fin.size else 0.0
            e = -127
            if a > 0:
                e = max(-127, math.frexp(a)[1] - 12)
                while a > 448.0 * 2.0 ** e:
                    e += 1
            q = np.where(np.isfinite(x), x, np.nan) / 2.0 ** e
            if e == 120:
                q = np.clip(q, -240.0, 240.0)
            codes[r, b * BLOCK:(b + 1) * BLOCK] = nearest_codes(q)
            scales[r, b] = e + 127
    return codes, scales


def values(codes, scales):
    col = np.arange(codes.shape[1]) // BLOCK
    return TABLE[codes] * 2.0 ** (scales[:, col].astype(np.float64) - 127)


def act(name, z):
    z = np.asarray(z, np.float64)
    with np.errstate(all="ignore"):
        if name == "none":
            return z
        if name == "relu":
            return np.where(z < 0, 0.0, z)
        if name == "silu":
            p = 1 / (1 + np.exp(-z))
        elif name == "gelu":
            p = 1 / (1 + np.exp(-2 * A * (z + B * z ** 3)))
        else:
            p = 0.5 * torch.erfc(torch.from_numpy(-z / math.sqrt(2))).numpy()
        return np.where(z == -np.inf, 0.0, z * p)


def act_grad(name, z):
    z = np.asarray(z, np.float64)
    with np.errstate(all="ignore"):
        if name == "none":
            return np.ones_like(z)
        if name == "relu":
            return np.where(np.isnan(z), z, (z > 0).astype(np.float64))
        c = np.clip(z, -40, 40)  # beyond, the derivative is 0 or 1 to fp64 precision (NaN stays)
        if name == "silu":
            p = 1 / (1 + np.exp(-c))
            return p + c * p * (1 - p)
        if name == "gelu":
            p = 1 / (1 + np.exp(-2 * A * (c + B * c ** 3)))
            return p + c * p * (1 - p) * 2 * A * (1 + 3 * B * c ** 2)
        p = 0.5 * torch.erfc(torch.from_numpy(-c / math.sqrt(2))).numpy()
        return p + c * np.exp(-c * c / 2) / math.sqrt(2 * math.pi)


def rms_norm(x, residual, w, eps):
    h = x if residual is None else x + residual
    rstd = 1 / np.sqrt((h * h).mean(1) + eps)
    return h, h * rstd[:, None] * w, rstd


def rms_norm_backward(dy, h, w, rstd, dres):
    n = h * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - n * (g * n).mean(1, keepdims=True))
    return dx if dres is None else dx + dres, (dy * n).sum(0)


# ---- tolerances

BF16 = 2.0 ** -8      # twice half a unit in the last place: the rounding, and fp32 error that may push it over
FP32 = 2.0 ** -23


def rounding(dtype):
    return BF16 if dtype is torch.bfloat16 else FP32


def product_bound(a, b):
    """Largest error of sum_k a[m,k] b[n,k] in fp32: products of bf16 are exact, a 16-term step loses at most 16 units of
    2^-23 of the magnitudes summed, and each of the K/16 additions to the accumulator one."""
    k = a.shape[1]
    return (k / 16 + 16) * FP32 * (np.abs(a) @ np.abs(b).T)


def check(got, want, tol, what):
    got = got.detach().double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaNs differ"
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), f"{what}: infinities differ"
    fine = np.isfinite(want)
    over = (np.abs(got - want) - tol)[fine] if got.size else np.zeros(0)
    assert not over.size or over.max() <= 0, f"{what}: {over.max()} over the tolerance"


def check_kept(codes, scales, want, err, what):
    """A checkpoint of values known to within `err` (elementwise): the scale is one that a value within err of the
    block's largest gives, and each kept value is as near as codes of that scale come."""
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    col = np.arange(want.shape[1]) // BLOCK
    for low, bound in ((True, np.less_equal), (False, np.greater_equal)):
        edge = np.maximum(np.abs(want) - err, 0) if low else np.abs(want) + err
        _, s = quantise(edge)
        assert bound(s, scales).all(), f"{what}: scales"
    s = 2.0 ** (scales[:, col].astype(np.float64) - 127)
    # Half the gap between codes: 2^-4 of a normal value, 2^-10 of the scale below.
    half = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * s)
    check(values(codes, scales), want, half + 1.07 * err, what)
