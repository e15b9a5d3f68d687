"""The training-block operators on the GPU against the 64-bit reference."""

import numpy as np
import pytest
import torch

import fsdp_layout_aware_gb300 as tide
import ops_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float32


def rand(shape, dtype, seed, scale=1.0, loud=True):
    """Seeded values with a few loud columns and a wide spread of magnitudes."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g, dtype=torch.float64)
    if loud and len(shape) == 2 and shape[1] > 3:
        x[:, shape[1] // 3] *= 30
    return (x * scale).to(dtype)


def put(x, lead=0, extra=0):
    """x on the GPU inside a larger buffer: `lead` elements before it, rows `extra` longer; the rest is NaN (or 0xAA)."""
    rows, cols = x.shape
    n = lead + rows * (cols + extra)
    if x.dtype == torch.uint8:
        buf = torch.full((n,), 0xAA, dtype=x.dtype, device=DEV)
    else:
        buf = torch.full((n,), float("nan"), dtype=x.dtype, device=DEV)
    v = buf[lead:].view(rows, cols + extra)[:, :cols]
    v.copy_(x)
    return v, buf


def blank(rows, cols, dtype, lead=0, extra=0):
    x = torch.zeros(rows, cols, dtype=dtype)
    return put(x, lead, extra)


def untouched(view, buf):
    """Nothing outside the view was written."""
    mask = torch.ones(buf.shape, dtype=torch.bool, device=DEV)
    lead = view.storage_offset()
    rows, cols = view.shape
    if rows:
        ld = view.stride(0) if rows > 1 else cols
        for r in range(rows):
            mask[lead + r * ld:lead + r * ld + cols] = False
    rest = buf[mask]
    return bool((rest == 0xAA).all() if buf.dtype == torch.uint8 else rest.isnan().all())


def f64(t):
    return t.double().cpu().numpy()


def checkpoint(rows, cols, lead=0, extra=0):
    c, cb = blank(rows, cols, torch.uint8, lead, extra)
    s, sb = blank(rows, -(-cols // 32), torch.uint8, lead, extra)
    return tide.Checkpoint8(c, s), cb, sb


LAYOUTS = [(0, 0), (8, 16), (1, 0), (3, 5)]  # (lead, extra): aligned, aligned with a stride, two odd ones
SHAPES = [(1, 1), (1, 31), (2, 32), (3, 33), (5, 64), (7, 100), (4, 1000), (13, 4095), (33, 256)]


# ---------------------------------------------------------------- checkpoints

@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("lead,extra", LAYOUTS)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_store_is_the_formats_nearest(rows, cols, lead, extra, dtype):
    x = rand((rows, cols), dtype, rows * 1000 + cols)
    dx, _ = put(x, lead, extra)
    ck, cb, sb = checkpoint(rows, cols, lead, extra)
    tide.tide_checkpoint_store(dx, ck)
    codes, scales = R.quantise(x.double().numpy())
    assert np.array_equal(ck.codes.cpu().numpy(), codes)
    assert np.array_equal(ck.scales.cpu().numpy(), scales)
    assert untouched(ck.codes, cb) and untouched(ck.scales, sb)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("cols", [64, 61])
def test_store_edge_values(cols, dtype):
    """Blocks of zeros, lowest and highest values, subnormals, infinities and NaN among finite values, and largest
    magnitudes on both sides of every scale's limit."""
    big = torch.finfo(dtype).max
    rows = [torch.zeros(cols), torch.full((cols,), -0.0), torch.full((cols,), big), torch.full((cols,), -big),
            torch.full((cols,), float("nan")), torch.full((cols,), float("inf")), torch.full((cols,), 1e-40),
            torch.full((cols,), 2.0 ** -133)]
    for at, v in ((0, float("inf")), (5, float("-inf")), (31, float("nan")), (40, -big)):
        r = torch.linspace(-3, 3, cols)
        r[at] = v
        rows.append(r)
    for e in (-126, -100, -1, 0, 1, 100, 119, 127):
        for m in (1.0, 1.75, 1.7578125, 1.9921875):
            r = torch.linspace(-1, 1, cols).double() * 2.0 ** e
            r[7] = m * 2.0 ** e
            rows.append(r.float())
    x = torch.stack([r.float() for r in rows]).to(dtype)
    ck, _, _ = checkpoint(*x.shape)
    tide.tide_checkpoint_store(x.to(DEV), ck)
    codes, scales = R.quantise(x.double().numpy())
    got = ck.codes.cpu().numpy()
    nan = codes & 127 == 127
    assert np.array_equal(got & 127 == 127, nan)
    assert np.array_equal(got[~nan], codes[~nan])
    assert np.array_equal(ck.scales.cpu().numpy(), scales)
    back = torch.empty(x.shape, dtype=FP, device=DEV)
    tide.tide_checkpoint_load(ck, back)
    assert np.array_equal(f64(back), R.values(codes, scales), equal_nan=True)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("cols", [256, 255])
def test_load_gives_every_code_and_scale(cols, dtype):
    codes = torch.arange(256, dtype=torch.uint8).repeat(248, 1)[:, :cols].contiguous()
    scales = torch.arange(248, dtype=torch.uint8)[:, None].repeat(1, 8)
    ck = tide.Checkpoint8(codes.to(DEV), scales.to(DEV))
    out = torch.empty(248, cols, dtype=dtype, device=DEV)
    tide.tide_checkpoint_load(ck, out)
    with np.errstate(over="ignore"):
        want = torch.from_numpy(R.values(codes.numpy(), scales.numpy())).float().to(dtype)
    assert torch.equal(out.cpu().nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("name", R.ACTS)
@pytest.mark.parametrize("lead,extra", [(0, 0), (1, 3)])
@pytest.mark.parametrize("with_grad", [False, True])
def test_load_with_activation(dtype, name, lead, extra, with_grad):
    rows, cols = 9, 200
    x = rand((rows, cols), BF, 5, scale=3.0)
    x[0, :8] = torch.tensor([0.0, -0.0, 80.0, -80.0, 300.0, -300.0, 1e-3, -1e-3])
    codes, scales = R.quantise(x.double().numpy())
    c, _ = put(torch.from_numpy(codes), lead, extra)
    s, _ = put(torch.from_numpy(scales), lead, extra)
    v = R.values(codes, scales)
    g = rand((rows, cols), dtype, 6)
    out, buf = blank(rows, cols, dtype, lead, extra)
    dg, _ = put(g, lead, extra)
    tide.tide_checkpoint_load(tide.Checkpoint8(c, s), out, act=name, grad=dg if with_grad else None)
    want = g.double().numpy() * R.act_grad(name, v) if with_grad else R.act(name, v)
    # fp32 error of f (or f') beside the output's rounding: the exponent's argument t is off by 2^-23 |t| (3 roundings),
    # so p by 4 * 2^-23 |t| p(1-p) <= 2^-23 * 2, and z p' by as much times |z| where p' is not 0 (|z| < 20).
    mag = np.abs(g.double().numpy()) if with_grad else np.abs(v)
    tol = R.rounding(dtype) * np.abs(want) + 64 * R.FP32 * np.minimum(mag * 20, mag + 20)
    R.check(out, want, tol, name)
    assert untouched(out, buf)
    if with_grad:  # in place
        tide.tide_checkpoint_load(tide.Checkpoint8(c, s), dg, act=name, grad=dg)
        assert torch.equal(dg, out)


@pytest.mark.parametrize("name", R.ACTS[1:])
def test_activations_at_their_ends(name):
    """Largest finite kept values and NaN, through f and f'."""
    codes = torch.tensor([[0x7E, 0xFE, 0x7F, 0x77, 0xF7, 0x00, 0x80, 0x38]], dtype=torch.uint8)
    for byte in (0, 127, 246):
        ck = tide.Checkpoint8(codes.to(DEV), torch.tensor([[byte]], dtype=torch.uint8, device=DEV))
        v = R.values(codes.numpy(), np.array([[byte]], np.uint8))
        for grad in (None, torch.ones(1, 8, device=DEV)):
            out = torch.empty(1, 8, device=DEV)
            tide.tide_checkpoint_load(ck, out, act=name, grad=grad)
            want = R.act(name, v) if grad is None else R.act_grad(name, v)
            R.check(out, want, 64 * R.FP32 * (np.abs(np.nan_to_num(want)) + 1e-3), name)


# ---------------------------------------------------------------- norm

NORM_SHAPES = [(1, 1), (1, 8), (3, 33), (5, 256), (9, 257), (4, 1024), (3, 1025), (6, 2048), (2, 4096), (5, 4095),
               (3, 8192), (2, 8193), (2, 16384), (1, 16383), (301, 72), (40, 640)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("lead,extra", [(0, 0), (16, 16), (1, 3)])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_norm(rows, cols, lead, extra, dtype):
    eps = 1e-5
    x, r = rand((rows, cols), dtype, 1), rand((rows, cols), dtype, 2)
    w = 1 + 0.2 * rand((cols,), dtype, 3)
    if rows > 2:
        x[1], r[1] = 0, 0  # rstd = eps^-1/2
    dx, dr = put(x, lead, extra)[0], put(r, lead, extra)[0]
    h, hb = blank(rows, cols, dtype, lead, extra)
    y, yb = blank(rows, cols, dtype, lead, extra)
    rstd = torch.empty(rows, device=DEV)
    y8, cb, sb = checkpoint(rows, cols, lead if lead % 8 else 16, extra if extra % 8 else 16)
    tide.tide_rms_norm(dx, w.to(DEV), eps, y=y, residual=dr, h=h, rstd=rstd, y8=y8)
    wh, wy, wr = R.rms_norm(x.double().numpy(), r.double().numpy(), w.double().numpy(), eps)
    # rstd: a sum of squares of positive terms, at most 64 roundings deep, then a division and a root: 2^-23 * 40.
    rerr = 40 * R.FP32
    R.check(rstd, wr, rerr * wr, "rstd")
    R.check(h, wh, R.rounding(dtype) * np.abs(wh), "h")
    R.check(y, wy, (R.rounding(dtype) + rerr + 4 * R.FP32) * np.abs(wy) * 1.01, "y")
    R.check_kept(y8.codes, y8.scales, wy, (rerr + 4 * R.FP32) * np.abs(wy), "y8")
    for v, b in ((h, hb), (y, yb), (y8.codes, cb), (y8.scales, sb)):
        assert untouched(v, b)
    # without the residual and the optional outputs, and in place
    x2 = dx.clone()
    tide.tide_rms_norm(x2, w.to(DEV), eps, y=x2)
    _, wy, _ = R.rms_norm(x.double().numpy(), None, w.double().numpy(), eps)
    R.check(x2, wy, (R.rounding(dtype) + rerr + 4 * R.FP32) * np.abs(wy) * 1.01, "y alone")
    r2 = dr.clone()
    tide.tide_rms_norm(dx, w.to(DEV), eps, y=y, residual=r2, h=r2)
    assert torch.equal(r2, h)


@pytest.mark.parametrize("cols", [512, 509])
def test_norm_keeps_bad_rows_to_themselves(cols):
    x = rand((6, cols), FP, 4, loud=False)
    x[1, 7], x[2, 9], x[4] = float("nan"), float("inf"), 0
    w = torch.ones(cols)
    y, rstd = torch.empty(6, cols, device=DEV), torch.empty(6, device=DEV)
    y8, _, _ = checkpoint(6, cols)
    tide.tide_rms_norm(x.to(DEV), w.to(DEV), 0.0, y=y, rstd=rstd, y8=y8)
    good = [0, 3, 5]
    wh, wy, _ = R.rms_norm(x[good].double().numpy(), None, w.double().numpy(), 0.0)
    R.check(y[good], wy, 64 * R.FP32 * np.abs(wy), "good rows")
    assert y[1].isnan().all() and rstd[1].isnan()
    assert y[2, 9].isnan() and (y[2, :9] == 0).all() and rstd[2] == 0  # 1 / sqrt(inf)
    assert y[4].isnan().all() and torch.isinf(rstd[4])  # 0 * inf: no eps, nothing to normalise
    got = y8.codes.cpu().numpy()
    assert (got[1] & 127 == 127).all() and got[2, 9] & 127 == 127 and (got[2, :9] & 127 == 0).all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("lead,extra", [(0, 0), (1, 3)])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES + [(2000, 96), (700, 1536), (400, 8200), (310, 10239), (309, 14336),
                                                         (305, 15361), (400, 16384)])
def test_norm_backward(rows, cols, lead, extra, kept, dtype):
    h, dy, dres = rand((rows, cols), dtype, 1), rand((rows, cols), dtype, 2), rand((rows, cols), dtype, 3)
    w = 1 + 0.2 * rand((cols,), dtype, 4)
    rstd = (1 / np.sqrt((h.double().numpy() ** 2).mean(1) + 1e-5)).astype(np.float32)
    if kept:
        codes, scales = R.quantise(h.double().numpy())
        hv = R.values(codes, scales)
        dh = tide.Checkpoint8(put(torch.from_numpy(codes), lead, extra)[0], put(torch.from_numpy(scales), lead, extra)[0])
    else:
        hv, dh = h.double().numpy(), put(h, lead, extra)[0]
    ddy, ddres = put(dy, lead, extra)[0], put(dres, lead, extra)[0]
    dx, xb = blank(rows, cols, dtype, lead, extra)
    dw = torch.empty(cols, dtype=dtype, device=DEV)
    tide.tide_rms_norm_backward(ddy, dh, w.to(DEV), torch.from_numpy(rstd).to(DEV), dx, dweight=dw, dres=ddres)
    args = (dy.double().numpy(), hv, w.double().numpy(), rstd.astype(np.float64))
    wx, ww = R.rms_norm_backward(*args, dres.double().numpy())
    n, g = hv * rstd[:, None].astype(np.float64), args[0] * args[2]
    # Each term of dx with a few roundings; the mean is a sum of at most 64 + log2 steps deep of |g n|.
    e = 96 * R.FP32
    size = rstd[:, None] * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(1, keepdims=True)) + np.abs(dres.double().numpy())
    R.check(dx, wx, R.rounding(dtype) * np.abs(wx) + e * size, "dx")
    # dw: rows / groups additions in a thread, groups / 32 and 32 after it.
    R.check(dw, ww, R.rounding(dtype) * np.abs(ww) + (rows / 4 + 96) * R.FP32 * np.abs(args[0] * n).sum(0), "dw")
    assert untouched(dx, xb)
    # in place, and each output by itself
    again = dw.clone()
    tide.tide_rms_norm_backward(ddy, dh, w.to(DEV), torch.from_numpy(rstd).to(DEV), None, dweight=again)
    assert torch.equal(again, dw)
    tide.tide_rms_norm_backward(ddy, dh, w.to(DEV), torch.from_numpy(rstd).to(DEV), ddy, dres=ddres)
    assert torch.equal(ddy, dx)
    wx0, _ = R.rms_norm_backward(*args, None)
    ddy2 = put(dy, lead, extra)[0]
    tide.tide_rms_norm_backward(ddy2, dh, w.to(DEV), torch.from_numpy(rstd).to(DEV), dx)
    R.check(dx, wx0, R.rounding(dtype) * np.abs(wx0) + e * size, "dx without dres")


def test_norm_backward_is_the_forwards_derivative():
    """GPU gradients against central differences of the 64-bit forward."""
    rows, cols, eps = 3, 40, 1e-3
    x, r, w, dy = (rand(s, FP, k, loud=False) for k, s in enumerate([(rows, cols), (rows, cols), (cols,), (rows, cols)]))
    xd, rd, wd, dyd = (t.double().numpy() for t in (x, r, w, dy))
    h, y, rstd = (torch.empty(s, device=DEV) for s in ((rows, cols), (rows, cols), (rows,)))
    dx, dw = torch.empty(rows, cols, device=DEV), torch.empty(cols, device=DEV)
    tide.tide_rms_norm(x.to(DEV), w.to(DEV), eps, y=y, residual=r.to(DEV), h=h, rstd=rstd)
    tide.tide_rms_norm_backward(dy.to(DEV), h, w.to(DEV), rstd, dx, dweight=dw)

    def loss(xx, ww):
        return (R.rms_norm(xx, rd, ww, eps)[1] * dyd).sum()

    d = 1e-5
    for at in np.ndindex(rows, cols):
        e = np.zeros((rows, cols))
        e[at] = d
        assert abs((loss(xd + e, wd) - loss(xd - e, wd)) / (2 * d) - dx[at].item()) < 2e-4
    for j in range(cols):
        e = np.zeros(cols)
        e[j] = d
        assert abs((loss(xd, wd + e) - loss(xd, wd - e)) / (2 * d) - dw[j].item()) < 2e-4


# ---------------------------------------------------------------- linear

PRODUCTS = [(1, 1, 1), (1, 64, 64), (2, 7, 5), (3, 128, 100), (17, 33, 65), (64, 64, 64), (100, 200, 300),
            (128, 512, 256), (129, 65, 257), (1, 2048, 768), (5, 1000, 2047), (257, 768, 520), (130, 4095, 33),
            (300, 24, 1000), (520, 136, 264)]  # rows, inner, outer


def product_case(rows, inner, outer, lead, extra):
    x = rand((rows, inner), BF, 1)
    w = rand((outer, inner), BF, 2, scale=max(1, inner) ** -0.5)
    return x, w, put(x, lead, extra)[0], put(w, lead, extra)[0]


@pytest.mark.parametrize("lead,extra", [(0, 0), (8, 8), (1, 3)])
@pytest.mark.parametrize("name", R.ACTS)
@pytest.mark.parametrize("rows,inner,outer", PRODUCTS)
def test_linear(rows, inner, outer, name, lead, extra):
    x, w, dx, dw = product_case(rows, inner, outer, lead, extra)
    b, r = rand((outer,), BF, 3), rand((rows, outer), BF, 4)
    y, yb = blank(rows, outer, BF, lead, extra)
    z, zb = blank(rows, outer, BF, lead, extra)
    dr = put(r, lead, extra)[0]
    tide.tide_linear(dx, dw, y, bias=b.to(DEV), act=name, residual=dr, z=z)
    xd, wd = x.double().numpy(), w.double().numpy()
    wz = xd @ wd.T + b.double().numpy()
    err = R.product_bound(xd, wd) + R.FP32 * np.abs(wz)
    R.check(z, wz, R.BF16 * np.abs(wz) + err, "z")
    rd = r.double().numpy()
    wy = R.act(name, wz) + rd
    # |f'| is at most 1.13; f's own fp32 error as in the checkpoint's load.
    ferr = 1.13 * err + 64 * R.FP32 * (np.abs(wz) + 20)
    R.check(y, wy, R.BF16 * np.abs(wy) + ferr + R.FP32 * np.abs(rd), "y")
    assert untouched(y, yb) and untouched(z, zb)
    z8, cb, sb = checkpoint(rows, outer, lead if lead % 8 else 16, extra if extra % 8 else 16)
    y2, _ = blank(rows, outer, BF, lead, extra)
    tide.tide_linear(dx, dw, y2, bias=b.to(DEV), act=name, residual=dr, z=z8)
    assert torch.equal(y, y2)
    R.check_kept(z8.codes, z8.scales, wz, err, "z8")
    assert untouched(z8.codes, cb) and untouched(z8.scales, sb)
    tide.tide_linear(dx, dw, dr, bias=b.to(DEV), act=name, residual=dr)  # in place
    assert torch.equal(dr, y)
    tide.tide_linear(dx, dw, y)
    w0 = xd @ wd.T
    R.check(y, w0, R.BF16 * np.abs(w0) + err, "plain product")


@pytest.mark.parametrize("lead,extra", [(0, 0), (8, 8), (1, 3)])
@pytest.mark.parametrize("kept", ["no", "bf16", "mx8"])
@pytest.mark.parametrize("rows,inner,outer", PRODUCTS)
def test_linear_grad_input(rows, inner, outer, kept, lead, extra):
    dy, w = rand((rows, outer), BF, 1), rand((outer, inner), BF, 2, scale=outer ** -0.5)
    z = rand((rows, inner), BF, 3, loud=False)
    ddy, dw = put(dy, lead, extra)[0], put(w, lead, extra)[0]
    dx, xb = blank(rows, inner, BF, lead, extra)
    yd, wd = dy.double().numpy(), w.double().numpy()
    base, err = yd @ wd, R.product_bound(yd, wd.T)
    if kept == "no":
        tide.tide_linear_grad_input(ddy, dw, dx)
        R.check(dx, base, R.BF16 * np.abs(base) + err, "dx")
        assert untouched(dx, xb)
        return
    if kept == "mx8":
        codes, scales = R.quantise(z.double().numpy())
        zv = R.values(codes, scales)
        dz = tide.Checkpoint8(put(torch.from_numpy(codes), lead, extra)[0], put(torch.from_numpy(scales), lead, extra)[0])
    else:
        zv, dz = z.double().numpy(), put(z, lead, extra)[0]
    for name in R.ACTS[1:]:
        tide.tide_linear_grad_input(ddy, dw, dx, act=name, z=dz)
        want = base * R.act_grad(name, zv)
        R.check(dx, want, R.BF16 * np.abs(want) + 1.13 * err + 64 * 20 * R.FP32 * np.abs(base), name)
        assert untouched(dx, xb)


@pytest.mark.parametrize("lead,extra", [(0, 0), (8, 8), (1, 3)])
@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("rows,inner,outer", PRODUCTS + [(3000, 40, 72)])
def test_linear_grad_weight(rows, inner, outer, kept, lead, extra):
    dy, x = rand((rows, outer), BF, 1), rand((rows, inner), BF, 2)
    ddy = put(dy, lead, extra)[0]
    dw, wb = blank(outer, inner, BF, lead, extra)
    db = torch.empty(outer, dtype=BF, device=DEV)
    if kept:
        codes, scales = R.quantise(x.double().numpy())
        xv = R.values(codes, scales)
        dx = tide.Checkpoint8(put(torch.from_numpy(codes), lead, extra)[0], put(torch.from_numpy(scales), lead, extra)[0])
    else:
        xv, dx = x.double().numpy(), put(x, lead, extra)[0]
    yd = dy.double().numpy()
    wb_sum = yd.sum(0)
    for name in (R.ACTS if kept else ("none",)):
        tide.tide_linear_grad_weight(ddy, dx, dw, db=db, act=name)
        f = R.act(name, xv)
        if name != "none":  # the operand is f rounded to bf16: its fp32 error may move it one bf16 step
            ferr = 2.0 ** -8 * np.abs(f) + 64 * R.FP32 * (np.abs(xv) + 20)
        else:
            ferr = np.zeros_like(f)
        want = yd.T @ f
        tol = R.BF16 * np.abs(want) + R.product_bound(yd.T, f.T) + np.abs(yd).T @ ferr
        R.check(dw, want, tol, "dw " + name)
        R.check(db, wb_sum, R.BF16 * np.abs(wb_sum) + (rows / 16 + 96) * R.FP32 * np.abs(yd).sum(0), "db")
        assert untouched(dw, wb)
    again = dw.clone()
    tide.tide_linear_grad_weight(ddy, dx, again, act=name)
    assert torch.equal(again, dw)


def test_linear_gradients_are_the_forwards_derivatives():
    """grad_input and grad_weight of y = f(x W1^T + b) W2^T against central differences in 64 bits."""
    t, k, m, n = 3, 6, 5, 4
    x, w1, b, w2, dy = (rand(s, BF, i, loud=False) for i, s in enumerate([(t, k), (m, k), (m,), (n, m), (t, n)]))
    d64 = [v.double().numpy() for v in (x, w1, b, w2, dy)]

    def loss(xx, ww1, bb, ww2, act):
        return (R.act(act, xx @ ww1.T + bb) @ ww2.T * d64[4]).sum()

    for act in ("gelu", "silu", "gelu_erf"):
        gpu = [v.to(DEV) for v in (x, w1, b, w2, dy)]
        a, z = torch.empty(t, m, dtype=BF, device=DEV), torch.empty(t, m, dtype=BF, device=DEV)
        tide.tide_linear(gpu[0], gpu[1], a, bias=gpu[2], act=act, z=z)
        dz, dx = torch.empty(t, m, dtype=BF, device=DEV), torch.empty(t, k, dtype=BF, device=DEV)
        tide.tide_linear_grad_input(gpu[4], gpu[3], dz, act=act, z=z)
        tide.tide_linear_grad_input(dz, gpu[1], dx)
        dw1, db = torch.empty(m, k, dtype=BF, device=DEV), torch.empty(m, dtype=BF, device=DEV)
        tide.tide_linear_grad_weight(dz, gpu[0], dw1, db=db)
        dw2 = torch.empty(n, m, dtype=BF, device=DEV)
        tide.tide_linear_grad_weight(gpu[4], a, dw2)
        for i, got in ((0, dx), (1, dw1), (2, db), (3, dw2)):
            num = np.zeros(d64[i].shape)
            for at in np.ndindex(*num.shape):
                args = [v.copy() for v in d64[:4]]
                args[i][at] += 1e-5
                up = loss(*args, act)
                args[i][at] -= 2e-5
                num[at] = (up - loss(*args, act)) / 2e-5
            # z, a, dz and the result are each rounded to bf16 (2^-9), with sums of up to 6 such terms
            R.check(got, num, 0.05 * np.abs(num) + 0.05 * np.abs(num).max(), f"{act} {i}")


def test_nothing_to_sum():
    """A product over no terms is zero: the epilogue still runs; no rows give zero gradients."""
    e = torch.empty
    y = torch.full((4, 6), 9.0, dtype=BF, device=DEV)
    b = rand((6,), BF, 1).to(DEV)
    tide.tide_linear(e(4, 0, dtype=BF, device=DEV), e(6, 0, dtype=BF, device=DEV), y, bias=b, act="relu")
    assert torch.equal(y, b.clamp(min=0).expand(4, 6))
    dx = torch.full((4, 5), 9.0, dtype=BF, device=DEV)
    tide.tide_linear_grad_input(e(4, 0, dtype=BF, device=DEV), e(0, 5, dtype=BF, device=DEV), dx)
    assert (dx == 0).all()
    dw, db = torch.full((6, 5), 9.0, dtype=BF, device=DEV), torch.full((6,), 9.0, dtype=BF, device=DEV)
    for x in (e(0, 5, dtype=BF, device=DEV), tide.Checkpoint8.empty(0, 5)):
        dw.fill_(9), db.fill_(9)
        tide.tide_linear_grad_weight(e(0, 6, dtype=BF, device=DEV), x, dw, db=db)
        assert (dw == 0).all() and (db == 0).all()
    g = torch.full((5,), 9.0, device=DEV)
    tide.tide_rms_norm_backward(e(0, 5, device=DEV), e(0, 5, device=DEV), torch.ones(5, device=DEV), e(0, device=DEV),
                                e(0, 5, device=DEV), dweight=g)
    assert (g == 0).all()
    tide.tide_linear(e(0, 5, dtype=BF, device=DEV), e(6, 5, dtype=BF, device=DEV), e(0, 6, dtype=BF, device=DEV))
    tide.tide_checkpoint_store(e(0, 5, device=DEV), tide.Checkpoint8.empty(0, 5))
    tide.tide_checkpoint_load(tide.Checkpoint8.empty(3, 0), e(3, 0, device=DEV))
    tide.tide_rms_norm(e(0, 5, device=DEV), torch.ones(5, device=DEV), 1e-5, y=e(0, 5, device=DEV))


def test_bad_values_stay_in_their_rows():
    """A NaN or infinite token touches its own row of y, dx alone, and padding never lends one to its neighbours."""
    rows, inner, outer = 70, 72, 136
    x, w = rand((rows, inner), BF, 1), rand((outer, inner), BF, 2)
    x[3, 5], x[60, 71] = float("nan"), float("inf")
    good = [r for r in range(rows) if r not in (3, 60)]
    y = torch.empty(rows, outer, dtype=BF, device=DEV)
    tide.tide_linear(put(x, 8, 8)[0], put(w, 8, 8)[0], y)  # NaN lies between the rows
    xd, wd = x.double().numpy(), w.double().numpy()
    want = xd[good] @ wd.T
    R.check(y[good], want, R.BF16 * np.abs(want) + R.product_bound(xd[good], wd), "good rows")
    assert y[3].isnan().all() and not y[60].isfinite().any()
    dx = torch.empty(rows, inner, dtype=BF, device=DEV)
    dy = rand((rows, outer), BF, 3)
    dy[3, 0] = float("inf")
    tide.tide_linear_grad_input(put(dy, 8, 8)[0], put(w, 8, 8)[0], dx)
    assert dx[good].isfinite().all() and not dx[3].isfinite().any()


# ---------------------------------------------------------------- how they are called

def block_calls(s):
    """One call of each operator on the tensors of `s`, in the order of a training step."""
    tide.tide_rms_norm(s["x"], s["nw"], 1e-5, y=s["n"], rstd=s["rstd"], y8=s["n8"], stream=s.get("stream"))
    tide.tide_linear(s["n"], s["w"], s["a"], bias=s["b"], act="gelu", z=s["z8"], stream=s.get("stream"))
    tide.tide_linear_grad_input(s["da"], s["w2"], s["dz"], act="gelu", z=s["z8"], stream=s.get("stream"))
    tide.tide_linear_grad_weight(s["dz"], s["n8"], s["dw"], db=s["db"], stream=s.get("stream"))
    tide.tide_linear_grad_input(s["dz"], s["w"], s["dn"], stream=s.get("stream"))
    tide.tide_rms_norm_backward(s["dn"], s["x"], s["nw"], s["rstd"], s["dx"], dweight=s["dnw"], stream=s.get("stream"))


def block_state(rows=70, d=136, f=200, seed=0):
    g = torch.Generator().manual_seed(seed)

    def r(*shape):
        return torch.randn(*shape, generator=g).to(BF).to(DEV)

    def e(*shape):
        return torch.zeros(*shape, dtype=BF, device=DEV)

    return {"x": r(rows, d), "nw": r(d), "n": e(rows, d), "rstd": torch.zeros(rows, device=DEV),
            "n8": tide.Checkpoint8.empty(rows, d), "w": r(f, d), "b": r(f), "a": e(rows, f),
            "z8": tide.Checkpoint8.empty(rows, f), "da": r(rows, d), "w2": r(d, f), "dz": e(rows, f), "dw": e(f, d),
            "db": e(f), "dn": e(rows, d), "dx": e(rows, d), "dnw": e(d)}


OUT = ("n", "a", "dz", "dw", "db", "dn", "dx", "dnw", "rstd")


@pytest.mark.parametrize("rows,d,f", [(70, 136, 200), (33, 61, 77)])
def test_side_stream_and_graph_replay(rows, d, f):
    s = block_state(rows, d, f)
    block_calls(s)
    torch.cuda.synchronize()
    want = {k: s[k].clone() for k in OUT}
    assert all(want[k].isfinite().all() and want[k].any() for k in OUT)
    side = torch.cuda.Stream()
    t = block_state(rows, d, f)
    t["stream"] = side
    side.wait_stream(torch.cuda.current_stream())
    block_calls(t)
    side.synchronize()
    assert all(torch.equal(t[k], want[k]) for k in OUT)
    g, u = torch.cuda.CUDAGraph(), block_state(rows, d, f, seed=1)
    with torch.cuda.graph(g):
        block_calls(u)
    for k, v in block_state(rows, d, f).items():
        if k in ("x", "nw", "w", "b", "da", "w2"):
            u[k].copy_(v)
    for _ in range(3):
        for k in OUT:
            u[k].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u[k], want[k]) for k in OUT)


def test_offsets_past_32_bits():
    """Rows more than 2^31 elements apart, in every operand."""
    ld, rows = (1 << 30) + 8, 3

    def far(cols, dtype, vals=None):
        buf = torch.empty(ld * (rows - 1) + cols, dtype=dtype, device=DEV)
        v = buf.as_strided((rows, cols), (ld, 1))
        if vals is not None:
            v.copy_(vals)
        return v

    cols, outer = 200, 72
    x, w = rand((rows, cols), BF, 1), rand((outer, cols), BF, 2, scale=0.1)
    dx, y = far(cols, BF, x), far(cols, BF)
    ck = tide.Checkpoint8(far(cols, torch.uint8), far(7, torch.uint8))
    near = tide.Checkpoint8.empty(rows, cols)
    tide.tide_checkpoint_store(dx, ck)
    tide.tide_checkpoint_store(x.to(DEV), near)
    assert torch.equal(ck.codes, near.codes) and torch.equal(ck.scales, near.scales)
    tide.tide_checkpoint_load(ck, y)
    near_y = torch.empty(rows, cols, dtype=BF, device=DEV)
    tide.tide_checkpoint_load(near, near_y)
    assert torch.equal(y, near_y)
    nw = torch.ones(cols, dtype=BF, device=DEV)
    tide.tide_rms_norm(dx, nw, 1e-5, y=y)
    tide.tide_rms_norm(x.to(DEV), nw, 1e-5, y=near_y)
    assert torch.equal(y, near_y)
    o, near_o = far(outer, BF), torch.empty(rows, outer, dtype=BF, device=DEV)
    tide.tide_linear(dx, w.to(DEV), o)
    tide.tide_linear(x.to(DEV), w.to(DEV), near_o)
    assert torch.equal(o, near_o)
    g, near_g = torch.empty(outer, cols, dtype=BF, device=DEV), torch.empty(outer, cols, dtype=BF, device=DEV)
    tide.tide_linear_grad_weight(o, ck, g)
    tide.tide_linear_grad_weight(near_o, near, near_g)
    assert torch.equal(g, near_g)


def test_many_rows():
    """More rows and elements than 32 bits of bytes: first and last rows come out as when called alone."""
    rows, cols = 70001, 32768 + 8
    x = torch.zeros(rows, cols, dtype=BF, device=DEV)
    x[-2:] = rand((2, cols), BF, 1).to(DEV)
    ck = tide.Checkpoint8.empty(rows, cols)
    tide.tide_checkpoint_store(x, ck)
    codes, scales = R.quantise(x[-2:].double().cpu().numpy())
    assert np.array_equal(ck.codes[-2:].cpu().numpy(), codes) and np.array_equal(ck.scales[-2:].cpu().numpy(), scales)
    assert not ck.codes[:-2].any() and not ck.scales[:-2].any()
    tide.tide_checkpoint_load(ck, x, act="silu")
    R.check(x[-2:], R.act("silu", R.values(codes, scales)), np.inf, "last rows")
    assert not x[:-2].any() and x[-1].any()


def test_refusals():
    """Bad arguments are refused before anything is launched, and the GPU stays usable."""
    def refused(status, f, *a, **k):
        with pytest.raises(tide.TideError) as e:
            f(*a, **k)
        assert e.value.status == status, e.value

    x, w = torch.zeros(4, 8, dtype=BF, device=DEV), torch.zeros(6, 8, dtype=BF, device=DEV)
    y, b = torch.zeros(4, 6, dtype=BF, device=DEV), torch.zeros(6, dtype=BF, device=DEV)
    refused(1, tide.tide_linear, x.float(), w, y)
    refused(1, tide.tide_linear, x, w, y.float())
    refused(1, tide.tide_linear, x, w[:, :7], y)
    refused(1, tide.tide_linear, x, w, y[:, :5])
    refused(1, tide.tide_linear, x.cpu(), w, y)
    refused(1, tide.tide_linear, x, w, y, bias=b[:5])
    refused(1, tide.tide_linear, x, w, y, act="tanh")
    refused(1, tide.tide_linear, x, w, y, residual=y.float())
    refused(1, tide.tide_linear, x.t().contiguous().t(), w, y)
    refused(1, tide.tide_linear, x[0], w, y)
    refused(1, tide.tide_linear, x, w, y, z=tide.Checkpoint8.empty(4, 5))
    refused(1, tide.tide_linear_grad_input, y, w, x, act="relu")
    refused(1, tide.tide_linear_grad_weight, y, x, w, act="relu")
    refused(1, tide.tide_linear_grad_weight, y, tide.Checkpoint8.empty(4, 8), w,
            workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
    refused(1, tide.tide_rms_norm, x, b, 1e-5, y=x)
    refused(1, tide.tide_rms_norm, x.half(), x[0].half(), 1e-5)
    refused(6, tide.tide_rms_norm, torch.zeros(1, 16385, device=DEV), torch.zeros(16385, device=DEV), 1e-5)
    refused(1, tide.tide_rms_norm_backward, x, x, x[0], torch.zeros(4, device=DEV), x, dweight=x[1],
            workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    refused(1, tide.tide_rms_norm_backward, x, x, x[0], torch.zeros(4, device=DEV)[:3], x)
    refused(1, tide.Checkpoint8, torch.zeros(4, 33, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8))
    refused(1, tide.Checkpoint8, torch.zeros(4, 33, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8))
    refused(1, tide.tide_checkpoint_store, x, tide.Checkpoint8.empty(4, 9))
    refused(1, tide.tide_checkpoint_load, tide.Checkpoint8.empty(4, 8), x, grad=x.float())
    torch.cuda.synchronize()
    tide.tide_linear(x, w, y, bias=b)
    torch.cuda.synchronize()


# ---------------------------------------------------------------- the pair-of-CTAs product, and bounded waits

# rows, inner, outer.  On 152 SMs these, and BIG_SUMS, take every tile in each of the three products: whole and in
# splits, with output rows that start on 16-byte boundaries and that do not.
BIG = [(2100, 200, 3100), (4096, 520, 2304), (2049, 1030, 2570), (3333, 72, 4100),
       (2631, 8, 672), (3562, 3017, 191), (2546, 3468, 64), (2511, 9352, 137),
       (648, 1334, 3256), (413, 4204, 4927), (136, 8384, 5392), (145, 14426, 4894),
       (1174, 8, 3607), (523, 272, 3576), (2756, 4663, 13), (68, 4624, 2256), (1820, 1313, 687), (260, 1787, 5936),
       (37, 509, 5413), (36, 5574, 504), (143, 994, 8), (141, 5416, 4683), (396, 2529, 4447), (309, 5816, 1236),
       (210, 357, 24), (1, 425, 4715), (6, 622, 538), (10, 410, 488),
       (163, 5343, 4824), (163, 5344, 4824), (806, 2688, 5240), (2930, 2726, 1587), (13, 4688, 33), (516, 3762, 2195)]
# The same for the weight gradient, whose sum runs over the rows.
BIG_SUMS = [(10, 152, 4912), (3314, 292, 3534), (2633, 4832, 64), (9352, 137, 2511), (3910, 2725, 841), (1300, 736, 3280),
            (8384, 5392, 136), (14426, 4894, 145), (8, 3790, 2253), (453, 4896, 384), (3799, 3353, 68), (4978, 3336, 72),
            (750, 11, 9), (710, 8, 9), (16384, 520, 512), (1, 5255, 792), (143, 994, 8)]


@pytest.mark.parametrize("rows,inner,outer", BIG_SUMS)
def test_large_weight_gradients(rows, inner, outer):
    dy, x = rand((rows, outer), BF, 1).to(DEV), rand((rows, inner), BF, 2).to(DEV)
    ck = tide.Checkpoint8.empty(rows, inner)
    tide.tide_checkpoint_store(x, ck)
    kept = torch.empty(rows, inner, device=DEV)
    tide.tide_checkpoint_load(ck, kept)
    yd, db = dy.double(), torch.empty(outer, dtype=BF, device=DEV)
    for operand, xd in ((x, x.double()), (ck, kept.double())):
        dw = torch.empty(outer, inner, dtype=BF, device=DEV)
        tide.tide_linear_grad_weight(dy, operand, dw, db=db)
        want, size = yd.t() @ xd, yd.abs().t() @ xd.abs()
        over = (dw.double() - want).abs() - R.BF16 * want.abs() - ((rows / 16 + 16) * R.FP32) * size
        assert over.max().item() <= 0
    want, size = yd.sum(0), yd.abs().sum(0)
    assert ((db.double() - want).abs() - R.BF16 * want.abs() - ((rows / 16 + 96) * R.FP32) * size).max().item() <= 0
    tide.tide_ops_check()


@pytest.mark.parametrize("rows,inner,outer", BIG)
def test_large_products(rows, inner, outer):
    """Every tile the products are built of, whole and ragged, against fp64 on the GPU."""
    x, w = rand((rows, inner), BF, 1).to(DEV), rand((outer, inner), BF, 2, scale=inner ** -0.5).to(DEV)
    b, r = rand((outer,), BF, 3).to(DEV), rand((rows, outer), BF, 4).to(DEV)
    xd, wd = x.double(), w.double()

    def near(got, want, size, k, what):
        # the output's rounding and the accumulation's (R.product_bound)
        tol = R.BF16 * want.abs() + ((k / 16 + 16) * R.FP32) * size + 64 * R.FP32 * (want.abs() + 20)
        over = (got.double() - want).abs() - tol
        assert over.max().item() <= 0, (what, over.max().item())

    z = xd @ wd.t() + b.double()
    size = xd.abs() @ wd.abs().t() + b.double().abs()
    y, kz, k8 = (torch.empty(rows, outer, dtype=BF, device=DEV), torch.empty(rows, outer, dtype=BF, device=DEV),
                 tide.Checkpoint8.empty(rows, outer))
    tide.tide_linear(x, w, y, bias=b, act="silu", residual=r, z=kz)
    near(kz, z, size, inner, "z")
    near(y, z * torch.sigmoid(z) + r.double(), 1.13 * size, inner, "y")
    tide.tide_linear(x, w, y, bias=b, z=k8)
    near(y, z, size, inner, "plain y")
    back = torch.empty(rows, outer, device=DEV)
    tide.tide_checkpoint_load(k8, back)
    s = torch.exp2(k8.scales.double() - 127).repeat_interleave(32, 1)[:, :outer]
    # half the gap between codes, and the product's own error
    over = (back.double() - z).abs() - torch.maximum(2.0 ** -4 * z.abs(), 2.0 ** -10 * s) - (inner / 16 + 16) * R.FP32 * size
    assert over.max().item() <= 0
    zv = back.double()
    dx = torch.empty(rows, outer, dtype=BF, device=DEV)
    wt = rand((inner, outer), BF, 5, scale=inner ** -0.5).to(DEV)
    tide.tide_linear_grad_input(x, wt, dx, act="silu", z=k8)
    p = torch.sigmoid(zv)
    f = p + zv * p * (1 - p)
    near(dx, (xd @ wt.double()) * f, 1.13 * (xd.abs() @ wt.double().abs()), inner, "dx")
    dw, db = torch.empty(outer, inner, dtype=BF, device=DEV), torch.empty(outer, dtype=BF, device=DEV)
    tide.tide_linear_grad_weight(r, x, dw, db=db)
    near(dw, r.double().t() @ xd, r.double().abs().t() @ xd.abs(), rows, "dw")
    near(db, r.double().sum(0), r.double().abs().sum(0), rows, "db")
    big = torch.empty(outer, outer, dtype=BF, device=DEV)
    tide.tide_linear_grad_weight(r, k8, big)
    near(big, r.double().t() @ zv, r.double().abs().t() @ zv.abs(), rows, "dw of a checkpoint")
    tide.tide_ops_check()


@pytest.mark.parametrize("rows,inner,outer", [(64, 4096, 256), (2100, 1024, 3100)])
def test_a_wait_that_runs_out_is_reported(rows, inner, outer):
    """A block whose loads are withheld: the kernels give up in time, say so once, and the next call is right."""
    x, w = rand((rows, inner), BF, 1).to(DEV), rand((outer, inner), BF, 2).to(DEV)
    y, want = (torch.empty(rows, outer, dtype=BF, device=DEV) for _ in range(2))
    tide.tide_linear(x, w, want)
    tide.tide_ops_check()
    tide.tide_ops_set_option(tide.TIDE_OPS_OPT_WAIT_LIMIT_NS, 20_000_000)
    tide.tide_ops_set_option(tide.TIDE_OPS_OPT_TEST_DROP_LOAD, 2)
    try:
        tide.tide_linear(x, w, y)
        with pytest.raises(tide.TideError) as e:
            tide.tide_ops_check()
        assert e.value.status == 8
    finally:
        tide.tide_ops_set_option(tide.TIDE_OPS_OPT_TEST_DROP_LOAD, -1)
        tide.tide_ops_set_option(tide.TIDE_OPS_OPT_WAIT_LIMIT_NS, 2_000_000_000)
    tide.tide_ops_check()
    tide.tide_linear(x, w, y)
    tide.tide_ops_check()
    assert torch.equal(y, want)


@pytest.mark.parametrize("rows,cols,kept", [(4000, 1024, False), (3000, 2048, True), (2000, 333, True), (900, 9000, False),
                                            (900, 16383, True)])
def test_a_copy_that_does_not_come_is_reported(rows, cols, kept):
    """The same for the norm's backward pass, whose rows are copied ahead."""
    h, dy = rand((rows, cols), BF, 1).to(DEV), rand((rows, cols), BF, 2).to(DEV)
    w, rstd = torch.ones(cols, dtype=BF, device=DEV), torch.ones(rows, device=DEV)
    if kept:
        ck = tide.Checkpoint8.empty(rows, cols)
        tide.tide_checkpoint_store(h, ck)
        h = ck
    out = [[torch.empty(rows, cols, dtype=BF, device=DEV), torch.empty(cols, dtype=BF, device=DEV)] for _ in range(2)]
    tide.tide_rms_norm_backward(dy, h, w, rstd, out[0][0], dweight=out[0][1])
    tide.tide_ops_check()
    tide.tide_ops_set_option(tide.TIDE_OPS_OPT_WAIT_LIMIT_NS, 20_000_000)
    tide.tide_ops_set_option(tide.TIDE_OPS_OPT_TEST_DROP_LOAD, 1)
    try:
        tide.tide_rms_norm_backward(dy, h, w, rstd, out[1][0], dweight=out[1][1])
        with pytest.raises(tide.TideError) as e:
            tide.tide_ops_check()
        assert e.value.status == 8
    finally:
        tide.tide_ops_set_option(tide.TIDE_OPS_OPT_TEST_DROP_LOAD, -1)
        tide.tide_ops_set_option(tide.TIDE_OPS_OPT_WAIT_LIMIT_NS, 2_000_000_000)
    tide.tide_rms_norm_backward(dy, h, w, rstd, out[1][0], dweight=out[1][1])
    tide.tide_ops_check()
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
