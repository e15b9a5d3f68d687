"""Host side of the training-block operators: the C entry points' argument
checks (no GPU call is reached), the header, and the 64-bit reference's own
consistency."""

import os
import re
import subprocess

import numpy as np
import pytest

import fsdp_layout_aware_gb300 as tide
import ops_reference as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # an address that is never followed
OK, INVALID, ALIGNMENT, OVERFLOW, UNIMPLEMENTED = 0, 1, 2, 3, 6


def lib():
    tide.tide_linear  # loads the operators' declarations
    from fsdp_layout_aware_gb300.tide import _lib
    return _lib


def store(rows=4, cols=40, dtype=0, x=P, ldx=40, codes=P, ldc=40, scales=P, lds=2):
    return lib().tide_checkpoint_store(rows, cols, dtype, x, ldx, codes, ldc, scales, lds, None)


def load(rows=4, cols=40, codes=P, ldc=40, scales=P, lds=2, act=0, dtype=0, grad=None, ldg=0, out=P, ldo=40):
    return lib().tide_checkpoint_load(rows, cols, codes, ldc, scales, lds, act, dtype, grad, ldg, out, ldo, None)


def norm(rows=4, cols=40, dtype=0, x=P, ldx=40, r=None, ldr=0, w=P, h=None, ldh=0, y=P, ldy=40, rstd=None, codes=None,
         ldc=0, scales=None, lds=0):
    return lib().tide_rms_norm(rows, cols, dtype, x, ldx, r, ldr, w, 1e-5, h, ldh, y, ldy, rstd, codes, ldc, scales,
                               lds, None)


def norm_grad(rows=4, cols=40, dtype=0, dy=P, lddy=40, h=P, ldh=40, codes=None, ldc=0, scales=None, lds=0, w=P, rstd=P,
              dres=None, ldd=0, dx=P, lddx=40, dw=None, ws=None, wsb=0):
    return lib().tide_rms_norm_backward(rows, cols, dtype, dy, lddy, h, ldh, codes, ldc, scales, lds, w, rstd, dres,
                                        ldd, dx, lddx, dw, ws, wsb, None)


def linear(rows=4, inner=8, outer=16, x=P, ldx=8, w=P, ldw=8, b=None, act=0, r=None, ldr=0, y=P, ldy=16, z=None, ldz=0,
           codes=None, ldc=0, scales=None, lds=0, ws=None, wsb=0):
    return lib().tide_linear(rows, inner, outer, x, ldx, w, ldw, b, act, r, ldr, y, ldy, z, ldz, codes, ldc, scales,
                             lds, ws, wsb, None)


def grad_input(rows=4, inner=8, outer=16, dy=P, lddy=16, w=P, ldw=8, act=0, z=None, ldz=0, codes=None, ldc=0,
               scales=None, lds=0, dx=P, lddx=8, ws=None, wsb=0):
    return lib().tide_linear_grad_input(rows, inner, outer, dy, lddy, w, ldw, act, z, ldz, codes, ldc, scales, lds, dx,
                                        lddx, ws, wsb, None)


def grad_weight(rows=4, inner=8, outer=16, dy=P, lddy=16, x=P, ldx=8, codes=None, ldc=0, scales=None, lds=0, act=0,
                dw=P, lddw=8, db=None, ws=None, wsb=0):
    return lib().tide_linear_grad_weight(rows, inner, outer, dy, lddy, x, ldx, codes, ldc, scales, lds, act, dw, lddw,
                                         db, ws, wsb, None)


CASES = [
    (store, dict(rows=-1), INVALID), (store, dict(cols=-1), INVALID), (store, dict(dtype=2), INVALID),
    (store, dict(x=None), INVALID), (store, dict(codes=None), INVALID), (store, dict(scales=None), INVALID),
    (store, dict(ldx=39), INVALID), (store, dict(ldc=39), INVALID), (store, dict(lds=1), INVALID),
    (store, dict(x=P + 1), ALIGNMENT), (store, dict(dtype=1, x=P + 2), ALIGNMENT),
    (store, dict(rows=1 << 40, ldx=1 << 40), OVERFLOW), (store, dict(rows=0), OK), (store, dict(cols=0), OK),
    (store, dict(rows=1 << 40, cols=64, ldx=64, ldc=64), UNIMPLEMENTED),
    (load, dict(act=5), INVALID), (load, dict(act=-1), INVALID), (load, dict(dtype=-1), INVALID),
    (load, dict(out=None), INVALID), (load, dict(out=P + 1), ALIGNMENT), (load, dict(grad=P, ldg=3), INVALID),
    (load, dict(ldo=39), INVALID), (load, dict(rows=0), OK), (load, dict(codes=None), INVALID),
    (norm, dict(cols=16385, ldx=20000, ldy=20000), UNIMPLEMENTED), (norm, dict(w=None), INVALID),
    (norm, dict(x=None), INVALID), (norm, dict(r=P, ldr=39), INVALID), (norm, dict(h=P, ldh=39), INVALID),
    (norm, dict(y=P + 1), ALIGNMENT), (norm, dict(rstd=P + 2), ALIGNMENT), (norm, dict(codes=P, ldc=40), INVALID),
    (norm, dict(scales=P, lds=2), INVALID), (norm, dict(rows=0), OK), (norm, dict(dtype=7), INVALID),
    (norm_grad, dict(codes=P, ldc=40, scales=P, lds=2), INVALID), (norm_grad, dict(h=None), INVALID),
    (norm_grad, dict(rstd=None), INVALID), (norm_grad, dict(dy=None), INVALID), (norm_grad, dict(w=None), INVALID),
    (norm_grad, dict(dres=P, ldd=39), INVALID), (norm_grad, dict(dx=None), OK), (norm_grad, dict(lddx=39), INVALID),
    (norm_grad, dict(cols=16385, lddy=20000, ldh=20000, lddx=20000), UNIMPLEMENTED), (norm_grad, dict(rows=-3), INVALID),
    (linear, dict(rows=-1), INVALID), (linear, dict(inner=-1), INVALID), (linear, dict(outer=-1), INVALID),
    (linear, dict(x=None), INVALID), (linear, dict(w=None), INVALID), (linear, dict(y=None), INVALID),
    (linear, dict(ldx=7), INVALID), (linear, dict(ldw=7), INVALID), (linear, dict(ldy=15), INVALID),
    (linear, dict(act=9), INVALID), (linear, dict(b=P + 1), ALIGNMENT), (linear, dict(r=P, ldr=15), INVALID),
    (linear, dict(z=P, ldz=15), INVALID), (linear, dict(codes=P, ldc=16), INVALID), (linear, dict(x=P + 1), ALIGNMENT),
    (linear, dict(rows=0), OK), (linear, dict(outer=0), OK), (linear, dict(ws=P + 8, wsb=64), ALIGNMENT),
    (grad_input, dict(act=1), INVALID), (grad_input, dict(act=1, z=P, ldz=7), INVALID),
    (grad_input, dict(act=1, z=P, ldz=8, codes=P, ldc=8, scales=P, lds=1), INVALID),
    (grad_input, dict(dy=None), INVALID), (grad_input, dict(w=None), INVALID), (grad_input, dict(dx=None), INVALID),
    (grad_input, dict(lddx=7), INVALID), (grad_input, dict(inner=0), OK), (grad_input, dict(act=-2), INVALID),
    (grad_weight, dict(act=1), INVALID), (grad_weight, dict(x=None), INVALID), (grad_weight, dict(dw=None), INVALID),
    (grad_weight, dict(x=None, codes=P, ldc=8, scales=P, lds=1), INVALID),  # no workspace for the loaded operand
    (grad_weight, dict(codes=P, ldc=8, scales=P, lds=1), INVALID), (grad_weight, dict(db=P + 1), ALIGNMENT),
    (grad_weight, dict(lddw=7), INVALID), (grad_weight, dict(outer=0), OK), (grad_weight, dict(dy=None), INVALID),
]


@pytest.mark.parametrize("f,args,status", CASES)
def test_arguments_are_checked_on_the_host(f, args, status):
    assert f(**args) == status, lib().tide_last_error()
    if status != OK:
        assert lib().tide_last_error()


def test_every_declared_operator_is_exported_and_bound():
    text = open(os.path.join(ROOT, "include", "tide_ops.h")).read()
    names = set(re.findall(r"^\w+ (tide_\w+)\(", text, re.M))
    assert len(names) == 13
    for n in names:
        assert getattr(lib(), n).argtypes is not None, n


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "tide_ops.h"\nint main(void) { return tide_linear_workspace(0, 0, 0, 0, 0, 0, 0) != 0; }\n')
    libdir = os.path.dirname(tide.LIB_PATH)
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I", os.path.join(ROOT, "include"),
                    str(src), "-L", libdir, "-l:" + os.path.basename(tide.LIB_PATH), "-Wl,-rpath," + libdir, "-o",
                    str(tmp_path / "t")], check=True, capture_output=True, text=True)
    assert subprocess.run([str(tmp_path / "t")], timeout=120).returncode == 0


# ---- the reference against itself

def test_reference_codes_round_trip():
    fin = ~np.isnan(R.TABLE)
    c = np.arange(256)[fin].astype(np.uint8)
    assert np.array_equal(R.nearest_codes(R.TABLE[c]), c)
    mid = (R.TABLE[:126] + R.TABLE[1:127]) / 2
    assert np.array_equal(R.nearest_codes(mid) % 2, np.zeros(126))  # ties to even


def test_reference_kept_values_are_near():
    v = np.random.RandomState(0).randn(40, 70) * np.exp(np.random.RandomState(1).randn(40, 70) * 3)
    k = R.values(*R.quantise(v))
    s = 2.0 ** (R.quantise(v)[1][:, np.arange(70) // 32].astype(float) - 127)
    assert (np.abs(k - v) <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * s)).all()


@pytest.mark.parametrize("name", R.ACTS)
def test_reference_derivatives(name):
    z = np.linspace(-9, 9, 731)
    z = z[np.abs(z) > 1e-3]
    d = 1e-6
    num = (R.act(name, z + d) - R.act(name, z - d)) / (2 * d)
    assert np.abs(num - R.act_grad(name, z)).max() < 1e-8
    assert R.act_grad(name, np.array([np.inf]))[0] == 1


def test_options():
    for option, value, status in ((1, 0, INVALID), (1, -5, INVALID), (2, -2, INVALID), (3, 1, INVALID), (2, -1, OK),
                                  (1, 2_000_000_000, OK)):
        assert lib().tide_ops_set_option(option, value) == status
