"""ctypes binding of libtide's training-block operators (include/tide_ops.h).

Argument marshalling only, as in tide.py: the calls read shapes, strides and
types off the tensors, check what only Python can see (device, type, shape) and
pass addresses on.  Outputs are the caller's tensors; a workspace the caller
does not give is taken from torch's allocator for the call.

    tide_rms_norm, tide_rms_norm_backward
    tide_linear, tide_linear_grad_input, tide_linear_grad_weight
    tide_checkpoint_store, tide_checkpoint_load, Checkpoint8
"""

import ctypes

import torch

from .tide import TideError, _check, _lib, _stream

TIDE_BF16, TIDE_F32 = 0, 1
TIDE_ACT_NONE, TIDE_ACT_RELU, TIDE_ACT_GELU, TIDE_ACT_GELU_ERF, TIDE_ACT_SILU = range(5)
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_erf": 3, "silu": 4, None: 0, 0: 0, 1: 1, 2: 2, 3: 3, 4: 4}
TIDE_OPS_OPT_WAIT_LIMIT_NS, TIDE_OPS_OPT_TEST_DROP_LOAD = 1, 2
TIDE_CKPT_BLOCK = 32  # columns that share a scale

_DTYPES = {torch.bfloat16: TIDE_BF16, torch.float32: TIDE_F32}
_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
_MAT = [_vp, _i64]  # address, row stride


def _declare():
    sig = {
        "tide_ops_check": (_i32, []),
        "tide_ops_set_option": (_i32, [_i32, _i64]),
        "tide_checkpoint_store": (_i32, [_i64, _i64, _i32] + 3 * _MAT + [_vp]),
        "tide_checkpoint_load": (_i32, [_i64, _i64] + 2 * _MAT + [_i32, _i32] + 2 * _MAT + [_vp]),
        "tide_rms_norm": (_i32, [_i64, _i64, _i32] + 2 * _MAT + [_vp, ctypes.c_float] + 2 * _MAT + [_vp] + 2 * _MAT +
                          [_vp]),
        "tide_rms_norm_backward_workspace": (_i64, [_i64, _i64]),
        "tide_rms_norm_backward": (_i32, [_i64, _i64, _i32] + 4 * _MAT + [_vp, _vp] + 2 * _MAT + [_vp, _vp, _i64, _vp]),
        "tide_linear_workspace": (_i64, 3 * [_i64] + 2 * _MAT),
        "tide_linear": (_i32, 3 * [_i64] + 2 * _MAT + [_vp, _i32] + 5 * _MAT + [_vp, _i64, _vp]),
        "tide_linear_grad_input_workspace": (_i64, 3 * [_i64] + 2 * _MAT),
        "tide_linear_grad_input": (_i32, 3 * [_i64] + 2 * _MAT + [_i32] + 4 * _MAT + [_vp, _i64, _vp]),
        "tide_linear_grad_weight_workspace": (_i64, 3 * [_i64] + 2 * _MAT),
        "tide_linear_grad_weight": (_i32, 3 * [_i64] + 4 * _MAT + [_i32] + _MAT + [_vp, _vp, _i64, _vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(_lib, name)
        fn.restype = res
        fn.argtypes = args


_declare()


def _refuse(message, status=1):
    raise TideError(status, message)


class Checkpoint8:
    """A matrix kept in 8 bits: e4m3 codes (rows, cols) and one scale byte per
    block of 32 columns, (rows, ceil(cols / 32)); both uint8 on the GPU."""

    __slots__ = ("codes", "scales")

    def __init__(self, codes, scales):
        if codes.dtype is not torch.uint8 or scales.dtype is not torch.uint8:
            _refuse("a checkpoint's codes and scales are uint8")
        rows, cols = codes.shape
        if tuple(scales.shape) != (rows, -(-cols // TIDE_CKPT_BLOCK)):
            _refuse(f"scales of a ({rows}, {cols}) checkpoint are ({rows}, {-(-cols // TIDE_CKPT_BLOCK)}), "
                    f"not {tuple(scales.shape)}")
        self.codes, self.scales = codes, scales

    @classmethod
    def empty(cls, rows, cols, device="cuda"):
        return cls(torch.empty(rows, cols, dtype=torch.uint8, device=device),
                   torch.empty(rows, -(-cols // TIDE_CKPT_BLOCK), dtype=torch.uint8, device=device))

    @property
    def shape(self):
        return self.codes.shape


_NO_MAT = (None, 0)


def _mat(t, name, shape, dtype):
    """(address, row stride) of a 2-D tensor, after checking it."""
    if t.dtype is not dtype:
        _refuse(f"{name} is {t.dtype}, not {dtype}")
    if t.shape != shape:
        _refuse(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if not t.is_cuda:
        _refuse(f"{name} is not on the GPU")
    if t.get_device() != torch.cuda.current_device():
        _refuse(f"{name} is on device {t.get_device()}, which is not the current one", 7)
    ld, step = t.stride()
    if step != 1 and shape[1] > 1:
        _refuse(f"{name}: the last axis is not contiguous")
    return t.data_ptr(), ld


def _vec(t, name, n, dtype):
    if t.dtype is not dtype:
        _refuse(f"{name} is {t.dtype}, not {dtype}")
    if t.dim() != 1 or t.shape[0] != n:
        _refuse(f"{name} has shape {tuple(t.shape)}, not ({n},)")
    if not t.is_cuda:
        _refuse(f"{name} is not on the GPU")
    if t.get_device() != torch.cuda.current_device():
        _refuse(f"{name} is on device {t.get_device()}, which is not the current one", 7)
    if n > 1 and t.stride(0) != 1:
        _refuse(f"{name} is not contiguous")
    return t.data_ptr()


def _ckpt(c, name, shape):
    """codes and scales of a checkpoint: (address, stride, address, stride)."""
    rows, cols = shape
    return _mat(c.codes, name + ".codes", shape, torch.uint8) + _mat(
        c.scales, name + ".scales", (rows, -(-cols // TIDE_CKPT_BLOCK)), torch.uint8)


def _opt(t, name, shape, dtype):
    return _NO_MAT if t is None else _mat(t, name, shape, dtype)


def _optv(t, name, n, dtype):
    return None if t is None else _vec(t, name, n, dtype)


def _dtype(t, name):
    code = _DTYPES.get(t.dtype)
    if code is None:
        _refuse(f"{name} is {t.dtype}; bfloat16 and float32 are built")
    return code


def _shape2(t, name):
    if t.dim() != 2:
        _refuse(f"{name} has {t.dim()} axes, not 2")
    return t.shape


def _act(act):
    code = ACTS.get(act)
    if code is None:
        _refuse(f"unknown activation {act!r}")
    return code


def _workspace(given, need, stream):
    """(tensor that keeps it alive, address, bytes)."""
    if given is not None:
        if not given.is_cuda or not given.is_contiguous():
            _refuse("workspace is not a contiguous tensor on the GPU")
        return given, given.data_ptr(), given.numel() * given.element_size()
    if need == 0:
        return None, None, 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    if stream is not None:
        # The block must not go to another call of the allocating stream while this one still uses it.
        ws.record_stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream))
    return ws, ws.data_ptr(), need


def tide_ops_check():
    """Synchronise and raise TideError(TIDE_ERR_TIMEOUT) if an operator's kernel gave up a wait on this device."""
    _check(_lib.tide_ops_check())


def tide_ops_set_option(option, value):
    _check(_lib.tide_ops_set_option(option, value))


def tide_checkpoint_store(x, ckpt, stream=None):
    """Keep x (rows, cols; bf16 or fp32) in ckpt (a Checkpoint8 of that shape)."""
    shape = _shape2(x, "x")
    _check(_lib.tide_checkpoint_store(*shape, _dtype(x, "x"), *_mat(x, "x", shape, x.dtype),
                                      *_ckpt(ckpt, "ckpt", shape), _stream(stream)))


def tide_checkpoint_load(ckpt, out, act=TIDE_ACT_NONE, grad=None, stream=None):
    """out = f(values), or grad * f'(values) when grad is given (out may be grad)."""
    shape = ckpt.shape
    _check(_lib.tide_checkpoint_load(*shape, *_ckpt(ckpt, "ckpt", shape), _act(act), _dtype(out, "out"),
                                     *_opt(grad, "grad", shape, out.dtype), *_mat(out, "out", shape, out.dtype),
                                     _stream(stream)))


def tide_rms_norm(x, weight, eps, y=None, residual=None, h=None, rstd=None, y8=None, stream=None):
    """h = x + residual; y (and y8, a Checkpoint8) = h * rstd * weight, rstd = (mean(h^2) + eps)^-1/2 per row."""
    shape = _shape2(x, "x")
    t = x.dtype
    _check(_lib.tide_rms_norm(*shape, _dtype(x, "x"), *_mat(x, "x", shape, t), *_opt(residual, "residual", shape, t),
                              _vec(weight, "weight", shape[1], t), eps, *_opt(h, "h", shape, t),
                              *_opt(y, "y", shape, t), _optv(rstd, "rstd", shape[0], torch.float32),
                              *(_NO_MAT + _NO_MAT if y8 is None else _ckpt(y8, "y8", shape)), _stream(stream)))


def tide_rms_norm_backward(dy, h, weight, rstd, dx=None, dweight=None, dres=None, workspace=None, stream=None):
    """Gradients of tide_rms_norm: dx (of x and of residual, dres added) and dweight; h may be a Checkpoint8."""
    shape = _shape2(dy, "dy")
    rows, cols = shape
    t = dy.dtype
    kept = (_NO_MAT + _ckpt(h, "h", shape) if isinstance(h, Checkpoint8)
            else _mat(h, "h", shape, t) + _NO_MAT + _NO_MAT)
    args = (rows, cols, _dtype(dy, "dy"), *_mat(dy, "dy", shape, t), *kept, _vec(weight, "weight", cols, t),
            _vec(rstd, "rstd", rows, torch.float32), *_opt(dres, "dres", shape, t), *_opt(dx, "dx", shape, t),
            _optv(dweight, "dweight", cols, t))
    need = 0 if dweight is None else _lib.tide_rms_norm_backward_workspace(rows, cols)
    keep, ws, ws_bytes = _workspace(workspace, need, stream)
    _check(_lib.tide_rms_norm_backward(*args, ws, ws_bytes, _stream(stream)))


def tide_linear(x, w, y, bias=None, act=TIDE_ACT_NONE, residual=None, z=None, workspace=None, stream=None):
    """y = f(x w^T + bias) + residual; z (bf16, or a Checkpoint8) keeps x w^T + bias for the backward pass."""
    rows, inner = _shape2(x, "x")
    outer = _shape2(w, "w")[0]
    bf, out = torch.bfloat16, (rows, outer)
    a, b = _mat(x, "x", (rows, inner), bf), _mat(w, "w", (outer, inner), bf)
    kept = (_NO_MAT + _ckpt(z, "z", out) if isinstance(z, Checkpoint8) else _opt(z, "z", out, bf) + _NO_MAT + _NO_MAT)
    args = (*a, *b, _optv(bias, "bias", outer, bf), _act(act), *_opt(residual, "residual", out, bf),
            *_mat(y, "y", out, bf), *kept)
    keep, ws, ws_bytes = _workspace(workspace, _lib.tide_linear_workspace(rows, inner, outer, *a, *b), stream)
    _check(_lib.tide_linear(rows, inner, outer, *args, ws, ws_bytes, _stream(stream)))


def tide_linear_grad_input(dy, w, dx, act=TIDE_ACT_NONE, z=None, workspace=None, stream=None):
    """dx = (dy w) * f'(z): z (bf16 or Checkpoint8) is the pre-activation behind this layer's input."""
    rows, outer = _shape2(dy, "dy")
    inner = _shape2(w, "w")[1]
    bf, out = torch.bfloat16, (rows, inner)
    a, b = _mat(dy, "dy", (rows, outer), bf), _mat(w, "w", (outer, inner), bf)
    kept = (_NO_MAT + _ckpt(z, "z", out) if isinstance(z, Checkpoint8) else _opt(z, "z", out, bf) + _NO_MAT + _NO_MAT)
    args = (*a, *b, _act(act), *kept, *_mat(dx, "dx", out, bf))
    keep, ws, ws_bytes = _workspace(workspace, _lib.tide_linear_grad_input_workspace(rows, inner, outer, *a, *b), stream)
    _check(_lib.tide_linear_grad_input(rows, inner, outer, *args, ws, ws_bytes, _stream(stream)))


def tide_linear_grad_weight(dy, x, dw, db=None, act=TIDE_ACT_NONE, workspace=None, stream=None):
    """dw = dy^T X, db = column sums of dy; X is x, or f(values) of a Checkpoint8 x."""
    rows, outer = _shape2(dy, "dy")
    bf = torch.bfloat16
    a = _mat(dy, "dy", (rows, outer), bf)
    if isinstance(x, Checkpoint8):
        inner = x.shape[1]
        plain, kept = _NO_MAT, _ckpt(x, "x", (rows, inner))
    else:
        inner = _shape2(x, "x")[1]
        plain, kept = _mat(x, "x", (rows, inner), bf), _NO_MAT + _NO_MAT
    args = (*a, *plain, *kept, _act(act), *_mat(dw, "dw", (outer, inner), bf), _optv(db, "db", outer, bf))
    keep, ws, ws_bytes = _workspace(workspace, _lib.tide_linear_grad_weight_workspace(rows, inner, outer, *a, *plain),
                                    stream)
    _check(_lib.tide_linear_grad_weight(rows, inner, outer, *args, ws, ws_bytes, _stream(stream)))
