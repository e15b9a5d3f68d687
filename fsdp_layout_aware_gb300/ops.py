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

from .tide import TideError, _check, _lib
from .tide import _stream as _stream_of

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
        "tide_linear_grad_weight_workspace": (_i64, 3 * [_i64] + 2 * _MAT + [_i32]),
        "tide_linear_grad_weight": (_i32, 3 * [_i64] + 4 * _MAT + [_i32] + _MAT + [_vp, _vp, _i64, _vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(_lib, name)
        fn.restype = res
        fn.argtypes = args


_declare()


# The current stream's handle without building a Stream object (a microsecond
# of a call), where this torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None and _raw_stream is not None:
        return _raw_stream(_device())
    return _stream_of(stream)


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
_NO_CKPT = (None, 0, None, 0)
_device = torch.cuda.current_device


def _wrong(t, name, shape, dtype, dev):
    """What is wrong with a tensor that _mat or _vec did not take."""
    if t.dtype is not dtype:
        _refuse(f"{name} is {t.dtype}, not {dtype}")
    if tuple(t.shape) != shape:
        _refuse(f"{name} has shape {tuple(t.shape)}, not {shape}")
    if not t.is_cuda:
        _refuse(f"{name} is not on the GPU")
    if t.get_device() != dev:
        _refuse(f"{name} is on device {t.get_device()}, which is not the current one", 7)
    _refuse(f"{name}: the last axis is not contiguous")


def _mat(t, name, rows, cols, dtype, dev):
    """(address, row stride) of a (rows, cols) tensor on device dev."""
    if t.dtype is dtype and t.get_device() == dev and t.shape == (rows, cols):
        ld, step = t.stride()
        if step == 1 or cols <= 1:
            return t.data_ptr(), ld
    _wrong(t, name, (rows, cols), dtype, dev)


def _vec(t, name, n, dtype, dev):
    """Address of an (n,) tensor on device dev."""
    if t.dtype is dtype and t.get_device() == dev and t.shape == (n,) and (n <= 1 or t.stride(0) == 1):
        return t.data_ptr()
    _wrong(t, name, (n,), dtype, dev)


def _ckpt(c, name, rows, cols, dev):
    """codes and scales of a checkpoint: (address, stride, address, stride)."""
    u8 = torch.uint8
    return (*_mat(c.codes, name + ".codes", rows, cols, u8, dev),
            *_mat(c.scales, name + ".scales", rows, -(-cols // TIDE_CKPT_BLOCK), u8, dev))


def _opt(t, name, rows, cols, dtype, dev):
    return _NO_MAT if t is None else _mat(t, name, rows, cols, dtype, dev)


def _optv(t, name, n, dtype, dev):
    return None if t is None else _vec(t, name, n, dtype, dev)


def _plain_or_kept(t, name, rows, cols, dtype, dev):
    """Arguments of a matrix given plain, as a Checkpoint8, or not at all: (address, stride) and _ckpt's four."""
    if t is None:
        return _NO_MAT + _NO_CKPT
    if isinstance(t, Checkpoint8):
        return _NO_MAT + _ckpt(t, name, rows, cols, dev)
    return _mat(t, name, rows, cols, dtype, dev) + _NO_CKPT


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


def _torch_stream(stream, dev):
    """The torch stream of a stream argument."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = _stream_of(stream)
    # 0 and 1 name the legacy default stream, which no external stream can.
    return torch.cuda.ExternalStream(handle, dev) if handle > 1 else torch.cuda.default_stream(dev)


def _workspace(given, need, stream, dev):
    """(tensor that keeps it alive, address, bytes)."""
    if given is not None:
        if given.get_device() != dev or not given.is_contiguous():
            _refuse("workspace is not a contiguous tensor on the current device")
        return given, given.data_ptr(), given.numel() * given.element_size()
    if need == 0:
        return None, None, 0
    if stream is None:
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        # A block of the call's own stream.  One of the current stream's may have been freed while kernels queued there
        # still use it, and nothing would make the given stream wait for those.
        with torch.cuda.stream(_torch_stream(stream, dev)):
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
    return ws, ws.data_ptr(), need


def tide_ops_check():
    """Synchronise and raise TideError(TIDE_ERR_TIMEOUT) if an operator's kernel gave up a wait on this device since this
    thread's last check of it."""
    _check(_lib.tide_ops_check())


def tide_ops_set_option(option, value):
    _check(_lib.tide_ops_set_option(option, value))


def tide_checkpoint_store(x, ckpt, stream=None):
    """Keep x (rows, cols; bf16 or fp32) in ckpt (a Checkpoint8 of that shape)."""
    dev = _device()
    rows, cols = _shape2(x, "x")
    _check(_lib.tide_checkpoint_store(rows, cols, _dtype(x, "x"), *_mat(x, "x", rows, cols, x.dtype, dev),
                                      *_ckpt(ckpt, "ckpt", rows, cols, dev), _stream(stream)))


def tide_checkpoint_load(ckpt, out, act=TIDE_ACT_NONE, grad=None, stream=None):
    """out = f(values), or grad * f'(values) when grad is given (out may be grad)."""
    dev = _device()
    rows, cols = ckpt.shape
    t = out.dtype
    _check(_lib.tide_checkpoint_load(rows, cols, *_ckpt(ckpt, "ckpt", rows, cols, dev), _act(act), _dtype(out, "out"),
                                     *_opt(grad, "grad", rows, cols, t, dev), *_mat(out, "out", rows, cols, t, dev),
                                     _stream(stream)))


def tide_rms_norm(x, weight, eps, y=None, residual=None, h=None, rstd=None, y8=None, stream=None):
    """h = x + residual; y (and y8, a Checkpoint8) = h * rstd * weight, rstd = (mean(h^2) + eps)^-1/2 per row."""
    dev = _device()
    rows, cols = _shape2(x, "x")
    t = x.dtype
    _check(_lib.tide_rms_norm(rows, cols, _dtype(x, "x"), *_mat(x, "x", rows, cols, t, dev),
                              *_opt(residual, "residual", rows, cols, t, dev), _vec(weight, "weight", cols, t, dev), eps,
                              *_opt(h, "h", rows, cols, t, dev), *_opt(y, "y", rows, cols, t, dev),
                              _optv(rstd, "rstd", rows, torch.float32, dev),
                              *(_NO_CKPT if y8 is None else _ckpt(y8, "y8", rows, cols, dev)), _stream(stream)))


def tide_rms_norm_backward(dy, h, weight, rstd, dx=None, dweight=None, dres=None, workspace=None, stream=None):
    """Gradients of tide_rms_norm: dx (of x and of residual, dres added) and dweight; h may be a Checkpoint8."""
    dev = _device()
    rows, cols = _shape2(dy, "dy")
    t = dy.dtype
    args = (rows, cols, _dtype(dy, "dy"), *_mat(dy, "dy", rows, cols, t, dev),
            *_plain_or_kept(h, "h", rows, cols, t, dev), _vec(weight, "weight", cols, t, dev),
            _vec(rstd, "rstd", rows, torch.float32, dev), *_opt(dres, "dres", rows, cols, t, dev),
            *_opt(dx, "dx", rows, cols, t, dev), _optv(dweight, "dweight", cols, t, dev))
    need = 0 if dweight is None else _lib.tide_rms_norm_backward_workspace(rows, cols)
    keep, ws, ws_bytes = _workspace(workspace, need, stream, dev)
    _check(_lib.tide_rms_norm_backward(*args, ws, ws_bytes, _stream(stream)))


def tide_linear(x, w, y, bias=None, act=TIDE_ACT_NONE, residual=None, z=None, workspace=None, stream=None):
    """y = f(x w^T + bias) + residual; z (bf16, or a Checkpoint8) keeps x w^T + bias for the backward pass."""
    dev = _device()
    rows, inner = _shape2(x, "x")
    outer = _shape2(w, "w")[0]
    bf = torch.bfloat16
    size = (rows, inner, outer)
    ab = (*_mat(x, "x", rows, inner, bf, dev), *_mat(w, "w", outer, inner, bf, dev))
    args = (_optv(bias, "bias", outer, bf, dev), _act(act), *_opt(residual, "residual", rows, outer, bf, dev),
            *_mat(y, "y", rows, outer, bf, dev), *_plain_or_kept(z, "z", rows, outer, bf, dev))
    keep, ws, ws_bytes = _workspace(workspace, _lib.tide_linear_workspace(*size, *ab), stream, dev)
    _check(_lib.tide_linear(*size, *ab, *args, ws, ws_bytes, _stream(stream)))


def tide_linear_grad_input(dy, w, dx, act=TIDE_ACT_NONE, z=None, workspace=None, stream=None):
    """dx = (dy w) * f'(z): z (bf16 or Checkpoint8) is the pre-activation behind this layer's input."""
    dev = _device()
    rows, outer = _shape2(dy, "dy")
    inner = _shape2(w, "w")[1]
    bf = torch.bfloat16
    size = (rows, inner, outer)
    ab = (*_mat(dy, "dy", rows, outer, bf, dev), *_mat(w, "w", outer, inner, bf, dev))
    args = (_act(act), *_plain_or_kept(z, "z", rows, inner, bf, dev), *_mat(dx, "dx", rows, inner, bf, dev))
    keep, ws, ws_bytes = _workspace(workspace, _lib.tide_linear_grad_input_workspace(*size, *ab), stream, dev)
    _check(_lib.tide_linear_grad_input(*size, *ab, *args, ws, ws_bytes, _stream(stream)))


def tide_linear_grad_weight(dy, x, dw, db=None, act=TIDE_ACT_NONE, workspace=None, stream=None):
    """dw = dy^T X, db = column sums of dy; X is x, or f(values) of a Checkpoint8 x."""
    dev = _device()
    rows, outer = _shape2(dy, "dy")
    inner = x.shape[1] if isinstance(x, Checkpoint8) else _shape2(x, "x")[1]
    bf = torch.bfloat16
    size = (rows, inner, outer)
    a, kept = _mat(dy, "dy", rows, outer, bf, dev), _plain_or_kept(x, "x", rows, inner, bf, dev)
    args = (_act(act), *_mat(dw, "dw", outer, inner, bf, dev), _optv(db, "db", outer, bf, dev))
    need = _lib.tide_linear_grad_weight_workspace(*size, *a, *kept[:2], db is not None)
    keep, ws, ws_bytes = _workspace(workspace, need, stream, dev)
    _check(_lib.tide_linear_grad_weight(*size, *a, *kept, *args, ws, ws_bytes, _stream(stream)))
