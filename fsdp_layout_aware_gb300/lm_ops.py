"""ctypes binding of libtide's operators at the two ends of a language model's
training step (include/tide_lm_ops.h); the same manner as ops.py.

    tide_embedding, tide_embedding_backward
    tide_log_probs, tide_log_probs_backward
    tide_grad_norm, tide_grad_clip, TensorList
"""

import ctypes

import torch

from .ops import (_DTYPES, _MAT, _NO_MAT, _device, _dtype, _i32, _i64, _lib, _mat, _opt, _optv, _refuse, _shape2, _stream,
                  _vec, _vp, _workspace)
from .tide import _check

TIDE_I32, TIDE_I64 = 0, 1
_INDEX = {torch.int32: TIDE_I32, torch.int64: TIDE_I64}
_f32 = ctypes.c_float


def _declare():
    lists = [_i32, _vp, _vp, _vp]  # count, addresses, numbers of elements, types
    sig = {
        "tide_embedding": (_i32, 3 * [_i64] + [_i32, _vp, _i32] + _MAT + [_f32] + _MAT + [_vp]),
        "tide_embedding_backward_workspace": (_i64, 3 * [_i64]),
        "tide_embedding_backward": (_i32, 3 * [_i64] + [_i32, _vp, _i32] + _MAT + [_f32] + _MAT + [_i32, _vp, _i64, _vp]),
        "tide_log_probs": (_i32, [_i64, _i64, _i32] + _MAT + [_f32, _i32] + 5 * [_vp] + [_i32] + 2 * _MAT + [_vp]),
        "tide_log_probs_backward": (_i32, [_i64, _i64, _i32] + _MAT + [_f32, _vp, _vp, _i32] + 4 * [_vp] +
                                    _MAT + [_vp]),
        "tide_grad_norm_workspace": (_i64, [_i32, _vp, _vp]),
        "tide_grad_norm": (_i32, lists + [_vp, _vp, _i64, _vp]),
        "tide_grad_clip": (_i32, [_i32, _vp, _vp, _vp, _vp, _vp, _f32, _f32, _vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(_lib, name)
        fn.restype = res
        fn.argtypes = args


_declare()


def _ids(t, name, n, dev):
    """(type, address) of n token ids."""
    code = _INDEX.get(t.dtype)
    if code is None:
        _refuse(f"{name} is {t.dtype}; int32 and int64 are taken")
    return code, _vec(t, name, n, t.dtype, dev)


def _shape1(t, name):
    if t.dim() != 1:
        _refuse(f"{name} has {t.dim()} axes, not 1")
    return t.shape[0]


def tide_embedding(ids, weight, out, scale=1.0, stream=None):
    """out[t] = scale * weight[ids[t]]; an id outside the vocabulary gives zeros."""
    dev = _device()
    tokens, (vocab, cols) = _shape1(ids, "ids"), _shape2(weight, "weight")
    t = weight.dtype
    _check(_lib.tide_embedding(tokens, vocab, cols, *_ids(ids, "ids", tokens, dev), _dtype(weight, "weight"),
                               *_mat(weight, "weight", vocab, cols, t, dev), scale, *_mat(out, "out", tokens, cols, t, dev),
                               _stream(stream)))


def tide_embedding_backward(ids, dy, dweight, scale=1.0, accumulate=False, workspace=None, stream=None):
    """dweight[v] = scale * sum of dy[t] over the t with ids[t] == v (added to what it holds with accumulate)."""
    dev = _device()
    tokens, (vocab, cols) = _shape1(ids, "ids"), _shape2(dweight, "dweight")
    t = dweight.dtype
    args = (tokens, vocab, cols, *_ids(ids, "ids", tokens, dev), _dtype(dweight, "dweight"),
            *_mat(dy, "dy", tokens, cols, t, dev), scale, *_mat(dweight, "dweight", vocab, cols, t, dev), bool(accumulate))
    need = _lib.tide_embedding_backward_workspace(tokens, vocab, cols)
    keep, ws, ws_bytes = _workspace(workspace, need, stream, dev)
    _check(_lib.tide_embedding_backward(*args, ws, ws_bytes, _stream(stream)))


def _parts(t, rows, dev):
    """Address of lse's parts, a contiguous (rows, 2) tensor or None."""
    if t is None:
        return None
    at, ld = _mat(t, "lse_parts", rows, 2, torch.float32, dev)
    if rows > 1 and ld != 2:
        _refuse("lse_parts is not contiguous")
    return at


def tide_log_probs(logits, targets=None, logp=None, lse=None, entropy=None, top=None, scale=1.0, lse_parts=None, stream=None):
    """For each row of z = scale * logits: logp = log softmax(z)[targets] (0 for a target outside the vocabulary), lse
    (and lse_parts, (rows, 2): the largest logit, and the rest of lse), entropy, and top, a pair (log probabilities, int32
    tokens) of (rows, k) tensors for the k likeliest tokens."""
    dev = _device()
    rows, vocab = _shape2(logits, "logits")
    f32 = torch.float32
    index, at = (0, None) if targets is None else _ids(targets, "targets", rows, dev)
    k, best = 0, _NO_MAT + _NO_MAT
    if top is not None:
        k = _shape2(top[0], "top[0]")[1]
        best = (*_mat(top[0], "top[0]", rows, k, f32, dev), *_mat(top[1], "top[1]", rows, k, torch.int32, dev))
    _check(_lib.tide_log_probs(rows, vocab, _dtype(logits, "logits"), *_mat(logits, "logits", rows, vocab, logits.dtype, dev),
                               scale, index, at, _optv(logp, "logp", rows, f32, dev), _optv(lse, "lse", rows, f32, dev),
                               _parts(lse_parts, rows, dev), _optv(entropy, "entropy", rows, f32, dev), k, *best, _stream(stream)))


def tide_log_probs_backward(logits, lse, dlogits, targets=None, dlogp=None, entropy=None, dentropy=None, scale=1.0,
                            lse_parts=None, stream=None):
    """dlogits of tide_log_probs' logp (dlogp, with targets) and entropy (dentropy, with entropy); may be logits.  lse_parts
    takes the place of lse, which may be None then: p is right by it whatever the logits' size."""
    dev = _device()
    rows, vocab = _shape2(logits, "logits")
    t, f32 = logits.dtype, torch.float32
    index, at = (0, None) if targets is None else _ids(targets, "targets", rows, dev)
    _check(_lib.tide_log_probs_backward(rows, vocab, _dtype(logits, "logits"), *_mat(logits, "logits", rows, vocab, t, dev),
                                        scale, _optv(lse, "lse", rows, f32, dev), _parts(lse_parts, rows, dev), index, at,
                                        _optv(dlogp, "dlogp", rows, f32, dev), _optv(entropy, "entropy", rows, f32, dev),
                                        _optv(dentropy, "dentropy", rows, f32, dev),
                                        *_mat(dlogits, "dlogits", rows, vocab, t, dev), _stream(stream)))


class TensorList:
    """Addresses, sizes and types of tensors (bf16 or fp32, contiguous, on one device), read once and passed to many calls.

    The tensors are held, and must stay where they are while the list is in use.
    """

    __slots__ = ("tensors", "count", "device", "addresses", "numels", "dtypes", "room", "_apart")

    def __init__(self, tensors):
        self.tensors = tensors = list(tensors)
        self.count = n = len(tensors)
        self.addresses, self.numels, self.dtypes = (_vp * n)(), (_i64 * n)(), (_i32 * n)()
        self.device = tensors[0].get_device() if n else None
        self.room = {}  # workspace bytes by device
        self._apart = None
        for i, t in enumerate(tensors):
            code = _DTYPES.get(t.dtype)
            if code is None:
                _refuse(f"tensor {i} is {t.dtype}; bfloat16 and float32 are built")
            if not t.is_cuda:
                _refuse(f"tensor {i} is not on the GPU")
            if t.get_device() != self.device:
                _refuse(f"tensor {i} is on another device than tensor 0", 7)
            if not t.is_contiguous():
                _refuse(f"tensor {i} is not contiguous")
            self.addresses[i], self.numels[i], self.dtypes[i] = t.data_ptr(), t.numel(), code

    def __len__(self):
        return self.count

    def apart(self):
        """Whether no two tensors share memory, as outputs must not (tied weights' gradient listed twice, for one)."""
        if self._apart is None:
            spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in self.tensors if t.numel())
            self._apart = all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
        return self._apart


def _list(tensors, dev):
    if not isinstance(tensors, TensorList):
        tensors = TensorList(tensors)
    if tensors.count and tensors.device != dev:
        _refuse(f"the tensors are on device {tensors.device}, which is not the current one", 7)
    return tensors


def tide_grad_norm(tensors, norm, workspace=None, stream=None):
    """norm (one fp32) = the square root of the sum of squares of all tensors (a TensorList, or any iterable)."""
    dev = _device()
    x = _list(tensors, dev)
    out = _vec(norm, "norm", 1, torch.float32, dev)
    need = x.room.get(dev)
    if need is None:
        need = x.room[dev] = _lib.tide_grad_norm_workspace(x.count, x.numels, x.dtypes)
    keep, ws, ws_bytes = _workspace(workspace, need, stream, dev)
    _check(_lib.tide_grad_norm(x.count, x.addresses, x.numels, x.dtypes, out, ws, ws_bytes, _stream(stream)))


def tide_grad_clip(tensors, norm, max_norm, eps=1e-6, out=None, stream=None):
    """out = tensors * min(1, max_norm / (norm + eps)), in place without out."""
    dev = _device()
    x = _list(tensors, dev)
    y = x if out is None else _list(out, dev)
    if y is not x:
        if y.count != x.count:
            _refuse(f"{y.count} outputs for {x.count} tensors")
        if bytes(y.numels) != bytes(x.numels) or bytes(y.dtypes) != bytes(x.dtypes):
            _refuse("an output has another size or type than its tensor")
    if not y.apart():
        _refuse("two of the outputs share memory")
    _check(_lib.tide_grad_clip(x.count, x.addresses, y.addresses, x.numels, x.dtypes,
                               _vec(norm, "norm", 1, torch.float32, dev), max_norm, eps, _stream(stream)))
