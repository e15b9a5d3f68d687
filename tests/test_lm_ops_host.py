"""Host side of the operators at the ends of a training step: the C entry
points' argument checks (no GPU call is reached), the binding's, the header, and the
64-bit reference's own consistency."""

import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

import fsdp_layout_aware_gb300 as tide
import lm_reference as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # an address that is never followed
OK, INVALID, ALIGNMENT, OVERFLOW, UNIMPLEMENTED = 0, 1, 2, 3, 6


def lib():
    tide.tide_embedding  # loads the operators' declarations
    from fsdp_layout_aware_gb300.tide import _lib
    return _lib


def embed(tokens=4, vocab=10, cols=8, index=0, ids=P, dtype=0, w=P, ldw=8, scale=1.0, out=P, ldo=8):
    return lib().tide_embedding(tokens, vocab, cols, index, ids, dtype, w, ldw, scale, out, ldo, None)


def embed_grad(tokens=4, vocab=10, cols=8, index=0, ids=P, dtype=0, dy=P, lddy=8, scale=1.0, dw=P, lddw=8, add=0, ws=P,
               wsb=1 << 20):
    return lib().tide_embedding_backward(tokens, vocab, cols, index, ids, dtype, dy, lddy, scale, dw, lddw, add, ws, wsb,
                                         None)


def probs(rows=4, vocab=40, dtype=0, z=P, ldz=40, scale=1.0, index=0, t=P, logp=P, lse=None, parts=None, h=None, top=0, tl=None,
          ldl=0, tt=None, ldt=0):
    return lib().tide_log_probs(rows, vocab, dtype, z, ldz, scale, index, t, logp, lse, parts, h, top, tl, ldl, tt, ldt, None)


def probs_grad(rows=4, vocab=40, dtype=0, z=P, ldz=40, scale=1.0, lse=P, parts=None, index=0, t=P, dlogp=P, h=None, dh=None, out=P,
               ldo=40):
    return lib().tide_log_probs_backward(rows, vocab, dtype, z, ldz, scale, lse, parts, index, t, dlogp, h, dh, out, ldo, None)


def arrays(addresses, numels, dtypes):
    n = len(addresses)
    return (ctypes.c_void_p * n)(*addresses), (ctypes.c_int64 * n)(*numels), (ctypes.c_int32 * n)(*dtypes)


def norm(count=2, at=(P, P), numels=(8, 8), dtypes=(0, 1), out=P, ws=None, wsb=0, null=False):
    a, n, d = arrays(at, numels, dtypes)
    return lib().tide_grad_norm(count, None if null else a, n, d, out, ws, wsb, None)


def clip(count=2, at=(P, P), outs=(P, P), numels=(8, 8), dtypes=(0, 1), norm=P, most=1.0, eps=0.0, null=False):
    a, n, d = arrays(at, numels, dtypes)
    o, _, _ = arrays(outs, numels, dtypes)
    return lib().tide_grad_clip(count, a, None if null else o, n, d, norm, most, eps, None)


BIG = 1 << 40
CASES = [
    (embed, dict(tokens=-1), INVALID), (embed, dict(vocab=-1), INVALID), (embed, dict(cols=-1), INVALID),
    (embed, dict(index=2), INVALID), (embed, dict(index=-1), INVALID), (embed, dict(dtype=3), INVALID),
    (embed, dict(ids=None), INVALID), (embed, dict(w=None), INVALID), (embed, dict(out=None), INVALID),
    (embed, dict(ldw=7), INVALID), (embed, dict(ldo=7), INVALID), (embed, dict(ids=P + 2), ALIGNMENT),
    (embed, dict(ids=P + 4, index=1), ALIGNMENT), (embed, dict(w=P + 1), ALIGNMENT), (embed, dict(out=P + 1), ALIGNMENT),
    (embed, dict(dtype=1, out=P + 2), ALIGNMENT), (embed, dict(tokens=0), OK), (embed, dict(cols=0), OK),
    (embed, dict(tokens=1 << 31, ldo=8), UNIMPLEMENTED), (embed, dict(vocab=1 << 31), UNIMPLEMENTED),
    (embed, dict(cols=(1 << 24) + 1, ldw=BIG, ldo=BIG), UNIMPLEMENTED), (embed, dict(vocab=1 << 30, ldw=BIG), OVERFLOW),
    (embed_grad, dict(tokens=-1), INVALID), (embed_grad, dict(dy=None), INVALID), (embed_grad, dict(dw=None), INVALID),
    (embed_grad, dict(tokens=1000, ws=None), INVALID), (embed_grad, dict(tokens=1000, wsb=15), INVALID), (embed_grad, dict(ws=P + 8), ALIGNMENT),
    (embed_grad, dict(lddy=7), INVALID), (embed_grad, dict(lddw=7), INVALID), (embed_grad, dict(index=5), INVALID),
    (embed_grad, dict(vocab=0), OK), (embed_grad, dict(cols=0), OK), (embed_grad, dict(tokens=0, add=1), OK),
    (embed_grad, dict(vocab=(1 << 31) - 1), UNIMPLEMENTED), (embed_grad, dict(dw=P + 1), ALIGNMENT),
    (embed_grad, dict(dtype=2), INVALID), (embed_grad, dict(ids=None), INVALID),
    (embed_grad, dict(cols=(1 << 24) + 1, lddy=BIG, lddw=BIG), UNIMPLEMENTED),
    (probs, dict(rows=-1), INVALID), (probs, dict(vocab=-1), INVALID), (probs, dict(dtype=2), INVALID),
    (probs, dict(z=None), INVALID), (probs, dict(ldz=39), INVALID), (probs, dict(z=P + 1), ALIGNMENT),
    (probs, dict(scale=0.0), INVALID), (probs, dict(scale=-1.0), INVALID), (probs, dict(scale=math.inf), INVALID),
    (probs, dict(scale=math.nan), INVALID), (probs, dict(scale=2.0 ** 65), INVALID), (probs, dict(t=None), INVALID), (probs, dict(logp=None), INVALID),
    (probs, dict(index=2), INVALID), (probs, dict(t=P + 2), ALIGNMENT), (probs, dict(lse=P + 2), ALIGNMENT),
    (probs, dict(h=P + 1), ALIGNMENT), (probs, dict(parts=P + 2), ALIGNMENT),
    (probs_grad, dict(parts=P + 1), ALIGNMENT), (probs_grad, dict(lse=None, parts=P, out=None), INVALID), (probs, dict(top=-1), INVALID), (probs, dict(top=33), INVALID),
    (probs, dict(vocab=4, top=5), INVALID), (probs, dict(top=5, tl=P, ldl=4), INVALID),
    (probs, dict(top=5, tt=P, ldt=4), INVALID), (probs, dict(top=5, tt=P + 2, ldt=5), ALIGNMENT),
    (probs, dict(rows=0, t=None), OK), (probs, dict(t=None, logp=None), OK), (probs, dict(t=None, logp=None, top=3), OK),
    (probs, dict(rows=1 << 31), UNIMPLEMENTED), (probs, dict(vocab=(1 << 31) - 8, ldz=1 << 31), UNIMPLEMENTED),
    (probs, dict(rows=1 << 30, ldz=BIG), OVERFLOW),
    (probs_grad, dict(t=None), INVALID), (probs_grad, dict(dlogp=None), INVALID), (probs_grad, dict(h=P), INVALID),
    (probs_grad, dict(dh=P), INVALID), (probs_grad, dict(lse=None), INVALID), (probs_grad, dict(out=None), INVALID),
    (probs_grad, dict(ldo=39), INVALID), (probs_grad, dict(out=P + 1), ALIGNMENT), (probs_grad, dict(scale=0.0), INVALID),
    (probs_grad, dict(rows=0), OK), (probs_grad, dict(vocab=0), OK), (probs_grad, dict(index=9), INVALID),
    (probs_grad, dict(dlogp=P + 2), ALIGNMENT), (probs_grad, dict(h=P, dh=P + 1), ALIGNMENT),
    (norm, dict(count=-1), INVALID), (norm, dict(null=True), INVALID), (norm, dict(out=None), INVALID),
    (norm, dict(out=P + 2), ALIGNMENT), (norm, dict(at=(P, None)), INVALID), (norm, dict(at=(P, P + 2)), ALIGNMENT),
    (norm, dict(at=(P + 1, P)), ALIGNMENT), (norm, dict(numels=(8, -1)), INVALID), (norm, dict(dtypes=(0, 2)), INVALID),
    (norm, dict(numels=(8, (1 << 40) + 1)), UNIMPLEMENTED), (norm, dict(ws=P + 8), ALIGNMENT),
    (clip, dict(count=-1), INVALID), (clip, dict(null=True), INVALID), (clip, dict(norm=None), INVALID),
    (clip, dict(most=-1.0), INVALID), (clip, dict(most=math.nan), INVALID), (clip, dict(eps=-1e-6), INVALID),
    (clip, dict(eps=math.nan), INVALID), (clip, dict(outs=(P, None)), INVALID), (clip, dict(outs=(P, P + 1)), ALIGNMENT),
    (clip, dict(count=0), OK), (clip, dict(norm=P + 1), ALIGNMENT), (clip, dict(dtypes=(-1, 0)), INVALID),
    (clip, dict(numels=(1, -2)), INVALID),
]


@pytest.mark.parametrize("f,args,status", CASES)
def test_arguments_are_checked_on_the_host(f, args, status):
    assert f(**args) == status, lib().tide_last_error()
    if status != OK:
        assert lib().tide_last_error()


def test_every_declared_operator_is_exported_and_bound():
    text = open(os.path.join(ROOT, "include", "tide_lm_ops.h")).read()
    names = set(re.findall(r"^\w+ (tide_\w+)\(", text, re.M))
    assert len(names) == 8
    for n in names:
        assert getattr(lib(), n).argtypes is not None, n


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "tide_lm_ops.h"\nint main(void) { return tide_grad_norm_workspace(0, 0, 0) != 0; }\n')
    libdir = os.path.dirname(tide.LIB_PATH)
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I", os.path.join(ROOT, "include"),
                    str(src), "-L", libdir, "-l:" + os.path.basename(tide.LIB_PATH), "-Wl,-rpath," + libdir, "-o",
                    str(tmp_path / "t")], check=True, capture_output=True, text=True)
    assert subprocess.run([str(tmp_path / "t")], timeout=120).returncode == 0


def test_workspace_queries():
    q = lib().tide_embedding_backward_workspace
    assert q(0, 10, 8) == q(10, 0, 8) == q(10, 10, 0) == q(-1, 10, 8) == 0
    assert q(1, 10, 8) == q(512, 10, 8) == q(512, 1 << 18, 8) == 0  # few tokens, few rows: one launch, nothing kept
    assert q(64, 1 << 21, 8) == 0 and q(65, 1 << 21, 8) >= 4 * 4 * 65 and q(1, 1 << 22, 8) >= 16
    assert q(513, 10, 8) >= 4 * 4 * 513  # four lists of ids
    assert q(100000, 10, 8) >= 4 * 400000 + 100000 // 64 * 32
    assert lib().tide_grad_norm_workspace(0, None, None) == 0
    _, n, d = arrays((P, P), (8, 8), (0, 1))
    assert lib().tide_grad_norm_workspace(2, n, d) == 0  # little: one launch, no partial sums


@pytest.mark.parametrize("make,message", [
    (lambda: tide.TensorList([torch.zeros(3)]), "not on the GPU"),
    (lambda: tide.TensorList([torch.zeros(3, dtype=torch.float16)]), "float16"),
])
def test_a_list_refuses_what_it_cannot_hold(make, message):
    with pytest.raises(tide.TideError, match=message):
        make()


# ---- the reference against itself

def test_reference_gradient_is_the_differences():
    torch.manual_seed(0)
    x = torch.randn(5, 9, dtype=torch.float64) * 2
    x[1, 3] = -math.inf
    t = torch.tensor([3, 4, -1, 8, 0])
    g, h = torch.randn(5, dtype=torch.float64), torch.randn(5, dtype=torch.float64)
    w, _ = R.log_probs(x, t, 0.8, 0)
    want, _ = R.log_probs_grad(x, w["lse"], t, g, w["entropy"], h, 0.8)

    def value(x):
        w, _ = R.log_probs(x, t, 0.8, 0)
        return float((w["logp"] * g).sum() + (w["entropy"] * h).sum())

    d = 1e-6
    for r in range(5):
        for c in range(9):
            if not x[r, c].isfinite():
                assert want[r, c] == 0
                continue
            up, down = x.clone(), x.clone()
            up[r, c] += d
            down[r, c] -= d
            assert abs((value(up) - value(down)) / (2 * d) - float(want[r, c])) < 1e-8


def test_reference_log_probs_agree_with_torch():
    torch.manual_seed(1)
    x = torch.randn(6, 50, dtype=torch.float64) * 3
    x[2, 10:] = -math.inf
    t = torch.randint(0, 10, (6,))
    w, _ = R.log_probs(x, t, 1.3, 4)
    logs = torch.log_softmax(x * 1.3, 1)
    assert torch.allclose(w["logp"], logs.gather(1, t[:, None])[:, 0], atol=1e-13)
    assert torch.allclose(w["entropy"], -torch.special.xlogy(logs.exp(), logs.exp()).sum(1), atol=1e-13)
    assert torch.allclose(w["lse"], torch.logsumexp(x * 1.3, 1), atol=1e-13)
    assert torch.allclose(w["top_logp"], logs.topk(4, 1).values, atol=1e-13)
