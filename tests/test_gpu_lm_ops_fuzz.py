"""Seeded random calls of the operators at the ends of a training step against the 64-bit reference."""

import math
import random

import pytest
import torch

import fsdp_layout_aware_gb300 as tide
import lm_reference as R
from test_gpu_lm_ops import DEV, check_log_probs, put, randn, tokens, untouched

pytestmark = pytest.mark.gpu
TYPES = (torch.bfloat16, torch.float32)


def size(r, lo, hi):
    n = int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))
    return n // 8 * 8 if n >= 8 and r.random() < 0.4 else n


@pytest.mark.parametrize("seed", range(40))
def test_embedding_and_its_gradient(seed):
    r = random.Random(seed)
    n, vocab, cols = size(r, 1, 9000), size(r, 1, 3000), size(r, 1, 600)
    dtype, index = r.choice(TYPES), r.choice([torch.int32, torch.int64])
    ids = tokens(n, vocab, seed, index, r.choice([0.0, 0.3, 0.95]), r.choice([0.0, 0.5]))
    lead, extra, scale = r.choice([0, 0, 8, 1, 3, 6]), r.choice([0, 0, 8, 5]), r.choice([1.0, -0.75])
    w = randn((vocab, cols), dtype, seed)
    out, buf = put(torch.zeros(n, cols, dtype=dtype), r.choice([0, lead, 2]), extra)
    tide.tide_embedding(ids.to(DEV), put(w, lead, extra)[0], out, scale=scale)
    R.check(out, *R.embedding(ids, w, scale), "out")
    assert untouched(out, buf)
    dy = randn((n, cols), dtype, seed + 1)
    add = r.random() < 0.3
    old = randn((vocab, cols), dtype, seed + 2)
    dw, buf = put(old, r.choice([0, lead, 5]), extra)
    tide.tide_embedding_backward(ids.to(DEV), put(dy, lead, extra)[0], dw, scale=scale, accumulate=add)
    R.check(dw, *R.embedding_grad(ids, dy, vocab, scale, old if add else None), "dweight")
    assert untouched(dw, buf)


@pytest.mark.parametrize("seed", range(60))
def test_log_probs_and_their_gradient(seed):
    r = random.Random(seed)
    vocab = size(r, 1, 40000)
    rows = min(size(r, 1, 400), max(1, 400000 // vocab))
    dtype, scale = r.choice(TYPES), r.choice([1.0, 0.5, 1.5])
    x = randn((rows, vocab), dtype, seed, r.choice([0.01, 1.0, 4.0, 100.0]))
    kind = r.choice(["", "", "masked", "coarse", "far"])
    if kind == "masked":
        x[torch.rand(rows, vocab, generator=torch.Generator().manual_seed(seed)) < r.choice([0.5, 0.99])] = -math.inf
    elif kind == "coarse":
        x = x.float().round().to(dtype)
    elif kind == "far":
        x = (x.float() + r.choice([-1e4, 1e3])).to(dtype)
    t = tokens(rows, vocab, seed + 1)
    lead, extra = r.choice([0, 0, 8, 1, 3, 6]), r.choice([0, 0, 8, 5])
    check_log_probs(x, t, scale, min(vocab, r.choice([0, 1, 7, 32])), lead, extra)
    want, _ = R.log_probs(x, t, scale, 0)
    lse, entropy, g, h = want["lse"].float(), want["entropy"].float(), randn((rows,), torch.float32, 5), randn((rows,), torch.float32, 6)
    out, buf = put(torch.zeros(rows, vocab, dtype=dtype), r.choice([0, lead, 7]), extra)
    tide.tide_log_probs_backward(put(x, lead, extra)[0], lse.to(DEV), out, targets=t.to(DEV), dlogp=g.to(DEV),
                                 entropy=entropy.to(DEV), dentropy=h.to(DEV), scale=scale)
    R.check(out, *R.log_probs_grad(x, lse, t, g, entropy, h, scale), "dlogits")
    assert untouched(out, buf)


@pytest.mark.parametrize("seed", range(20))
def test_norm_and_clip(seed):
    r = random.Random(seed)
    sizes = [0 if r.random() < 0.1 else size(r, 1, 60000) for _ in range(size(r, 1, 150))]
    xs, dev = [], []
    for i, n in enumerate(sizes):
        x = randn((n,), r.choice(TYPES), seed * 1000 + i, r.choice([1e-3, 1.0]))
        at = r.randrange(0, 9)
        buf = torch.zeros(at + n, dtype=x.dtype, device=DEV)
        buf[at:] = x.to(DEV)
        xs.append(x)
        dev.append(buf[at:])
    norm = torch.empty(1, device=DEV)
    tide.tide_grad_norm(dev, norm)
    want, tol = R.norm(xs)
    assert abs(norm.item() - want) <= tol * want
    n = norm.item()
    tide.tide_grad_clip(dev, norm, 0.3)
    for x, y in zip(xs, dev):
        R.check(y, *R.clip(x, n, float(torch.tensor(0.3)), float(torch.tensor(1e-6))), "clipped")
