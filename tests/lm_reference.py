"""The operators at the ends of a training step in 64 bits on the CPU, written
from their formulas (include/tide_lm_ops.h), and the tolerances the GPU tests use.

Inputs are bf16 or fp32 values held exactly in fp64, so a reference value's own
error is far below any tolerance here.  A rounding to a type is off by at most half a
step, eps / 2 of the value.
"""

import math

import torch

U = 2.0 ** -24  # half a step of fp32


def half(dtype):
    return torch.finfo(dtype).eps / 2


def embedding(ids, weight, scale):
    """(values, tolerance): one product in fp32, one rounding."""
    vocab = weight[0].shape[0] if isinstance(weight, tuple) else weight.shape[0]
    ids = ids.long()
    here = (ids >= 0) & (ids < vocab)
    out = torch.zeros(len(ids), weight.shape[1], dtype=torch.float64)
    out[here] = weight.double()[ids[here]] * scale
    return out, (half(weight.dtype) + U) * out.abs()


def embedding_grad(ids, dy, vocab, scale, old=None):
    """(values, tolerance): n additions in fp32 are off by n U of the magnitudes added, whatever their order."""
    ids = ids.long()
    here = (ids >= 0) & (ids < vocab)
    cols = dy.shape[1]
    total, size, count = (torch.zeros(vocab, w, dtype=torch.float64) for w in (cols, cols, 1))
    total.index_add_(0, ids[here], dy.double()[here])
    size.index_add_(0, ids[here], dy.double()[here].abs())
    count.index_add_(0, ids[here], torch.ones(int(here.sum()), 1, dtype=torch.float64))
    out = total * scale if old is None else old.double() + total * scale
    return out, half(dy.dtype) * out.abs() + (count + 3) * U * size * abs(scale) + U * out.abs()


def log_probs(logits, targets, scale, top):
    """A dict of values and one of tolerances."""
    rows, vocab = logits.shape
    x = logits.double()
    z = x * scale
    bad = (x.isnan() | (x == math.inf)).any(1)
    m = torch.where(x.isnan(), -math.inf, x).amax(1) if vocab else torch.full((rows,), -math.inf, dtype=torch.float64)
    empty = (m == -math.inf) & ~bad
    lone = torch.where(m.isfinite(), m, 0.0)
    d = (x - lone[:, None]) * scale
    e = torch.exp(d)
    s = e.sum(1)
    ed = torch.where(e > 0, e * d, 0.0).sum(1)
    log_s = torch.log(s)
    t = targets.long()
    here = (t >= 0) & (t < vocab)
    zt = x.gather(1, t.clamp(0, max(0, vocab - 1))[:, None])[:, 0] if vocab else torch.zeros(rows, dtype=torch.float64)
    nan = torch.tensor(math.nan, dtype=torch.float64)
    ninf = torch.tensor(-math.inf, dtype=torch.float64)

    def settle(v, at_empty):
        return torch.where(bad, nan, torch.where(empty, at_empty, v))

    want = {"lse": settle(lone * scale + log_s, ninf), "entropy": settle(log_s - ed / s, torch.zeros((), dtype=torch.float64)),
            "logp": torch.where(here, settle((zt - lone) * scale - log_s, ninf), 0.0)}
    # Tolerances.  A term's exponent is off by 4 roundings (the difference, scale * log2 e twice, the product), its power by
    # 4 U (the approximate instruction's 2^-22); a thread adds at most `each` terms and its sum is rescaled, at 6 U, once
    # for 8 of them at most, by exponents that add up to the row's range (beyond 150 a term is nothing); 16 more joins.
    each = 8.0 * -(-vocab // 256)
    fin = torch.where(x.isfinite(), x, lone[:, None])
    span = torch.clamp((fin.amax(1) - fin.amin(1)) * scale if vocab else torch.zeros(rows), max=150.0)
    rel = U * (each + 6 * (each / 8 + 16) + 4 * span + 32)
    log_tol = rel + 4 * U * log_s.abs()
    tol = {"lse": log_tol + 3 * U * want["lse"].abs() + 2 * U * (lone * scale).abs(),
           "entropy": rel * (2 + (ed / s).abs()) + 8 * U * (log_s.abs() + (ed / s).abs()),
           "logp": log_tol + 4 * U * (((zt - lone) * scale).abs() + want["logp"].abs())}
    if top:
        v = torch.where(x.isnan(), -math.inf, x)
        order = torch.sort(v, dim=1, descending=True, stable=True).indices[:, :top]
        want["top_tokens"] = order
        zk = v.gather(1, order)
        lp = (zk - lone[:, None]) * scale - log_s[:, None]
        want["top_logp"] = torch.where(bad[:, None], nan, torch.where(empty[:, None], ninf, lp))
        tol["top_logp"] = log_tol[:, None] + 4 * U * (((zk - lone[:, None]) * scale).abs() + lp.abs())
    return want, tol


def log_probs_grad(logits, lse, targets, dlogp, entropy, dentropy, scale, parts=None):
    """(values, tolerance), from the lse (or its parts) and entropy given."""
    rows, vocab = logits.shape
    x, peak, rest = logits.double(), 0.0, lse.double() if parts is None else parts[:, 1].double()
    empty = rest == -math.inf
    if parts is not None:
        peak = torch.where(empty, 0.0, parts[:, 0].double())[:, None]
    d = (x - peak) * scale - torch.where(empty, math.inf, rest)[:, None]
    p = torch.exp(d)
    far = torch.clamp(d, min=-200.0)
    g = torch.zeros(rows, dtype=torch.float64)
    onehot = torch.zeros(rows, vocab, dtype=torch.float64)
    if targets is not None:
        t = targets.long()
        here = (t >= 0) & (t < vocab)
        g = torch.where(here & ~empty, dlogp.double(), 0.0)
        onehot[torch.arange(rows)[here], t[here]] = 1.0
    h = dentropy.double() if dentropy is not None else torch.zeros(rows, dtype=torch.float64)
    hh = entropy.double() if entropy is not None else torch.zeros(rows, dtype=torch.float64)
    inner = g[:, None] + torch.where(p > 0, h[:, None] * (far + hh[:, None]), 0.0)
    want = scale * (g[:, None] * onehot - p * inner)
    # p: three roundings of its exponent and 8 U; the factor: a few roundings of its parts.
    size = p * (g.abs()[:, None] + h.abs()[:, None] * (far.abs() + hh.abs()[:, None])) * scale
    tol = size * U * (4 * far.abs() + 16) + 4 * U * scale * g.abs()[:, None] * onehot + half(logits.dtype) * want.abs()
    return want, tol + 1e-36  # what the exponential flushes


def norm(tensors):
    """(value, relative tolerance): 18 additions in fp32 to a chunk's sum, fp64 beyond, halved by the root; one rounding."""
    total = sum(float(t.double().square().sum()) for t in tensors)
    return math.sqrt(total), 12 * U


def clip(x, norm, max_norm, eps):
    """(values, tolerance) for the fp32 norm given."""
    q = max_norm / (norm + eps) if norm + eps > 0 else math.inf
    by = q if q < 1 else math.nan if math.isnan(norm) else 1.0
    want = x.double() * by
    return want, (half(x.dtype) + (4 * U if by != 1.0 else 0)) * want.abs() + 1e-44


def check(got, want, tol, what):
    got = got.detach().double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: NaNs differ"
    inf = want.isinf()
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    fine = want.isfinite()
    over = ((got - want).abs() - torch.nan_to_num(tol, nan=0.0))[fine]  # of an empty row: exact
    if over.numel() and not over.max() <= 0:
        at = int(over.argmax())
        raise AssertionError(f"{what}: {float(over.max())} over the tolerance at the {at}th of {over.numel()}: "
                             f"{float(got[fine][at])} for {float(want[fine][at])}")
