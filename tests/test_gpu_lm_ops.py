"""The operators at the ends of a training step on the GPU against the 64-bit reference."""

import math

import pytest
import torch

import fsdp_layout_aware_gb300 as tide
import lm_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float32
LAYOUTS = [(0, 0), (8, 16), (1, 0), (3, 5)]  # (lead, extra) elements: aligned, aligned with a stride, two odd ones


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=gen(seed), dtype=torch.float64) * scale).to(dtype)


def put(x, lead=0, extra=0):
    """x on the GPU inside a larger buffer of NaN: `lead` elements before it, rows `extra` longer."""
    rows, cols = x.shape
    buf = torch.full((lead + rows * (cols + extra),), float("nan"), dtype=x.dtype, device=DEV)
    v = buf[lead:].view(rows, cols + extra)[:, :cols]
    v.copy_(x)
    return v, buf


def untouched(view, buf):
    """Nothing outside the view was written."""
    mask = torch.ones(buf.shape, dtype=torch.bool, device=DEV)
    rows, cols = view.shape
    if rows and cols:
        torch.as_strided(mask, (rows, cols), (view.stride(0) if rows > 1 else cols, 1), view.storage_offset()).fill_(False)
    return bool(buf[mask].isnan().all())


def tokens(n, vocab, seed, index=torch.int64, hot=0.0, outside=0.2):
    """Ids, some of them one id, some outside the vocabulary in every way the type allows."""
    g = gen(seed)
    t = torch.randint(0, max(1, vocab), (n,), generator=g)
    t = torch.where(torch.rand(n, generator=g) < hot, vocab // 2, t)
    info = torch.iinfo(index)
    odd = torch.tensor([-1, vocab, info.min, info.max, vocab + 1, -vocab - 1] + ([1 << 32, (1 << 32) + 1] if index is torch.int64 else []))
    t = torch.where(torch.rand(n, generator=g) < outside, odd[torch.randint(0, len(odd), (n,), generator=g)], t)
    return t.to(index)


# ---------------------------------------------------------------- embedding

@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("lead,extra", LAYOUTS)
@pytest.mark.parametrize("n,vocab,cols", [(1, 1, 1), (3, 7, 9), (5, 40, 64), (33, 300, 200), (2, 5, 4095), (700, 50, 1024),
                                          (1, 9, 8192)])
def test_embedding(n, vocab, cols, lead, extra, dtype):
    index = torch.int32 if (n + lead) % 2 else torch.int64
    w, ids = randn((vocab, cols), dtype, n + cols), tokens(n, vocab, n, index)
    dw, _ = put(w, lead, extra)
    out, buf = put(torch.zeros(n, cols, dtype=dtype), (lead * 3) % 7, extra)
    tide.tide_embedding(ids.to(DEV), dw, out, scale=1.75)
    R.check(out, *R.embedding(ids, w, 1.75), "out")
    assert untouched(out, buf)


def test_embedding_keeps_what_a_row_holds():
    w = torch.tensor([[math.inf, -math.inf, math.nan, -0.0, 1e-40, 3.4e38, 0.0, 1.0]])
    out = torch.empty(2, 8, device=DEV)
    tide.tide_embedding(torch.tensor([0, 1], device=DEV), w.to(DEV), out, scale=1.0)
    assert torch.equal(out[0].cpu().nan_to_num(nan=7.0), w[0].nan_to_num(nan=7.0))
    assert (out[1] == 0).all()  # not in the vocabulary: whatever the table holds


def test_embedding_of_no_vocabulary_is_zero():
    out = torch.full((3, 16), 5.0, device=DEV)
    tide.tide_embedding(torch.tensor([0, 1, -1], device=DEV), torch.empty(0, 16, device=DEV), out)
    assert (out == 0).all()


GRADS = [  # tokens, vocab, columns, share of one id
    (0, 5, 24, 0.0), (512, 700, 48, 0.0), (512, 30, 1040, 0.9), (513, 30, 1040, 0.9), (511, 129, 2047, 0.1), (0, 70000, 33, 0.0), (300, 70000, 40, 0.3), (512, 1030, 2047, 0.9), (3, 40000, 65, 0.0), (64, 20000, 130, 0.5), (65, 20000, 130, 0.5), (1, 1, 1, 0.0), (1, 300, 16, 0.0), (7, 3, 33, 0.0), (64, 9, 64, 0.5), (65, 64, 40, 1.0),
    (257, 100, 100, 1.0), (300, 33, 130, 0.7), (1000, 70000, 24, 0.1), (4096, 300, 56, 0.3), (4097, 257, 72, 0.9),
    (9000, 65536, 17, 0.2), (3000, 300000, 9, 0.1), (400000, 5000, 8, 0.3), (20011, 1000, 31, 0.05), (5000, 40, 1032, 0.6), (4099, 2, 2056, 0.4)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("lead,extra", LAYOUTS)
@pytest.mark.parametrize("n,vocab,cols,hot", GRADS)
def test_embedding_gradient(n, vocab, cols, hot, lead, extra, dtype):
    index = torch.int64 if (n + lead) % 2 else torch.int32
    dy, ids = randn((n, cols), dtype, n + cols), tokens(n, vocab, n, index, hot)
    ddy, _ = put(dy, lead, extra)
    dw, buf = put(torch.full((vocab, cols), 3.0, dtype=dtype), (lead * 3) % 7, extra)
    tide.tide_embedding_backward(ids.to(DEV), ddy, dw, scale=0.5)
    R.check(dw, *R.embedding_grad(ids, dy, vocab, 0.5), "dweight")
    assert untouched(dw, buf)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n,vocab,cols,hot", [(1, 3, 8, 0.0), (300, 50, 96, 0.5), (6000, 4000, 33, 0.3)])
def test_embedding_gradient_added(n, vocab, cols, hot, dtype):
    dy, ids = randn((n, cols), dtype, 1), tokens(n, vocab, 2, torch.int64, hot)
    old = randn((vocab, cols), dtype, 3)
    old[0] = math.nan
    ids = torch.where(ids == 0, 1 if vocab > 1 else -1, ids)
    dw = old.to(DEV)
    tide.tide_embedding_backward(ids.to(DEV), dy.to(DEV), dw, scale=-2.0, accumulate=True)
    want, tol = R.embedding_grad(ids, dy, vocab, -2.0, old)
    R.check(dw, want, tol, "dweight")
    named = torch.zeros(vocab, dtype=torch.bool)
    named[ids[(ids >= 0) & (ids < vocab)]] = True
    assert torch.equal(dw.cpu()[~named].view(torch.uint8), old[~named].view(torch.uint8))  # bit for bit


def test_embedding_gradient_takes_no_part_of_rows_outside():
    """NaN in the gradient of a padded place stays there."""
    ids = torch.tensor([2, -1, 2, 5, 0])
    dy = torch.ones(5, 16)
    dy[1] = math.nan
    dy[3] = math.inf
    dw = torch.empty(5, 16, device=DEV)
    tide.tide_embedding_backward(ids.to(DEV), dy.to(DEV), dw)
    assert torch.equal(dw.cpu()[:, 0], torch.tensor([1.0, 0.0, 2.0, 0.0, 0.0]))


@pytest.mark.parametrize("n,vocab,hot,outside", [(5000, 100, 0.5, 0.1), (40000, 50000, 0.3, 0.0), (3000, 10, 0.0, 1.0)])
def test_embedding_gradient_is_the_same_every_time(n, vocab, hot, outside):
    dy = randn((n, 264), BF, 1).to(DEV)
    ids = tokens(n, vocab, 2, torch.int64, hot, outside).to(DEV)
    first = torch.empty(vocab, 264, dtype=BF, device=DEV)
    tide.tide_embedding_backward(ids, dy, first)
    for _ in range(5):
        again = torch.full_like(first, 9.0)
        tide.tide_embedding_backward(ids, dy, again)
        assert torch.equal(first, again)
    if outside == 1.0:
        assert (first == 0).all()


def test_embedding_gradient_sums_of_thousands():
    """Sums whose parts cancel, against a tolerance of the magnitudes added."""
    n = 30000
    dy = torch.cat([torch.full((n // 2, 8), 1000.0), torch.full((n // 2, 8), -1000.0), torch.full((1, 8), 0.5)])
    ids = torch.zeros(n + 1, dtype=torch.int32)
    dw = torch.empty(1, 8, device=DEV)
    tide.tide_embedding_backward(ids.to(DEV), dy.to(DEV), dw)
    R.check(dw, *R.embedding_grad(ids, dy, 1, 1.0), "dweight")


# ---------------------------------------------------------------- log probabilities

def logits(rows, vocab, dtype, seed, spread=3.0):
    return randn((rows, vocab), dtype, seed, spread)


def run_log_probs(x, t, scale=1.0, top=0, lead=0, extra=0):
    rows = x.shape[0]
    dx, _ = put(x, lead, extra)
    out = {k: torch.full((rows,), 77.0, device=DEV) for k in ("logp", "lse", "entropy")}
    best = None
    if top:
        values, vbuf = put(torch.zeros(rows, top), 1, 2)
        names = torch.full((rows, top + 1), -7, dtype=torch.int32, device=DEV)
        best = (values, names[:, :top])
    tide.tide_log_probs(dx, t.to(DEV), out["logp"], lse=out["lse"], entropy=out["entropy"], top=best, scale=scale)
    if top:
        assert untouched(values, vbuf) and (names[:, top] == -7).all()
        out["top_logp"], out["top_tokens"] = best
    return out


def check_log_probs(x, t, scale=1.0, top=0, lead=0, extra=0):
    got = run_log_probs(x, t, scale, top, lead, extra)
    want, tol = R.log_probs(x, t, scale, top)
    for k in want:
        if k == "top_tokens":
            assert torch.equal(got[k].cpu().long(), want[k]), k
        else:
            R.check(got[k], want[k], tol[k], k)
    return got


ROWS = [(1, 1), (2, 5), (9, 8), (3, 33), (17, 257), (5, 1000), (3, 1024), (4, 1033), (2, 4999), (3, 8192), (2, 8200),
        (1, 20000), (300, 9001), (1, 131072), (2, 50001)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("lead,extra", LAYOUTS)
@pytest.mark.parametrize("rows,vocab", ROWS)
def test_log_probs(rows, vocab, lead, extra, dtype):
    x, t = logits(rows, vocab, dtype, rows + vocab), tokens(rows, vocab, vocab, torch.int32 if lead else torch.int64)
    check_log_probs(x, t, 1.0 if extra else 0.7, min(vocab, 20) if lead != 3 else 0, lead, extra)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("vocab", [32, 100, 2000, 30000])
@pytest.mark.parametrize("top", [1, 2, 31, 32])
def test_alternatives_with_ties(vocab, top, dtype):
    """Few different values, so that nearly every one of them ties; the lowest tokens win."""
    x = torch.randint(-2, 3, (6, vocab), generator=gen(vocab + top)).to(dtype)
    x[1] = 0.0
    x[2] = torch.where(torch.arange(vocab) % 2 == 0, 0.0, -0.0)
    x[3] = torch.sort(x[3].float()).values.to(dtype)
    x[4] = torch.sort(randn((vocab,), dtype, 5).float(), descending=True).values.to(dtype)
    x[5] = torch.sort(randn((vocab,), dtype, 6).float()).values.to(dtype)
    check_log_probs(x, tokens(6, vocab, 3), 1.0, top)


@pytest.mark.parametrize("top", [5, 32])
@pytest.mark.parametrize("vocab", [64, 8000, 40000])
def test_alternatives_that_one_thread_has_met(vocab, top):
    """The largest logits at places that lie a thread's step apart, whichever it is."""
    x = logits(8, vocab, FP, 1)
    for r, step in enumerate((1, 8, 256, 1024, 2048, 4096, 16384, 32768)):
        at = (torch.arange(40) * step + r) % vocab
        x[r, at] = 50.0 + torch.rand(40, generator=gen(r))
    check_log_probs(x, tokens(8, vocab, 2), 1.0, top)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("rows,vocab", [(12, 40), (12, 3000), (12, 20000), (700, 9000)])
def test_masked_rows(rows, vocab, dtype):
    x = logits(rows, vocab, dtype, 3)
    low = torch.finfo(dtype).min
    x[0] = -math.inf                       # nothing left
    x[1] = -math.inf
    x[1, vocab - 1] = 2.0                  # one token
    x[2] = low                             # all at the type's lowest value: all alike
    x[3, ::2] = low
    x[4, ::3] = -math.inf
    x[5] = -math.inf
    x[5, :3] = low
    x[6] = torch.finfo(dtype).max          # all at the highest
    x[7, 5] = torch.finfo(dtype).max
    x[8] = 0.0
    x[9] = torch.linspace(-300, 300, vocab).to(dtype)
    x[10, :] = -math.inf
    x[10, vocab // 2:vocab // 2 + 2] = -1e30
    x[11] *= 1e-30
    t = tokens(rows, vocab, 4)
    t[:3] = torch.tensor([1, vocab - 1, 0])
    t[5] = vocab - 1  # a token of probability 0
    check_log_probs(x, t, 1.0, min(vocab, 32))
    check_log_probs(x, t, 0.5, 3, 1, 1)


@pytest.mark.parametrize("vocab", [40, 3000, 20000])
def test_rows_with_nan_and_infinity(vocab):
    x = logits(6, vocab, FP, 3)
    x[0, 7] = math.nan
    x[1, 7] = math.inf
    x[2, vocab - 1] = math.inf
    x[2, 0] = math.nan
    x[3] = math.nan
    x[4, :] = -math.inf
    x[4, 3] = math.nan
    t = torch.tensor([1, 7, -1, 0, 1, 2])
    got = run_log_probs(x, t, 1.0, 4)
    want, tol = R.log_probs(x, t, 1.0, 4)
    for k in ("lse", "entropy", "logp", "top_logp"):
        R.check(got[k], want[k], tol[k], k)
    assert torch.equal(got["top_tokens"].cpu().long(), want["top_tokens"])


def test_parts_of_empty_rows_and_their_gradient():
    x = torch.full((3, 50), -math.inf)
    x[1] = -1e9
    parts = torch.empty(3, 2, device=DEV)
    tide.tide_log_probs(x.to(DEV), lse_parts=parts)
    assert (parts[[0, 2]] == -math.inf).all()
    t, g, d = torch.tensor([1, 2, 3], device=DEV), torch.ones(3, device=DEV), torch.full((3, 50), 9.0, device=DEV)
    tide.tide_log_probs_backward(x.to(DEV), None, d, targets=t, dlogp=g, lse_parts=parts)
    assert (d[[0, 2]] == 0).all() and abs(d[1, 2].item() - 0.98) < 1e-6 and abs(d[1, 0].item() + 0.02) < 1e-6


def test_log_probs_of_no_vocabulary():
    got = run_log_probs(torch.empty(3, 0), torch.tensor([0, -1, 5]))
    assert (got["logp"] == 0).all() and (got["lse"] == -math.inf).all() and (got["entropy"] == 0).all()


def test_log_probs_outputs_one_by_one():
    """Which outputs are asked for may change the order of the sums, not what they are within their tolerances."""
    x, t = logits(5, 3000, BF, 1), tokens(5, 3000, 1)
    dx, dt = x.to(DEV), t.to(DEV)
    want, tol = R.log_probs(x, t, 1.0, 6)
    one = {k: torch.empty(5, device=DEV) for k in ("logp", "lse", "entropy")}
    best = torch.empty(5, 6, device=DEV), torch.empty(5, 6, dtype=torch.int32, device=DEV)
    tide.tide_log_probs(dx, dt, one["logp"])
    tide.tide_log_probs(dx, lse=one["lse"])
    tide.tide_log_probs(dx, entropy=one["entropy"])
    tide.tide_log_probs(dx, top=best)
    for k, v in one.items():
        R.check(v, want[k], tol[k], k)
    R.check(best[0], want["top_logp"], tol["top_logp"], "top_logp")
    assert torch.equal(best[1].cpu().long(), want["top_tokens"])


def grad_inputs(rows, vocab, seed, scale):
    t = tokens(rows, vocab, seed)
    x = logits(rows, vocab, torch.float64, seed)
    return t, x, randn((rows,), FP, seed + 1), randn((rows,), FP, seed + 2)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("lead,extra", LAYOUTS)
@pytest.mark.parametrize("rows,vocab", [(1, 1), (2, 5), (9, 8), (3, 33), (17, 264), (4, 1033), (2, 4999), (3, 8192), (60, 3001),
                                        (1, 50001)])
def test_log_probs_gradient(rows, vocab, lead, extra, dtype):
    scale = 1.0 if extra else 1.25
    t, x, g, h = grad_inputs(rows, vocab, rows * vocab, scale)
    x = x.to(dtype)
    if vocab > 4:
        x[:, vocab // 3] = -math.inf
    w, _ = R.log_probs(x, t, scale, 0)
    lse, entropy = w["lse"].float(), w["entropy"].float()
    for out_lead in {lead, (lead + 3) % 5}:
        for parts in ("g", "h", "gh"):
            dx, _ = put(x, lead, extra)
            out, buf = put(torch.zeros(rows, vocab, dtype=dtype), out_lead, extra)
            given_t = dict(targets=t, dlogp=g) if "g" in parts else {}
            given_h = dict(entropy=entropy, dentropy=h) if "h" in parts else {}
            tide.tide_log_probs_backward(dx, lse.to(DEV), out, scale=scale,
                                         **{k: v.to(DEV) for k, v in {**given_t, **given_h}.items()})
            want, tol = R.log_probs_grad(x, lse, given_t.get("targets"), given_t.get("dlogp"), given_h.get("entropy"),
                                         given_h.get("dentropy"), scale)
            R.check(out, want, tol, parts)
            assert untouched(out, buf)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("vocab", [64, 4999])
def test_log_probs_gradient_in_place_and_of_masked_rows(vocab, dtype):
    x = logits(6, vocab, dtype, 2)
    x[0] = -math.inf
    x[1] = torch.finfo(dtype).min
    x[2, ::2] = torch.finfo(dtype).min
    x[3] = -math.inf
    x[3, 5] = 1.0
    x[4, 0] = math.nan
    t = torch.tensor([1, 2, 3, 5, 1, -1])
    g, h = randn((6,), FP, 3), randn((6,), FP, 4)
    got = run_log_probs(x, t)
    lse, entropy = got["lse"].cpu(), got["entropy"].cpu()
    d = x.to(DEV)
    tide.tide_log_probs_backward(d, lse.to(DEV), d, targets=t.to(DEV), dlogp=g.to(DEV), entropy=entropy.to(DEV),
                                 dentropy=h.to(DEV))
    want, tol = R.log_probs_grad(x, lse, t, g, entropy, h, 1.0)
    keep = [0, 1, 2, 3, 5]
    R.check(d[keep], want[keep], tol[keep], "in place")
    assert (d[0] == 0).all() and d[4].isnan().all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("scale", [1.0, 0.7])
@pytest.mark.parametrize("vocab", [40, 4999])
def test_log_probs_gradient_of_rows_far_from_zero(vocab, scale, dtype):
    """Rows whose logits are all a mask's value, or lie about one: lse alone has no bits left for the sum."""
    at = [torch.finfo(dtype).min, -1e9, -3e4, 1e6, 3e4, torch.finfo(dtype).max, -1e30, 0.0]
    x = torch.stack([torch.full((vocab,), v) for v in at]).to(dtype)
    x[2:5] += torch.randint(-2, 3, (3, vocab), generator=gen(1)).to(dtype)
    rows = len(at)
    t = torch.arange(rows) % vocab
    parts, entropy = torch.empty(rows, 2, device=DEV), torch.empty(rows, device=DEV)
    tide.tide_log_probs(x.to(DEV), lse_parts=parts, entropy=entropy, scale=scale)
    scale = float(torch.tensor(scale))
    # The largest logit is exact; the sum's logarithm is known as in the reference's tolerance, here for 160 terms a
    # thread, a range of 4 and a logarithm of 9: 460 U.
    peak = x.double().amax(1)
    assert torch.equal(parts[:, 0].cpu().double(), peak)
    rest = torch.logsumexp((x.double() - peak[:, None]) * scale, 1)
    assert ((parts[:, 1].cpu().double() - rest).abs() <= 2.0 ** -15).all()
    g, h = randn((rows,), FP, 3), randn((rows,), FP, 4)
    d = torch.empty(rows, vocab, dtype=dtype, device=DEV)
    tide.tide_log_probs_backward(x.to(DEV), None, d, targets=t.to(DEV), dlogp=g.to(DEV), entropy=entropy,
                                 dentropy=h.to(DEV), scale=scale, lse_parts=parts)
    want, tol = R.log_probs_grad(x, None, t, g, entropy.cpu(), h, scale, parts.cpu())
    R.check(d, want, tol, "dlogits")
    p = torch.exp((x.double() - peak[:, None]) * scale - rest[:, None])
    alone = torch.empty_like(d)
    tide.tide_log_probs_backward(x.to(DEV), None, alone, targets=t.to(DEV), dlogp=g.to(DEV), scale=scale, lse_parts=parts)
    onehot = torch.nn.functional.one_hot(t, vocab).double()
    exact = scale * g.double()[:, None] * (onehot - p)
    # p by that, and its own 32 roundings at most.
    tol = R.half(dtype) * exact.abs() + scale * g.double().abs()[:, None] * (2.0 ** -14 * p + 4 * R.U * onehot)
    assert ((alone.double().cpu() - exact).abs() <= tol).all()


def test_log_probs_gradient_is_the_differences():
    """Central differences of the forward call in fp32: off by the values' own error over the step, and by its square."""
    x = logits(3, 70, FP, 5, 1.0)
    t = torch.tensor([4, 69, 11])
    g, h = torch.tensor([1.0, -0.5, 2.0]), torch.tensor([0.5, 1.0, -1.0])
    w, _ = R.log_probs(x, t, 1.0, 0)
    out = torch.empty(3, 70, device=DEV)
    tide.tide_log_probs_backward(x.to(DEV), w["lse"].float().to(DEV), out, targets=t.to(DEV), dlogp=g.to(DEV),
                                 entropy=w["entropy"].float().to(DEV), dentropy=h.to(DEV))
    step = 2.0 ** -6
    cols = torch.arange(70)
    up, down = x.repeat_interleave(70, 0), x.repeat_interleave(70, 0)
    at = (torch.arange(210), cols.repeat(3))
    up[at] += step
    down[at] -= step
    width = up[at].double() - down[at].double()
    values = []
    for y in (up, down):
        got = run_log_probs(y, t.repeat_interleave(70))
        values.append(got["logp"].double().cpu() * g.repeat_interleave(70) + got["entropy"].double().cpu() *
                      h.repeat_interleave(70))
    num = ((values[0] - values[1]) / width).view(3, 70)
    # Third derivatives of both are below 8 in magnitude, so the differences are off by 3 * 8 * step^2 / 6 = 1e-3; two fp32
    # values of about 6, off by 2^-20, over 2 step: 6e-5 more.
    assert (num - out.double().cpu()).abs().max() < 1.1e-3


# ---------------------------------------------------------------- norm and clipping

def lists(sizes, dtypes, seed, lead=0, scale=1.0):
    """(host tensors, GPU tensors at odd places of one buffer a type, the buffers)."""
    host, dev, bufs = [], [], []
    for i, n in enumerate(sizes):
        x = randn((n,), dtypes[i % len(dtypes)], seed + i, scale)
        at = (lead + 3 * i) % 11 if lead else 0
        buf = torch.full((at + n + 5,), float("nan"), dtype=x.dtype, device=DEV)
        buf[at:at + n] = x.to(DEV)
        host.append(x)
        dev.append(buf[at:at + n])
        bufs.append(buf)
    return host, dev, bufs


SIZES = [[], [0], [1], [7], [8], [0, 5, 0], [16384], [16385, 3], [8192 * 9 + 1], list(range(1, 70)),
         [100003, 1, 65536, 31, 0, 250000], [5] * 2500, [700000, 12, 300001], [3000000]]


@pytest.mark.parametrize("lead", [0, 1, 2])
@pytest.mark.parametrize("dtypes", [(BF,), (FP,), (BF, FP)])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s, default=0)}")
def test_norm_and_clip(sizes, dtypes, lead):
    host, dev, _ = lists(sizes, dtypes, 7, lead)
    norm = torch.full((1,), -1.0, device=DEV)
    tide.tide_grad_norm(dev, norm)
    want, tol = R.norm(host)
    assert abs(norm.item() - want) <= tol * want
    n = norm.item()
    for most in (0.5 * n, 2 * n + 1):
        _, outs, bufs = lists(sizes, dtypes, 7, (lead + 2) % 3)
        tide.tide_grad_clip(tide.TensorList(dev), norm, most, eps=1e-3, out=outs)
        for x, y in zip(host, outs):
            R.check(y, *R.clip(x, n, float(torch.tensor(most)), float(torch.tensor(1e-3))), "clipped")
        for y, b in zip(outs, bufs):
            assert int(b.isnan().sum()) == b.numel() - y.numel()
    tide.tide_grad_clip(dev, norm, 0.25 * n)  # in place
    for x, y in zip(host, dev):
        R.check(y, *R.clip(x, n, float(torch.tensor(0.25 * n)), 1e-6), "in place")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n", [5, 20000, 3000001])
@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-20, 1e-16, 1e16, 1e19, 1e30, 1e35])
def test_norm_of_any_magnitude(scale, n, dtype):
    x = randn((n,), dtype, 3, scale)
    norm = torch.empty(1, device=DEV)
    tide.tide_grad_norm([x.to(DEV)], norm)
    want, tol = R.norm([x])
    assert abs(norm.item() - want) <= tol * want + 2.0 ** -149


def test_norm_of_mixed_magnitudes():
    """Single values far above and below all others, zeros between."""
    for at, big in ((0, 1e25), (31, 3e38), (40000, 1e-25)):
        x = torch.zeros(50000)
        x[::7] = 1e-30
        x[at] = big
        norm = torch.empty(1, device=DEV)
        tide.tide_grad_norm([x.to(DEV), torch.full((9,), 1e-20, dtype=BF, device=DEV)], norm)
        want, tol = R.norm([x, torch.full((9,), 1e-20, dtype=BF)])
        assert abs(norm.item() - want) <= tol * want


@pytest.mark.parametrize("size", [100, 500000])
def test_norm_and_clip_of_infinity_and_nan(size):
    norm = torch.empty(1, device=DEV)
    x = torch.ones(size, device=DEV)
    x[size // 2] = math.inf
    tide.tide_grad_norm([x], norm)
    assert norm.item() == math.inf
    y = torch.empty_like(x)
    tide.tide_grad_clip([x], norm, 1.0, out=[y])
    assert y[size // 2].isnan() and (y.nan_to_num(nan=0.0) == 0).all()
    tide.tide_grad_clip([x], norm, math.inf, out=[y])  # nothing to clip to
    assert torch.equal(x, y)
    x[1] = math.nan
    tide.tide_grad_norm([x], norm)
    assert math.isnan(norm.item())
    tide.tide_grad_clip([x], norm, 1.0)
    assert x.isnan().all()


def test_norm_of_norms():
    host, dev, _ = lists([1000, 77, 300000], (BF, FP), 1)
    parts = torch.empty(3, device=DEV)
    for i, x in enumerate(dev):
        tide.tide_grad_norm([x], parts[i:i + 1])
    norm = torch.empty(1, device=DEV)
    tide.tide_grad_norm([parts], norm)
    want, tol = R.norm(host)
    assert abs(norm.item() - want) <= 2 * tol * want


@pytest.mark.parametrize("sizes", [
    [5] * 24, [5] * 25, [5] * 64, [5] * 65, [8192] * 32, [8192] * 33, [8192 * 62], [8192 * 65],
    [0] * 300 + [9000] * 3 + [0] * 1400 + [1], [0] * 40, [8192 * 40, 0, 3] + [1] * 30,
])
@pytest.mark.parametrize("lead", [0, 1])
def test_norm_of_lists_of_few_chunks(sizes, lead):
    """Lists at the sizes where one launch, or blocks of another size, take their place."""
    host, dev, _ = lists(sizes, (FP,), 11, lead)
    norm = torch.full((1,), -1.0, device=DEV)
    tide.tide_grad_norm(dev, norm)
    want, tol = R.norm(host)
    assert abs(norm.item() - want) <= tol * want


def test_norm_is_the_same_every_time():
    _, dev, _ = lists([700000, 12, 300001, 5000000], (FP, BF), 1, 1)
    x = tide.TensorList(dev)
    norms = [torch.empty(1, device=DEV) for _ in range(6)]
    for n in norms:
        tide.tide_grad_norm(x, n)
    assert all(torch.equal(n, norms[0]) for n in norms)


# ---------------------------------------------------------------- refusals that need a GPU

def test_the_binding_refuses():
    ids, x = torch.zeros(4, dtype=torch.int64, device=DEV), torch.zeros(4, 16, device=DEV)
    row, one = torch.zeros(4, device=DEV), torch.zeros(1, device=DEV)
    bad = [
        lambda: tide.tide_embedding(ids.float(), x, x.clone()),
        lambda: tide.tide_embedding(ids.cpu(), x, x.clone()),
        lambda: tide.tide_embedding(ids, x, x.bfloat16()),
        lambda: tide.tide_embedding(ids, x, x[:3]),
        lambda: tide.tide_embedding(ids[::2], x, x[:2]),
        lambda: tide.tide_embedding(ids, x.half(), x.half()),
        lambda: tide.tide_embedding(ids, x.t(), x.t()),
        lambda: tide.tide_embedding_backward(ids, x, x.clone(), workspace=torch.empty(16, dtype=torch.uint8)),
        lambda: tide.tide_embedding_backward(torch.zeros(600, dtype=torch.int32, device=DEV), torch.zeros(600, 16, device=DEV), x.clone(),
                                             workspace=torch.empty(16, dtype=torch.uint8, device=DEV)),
        lambda: tide.tide_embedding_backward(ids, x[:3], x.clone()),
        lambda: tide.tide_log_probs(x, ids, None),
        lambda: tide.tide_log_probs(x, ids, row.double()),
        lambda: tide.tide_log_probs(x, ids, row, top=(x[:, :3], ids[:, None].expand(4, 3))),
        lambda: tide.tide_log_probs(x, ids, row, top=(torch.zeros(4, 40, device=DEV), torch.zeros(4, 40, dtype=torch.int32, device=DEV))),
        lambda: tide.tide_log_probs(x, ids, row, scale=0.0),
        lambda: tide.tide_log_probs_backward(x, row, x.clone(), targets=ids),
        lambda: tide.tide_log_probs_backward(x, row[:3], x.clone()),
        lambda: tide.tide_log_probs_backward(x, None, x.clone()),
        lambda: tide.tide_log_probs_backward(x, None, x.clone(), lse_parts=row),
        lambda: tide.tide_log_probs(x, lse_parts=x[:, :2]),
        lambda: tide.tide_grad_norm([x, x.half()], one),
        lambda: tide.tide_grad_norm([x.t()], one),
        lambda: tide.tide_grad_norm([x], row),
        lambda: tide.tide_grad_clip([x], one, -1.0),
        lambda: tide.tide_grad_clip([x, x], one, 1.0),
        lambda: tide.tide_grad_clip([x, x[1:]], one, 1.0),
        lambda: tide.tide_grad_clip([x, x], one, 1.0, out=[x.clone()] * 2),
        lambda: tide.tide_grad_clip([x], one, 1.0, out=[x, x]),
        lambda: tide.tide_grad_clip([x], one, 1.0, out=[x[:2]]),
        lambda: tide.tide_grad_clip([x], one, 1.0, out=[x.bfloat16()]),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(tide.TideError):
            f()
            print("not refused:", i)
