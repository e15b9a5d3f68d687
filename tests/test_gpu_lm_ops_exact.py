"""The operators at the ends of a training step on inputs whose results are exact or known in closed form, so that one
element left out, counted twice or written from a list that is not complete shows."""

import math

import pytest
import torch

import fsdp_layout_aware_gb300 as tide
from test_gpu_lm_ops import BF, DEV, FP, check_log_probs, gen, logits, put, randn, tokens

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- embedding

def all_zero_bits(x):
    return not x.contiguous().view(torch.uint8).any()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("scale", [-1.5, math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("lead,extra", [(0, 0), (1, 0), (3, 5)])
@pytest.mark.parametrize("n,vocab,cols", [(40, 300, 64), (40, 300, 61), (900, 2000, 64), (900, 2000, 61), (3000, 40, 24)])
def test_padding_is_zeros_whatever_the_scale(n, vocab, cols, lead, extra, scale, dtype):
    """Rows that no token stands for are +0 on rows of any alignment, for few tokens and many."""
    ids = tokens(n, vocab, n).to(DEV)
    here = (ids >= 0) & (ids < vocab)
    w, _ = put(randn((vocab, cols), dtype, 1), lead, extra)
    out, _ = put(torch.full((n, cols), 9.0, dtype=dtype), lead, extra)
    tide.tide_embedding(ids, w, out, scale=scale)
    assert all_zero_bits(out[~here]) and not all_zero_bits(out[here])
    dw, _ = put(torch.full((vocab, cols), 9.0, dtype=dtype), lead, extra)
    ids = torch.where(ids == vocab // 2, 0, ids)
    tide.tide_embedding_backward(ids, put(randn((n, cols), dtype, 2), lead, extra)[0], dw, scale=scale)
    named = torch.zeros(vocab, dtype=torch.bool, device=DEV)
    named[ids[(ids >= 0) & (ids < vocab)]] = True
    assert not named.all() and all_zero_bits(dw[~named]) and not all_zero_bits(dw[named])


def runs_of(tile, n, vocab, seed):
    """n ids whose runs, sorted, are of one place up to more than 512 tiles, begin anywhere in a tile, and leave rows out;
    in any order."""
    lengths = [1, tile - 1, tile, tile + 1, 2, 2 * tile - 1, 2 * tile, 3, 2 * tile + 1, 3 * tile + 5, 1, 10 * tile + 1, 17 * tile]
    if n > 520 * tile + 7:
        lengths.append(520 * tile + 7)
    ids, at = [], 0
    while at < n:
        length = min(lengths[len(ids) % len(lengths)], n - at)
        ids.append(torch.full((length,), 2 * len(ids) % vocab))  # beyond vocab / 2 runs: the same ids again
        at += length
    return torch.cat(ids)[torch.randperm(n, generator=gen(seed))]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("lead,extra", [(0, 0), (3, 5)])
@pytest.mark.parametrize("n,cols,tile", [(20011, 8, 8), (20011, 2056, 16), (20011, 4104, 32), (20011, 8200, 64), (400000, 16, 8),
                                         (400000, 104, 16), (400000, 208, 32), (400000, 408, 64), (513, 40, 8), (700, 33, 8)])
def test_embedding_gradient_adds_every_row_once(n, cols, tile, lead, extra, dtype):
    """Small whole numbers, whose sums fp32 holds exactly in any order, by tiles of each size on a GPU of 152 SMs."""
    vocab = 4001
    ids = runs_of(tile, n, vocab, n + cols).to(DEV)
    row, col = torch.arange(n, device=DEV)[:, None], torch.arange(cols, device=DEV)
    value = ((row * 7 + col * 3) % 11 - 4).to(dtype)  # not 0 on average: one row more or less shows
    dy, _ = put(value, lead, extra)
    dw, _ = put(torch.full((vocab, cols), 9.0, dtype=dtype), (lead * 3) % 7, extra)
    tide.tide_embedding_backward(ids.int() if lead else ids, dy, dw)
    want = torch.zeros(vocab, cols, dtype=torch.float64, device=DEV).index_add_(0, ids, value.double())
    assert want.abs().max() < 1 << 24
    assert torch.equal(dw, want.to(dtype))
    old = (torch.arange(vocab, device=DEV) % 5 - 2).to(dtype)[:, None].expand(vocab, cols)
    dw.copy_(old)
    tide.tide_embedding_backward(ids, dy, dw, scale=-2.0, accumulate=True)
    assert torch.equal(dw, (old.double() - 2 * want).to(dtype))


# ---------------------------------------------------------------- alternatives

# Rows and vocabularies at which 32, 128, 256 and 512 threads share a row with alternatives, and a cluster of blocks.
SHARED = [(3000, 1000), (600, 4000), (300, 4000), (64, 4096), (400, 13000), (400, 20000), (200, 32000), (64, 20000), (2, 131072)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("rows,vocab", SHARED)
def test_alternatives_of_few_tokens_every_time(rows, vocab, dtype):
    """Fewer tokens than alternatives are left, none are, or all are alike: the list is filled up in the tokens' order,
    the same in each of many calls."""
    top = 20
    x = torch.full((rows, vocab), -math.inf)
    want = torch.arange(top).repeat(rows, 1)
    left = torch.arange(rows) % 7  # of them: 0 none, 6 all alike
    for n in range(1, 6):
        at = torch.tensor([vocab - 1, vocab // 2, 40, vocab // 3, 7 * vocab // 8][:n])
        some = left == n
        x[some[:, None] & torch.zeros(vocab, dtype=torch.bool).index_fill(0, at, True)] = 3.0
        first = torch.sort(at).values
        rest = torch.tensor([t for t in range(64) if t not in at.tolist()])[:top - n]
        want[some] = torch.cat([first, rest])
    x[left == 6] = 0.5
    count = torch.where(left == 6, vocab, left).double()
    logp = torch.where(torch.arange(top) < count[:, None], -torch.log(count)[:, None], -math.inf)
    x, want, logp = x.to(dtype).to(DEV), want.to(DEV), logp.to(DEV)
    values, names = torch.empty(rows, top, device=DEV), torch.empty(rows, top, dtype=torch.int32, device=DEV)
    wrong = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(200 if rows * vocab < 1 << 22 else 60):
        values.fill_(7.0), names.fill_(-7)
        tide.tide_log_probs(x, top=(values, names))
        wrong += (names != want).sum()
        # ln of a whole number below 2^18: exact sum, ln to 2 steps, the difference from 0 exact.
        far = (values.double() - logp).abs() > 4 * 2.0 ** -24 * 13
        wrong += (torch.where(logp.isinf(), values != logp.float(), far)).sum()
    assert wrong.item() == 0


# ---------------------------------------------------------------- log probabilities

@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("lead", [0, 1, 3])
@pytest.mark.parametrize("top", [0, 3])
@pytest.mark.parametrize("rows,vocab", [(2000, 1000), (300, 4003), (64, 4096), (400, 13001), (400, 20000), (200, 32005), (64, 20000),
                                        (37, 131077), (2, 131072), (1, 500009)])
def test_every_logit_counts_once(rows, vocab, top, lead, dtype):
    """Rows of equal logits, a few of them masked: the sum is their number, which fp32 holds, and lse is its logarithm."""
    x = torch.full((rows, vocab), 1.5, dtype=dtype, device=DEV)
    hole = torch.arange(rows, device=DEV)
    at = torch.stack([(hole * 7919) % vocab, vocab - 1 - hole % 40, (hole * 8) % vocab, (hole * 4096 + 4095) % vocab], 1)
    for r in range(4):  # rows of no hole, one, two, and four
        some = hole % 4 == r
        x[some] = x[some].scatter(1, at[some][:, :r if r < 3 else 4], -math.inf)
    x, _ = put(x, lead, lead)
    count = (x == 1.5).sum(1).double()
    parts, (lse, entropy) = torch.empty(rows, 2, device=DEV), (torch.empty(rows, device=DEV) for _ in range(2))
    best = (torch.empty(rows, top, device=DEV), torch.empty(rows, top, dtype=torch.int32, device=DEV)) if top else None
    tide.tide_log_probs(x, lse=lse, lse_parts=parts, entropy=entropy, top=best)
    alone = torch.empty(rows, device=DEV)
    tide.tide_log_probs(x, lse=alone)
    # ln of a number below 2^19 to one step and a half, 2^-20 each; lse is rounded once more.
    log_count = torch.log(count)
    off = 1.5 * 2.0 ** -20
    assert bool((parts[:, 0] == 1.5).all())
    assert ((parts[:, 1].double() - log_count).abs() <= off).all()
    assert ((entropy.double() - log_count).abs() <= off).all()  # no logit is away from the largest
    for v in (lse, alone):
        assert ((v.double() - 1.5 - log_count).abs() <= off + 2.0 ** -21).all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("rows,vocab", SHARED)
def test_rows_without_a_token_are_exact(rows, vocab, dtype):
    x = torch.full((rows, vocab), -math.inf, dtype=dtype, device=DEV)
    x[1::2] = 0.0
    t = torch.tensor([-1, -1, vocab, 5, 3, vocab + 7], device=DEV).repeat(rows)[:rows]
    logp, lse, entropy, parts = *(torch.full((rows,), 9.0, device=DEV) for _ in range(3)), torch.full((rows, 2), 9.0, device=DEV)
    tide.tide_log_probs(x, t, logp, lse=lse, entropy=entropy, lse_parts=parts)
    outside = (t < 0) | (t >= vocab)
    assert bool((logp[outside] == 0).all())
    assert bool((logp[::2][~outside[::2]] == -math.inf).all()) and bool((lse[::2] == -math.inf).all())
    assert bool((entropy[::2] == 0).all()) and bool((parts[::2] == -math.inf).all())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("scale", [2.0 ** -120, 2.0 ** -100, 2.0 ** -64, 0.25])
@pytest.mark.parametrize("vocab", [9, 4999, 30000])
def test_logits_further_apart_than_fp32_reaches(vocab, scale, dtype):
    """logp and top_logp of a logit that lies more than fp32's range below the largest, at a scale that brings it back."""
    big = torch.finfo(dtype).max
    x = logits(3, vocab, dtype, 1)
    x[0, 3], x[0, 5] = big, -big
    x[1] = -big
    x[1, vocab - 1] = big / 2
    x[2, 1:] = -big
    check_log_probs(x, torch.tensor([5, 0, 2]), scale, min(vocab, 9))


# ---------------------------------------------------------------- the gradient

@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("parts", [False, True])
@pytest.mark.parametrize("vocab,lead", [(64, 0), (64, 1), (4999, 0)])
@pytest.mark.parametrize("given", [math.nan, math.inf, -math.inf])
def test_rows_without_a_token_have_no_gradient(given, vocab, lead, parts, dtype):
    """Whatever comes back for their entropy (0) and log probability (-inf); nor does a target outside take dlogp in."""
    rows = 6
    x = logits(rows, vocab, dtype, 1)
    x[[0, 3]] = -math.inf
    x, _ = put(x, lead, 0)
    t = torch.tensor([2, 5, vocab, -1, 7, 1], device=DEV)
    g, h = randn((rows,), FP, 2).to(DEV), randn((rows,), FP, 3).to(DEV)
    logp, lse, entropy = (torch.empty(rows, device=DEV) for _ in range(3))
    two = torch.empty(rows, 2, device=DEV)
    tide.tide_log_probs(x, t, logp, lse=lse, entropy=entropy, lse_parts=two)
    source = dict(lse=None, lse_parts=two) if parts else dict(lse=lse)

    def grad(g, h):
        d = torch.full((rows, vocab), 9.0, dtype=dtype, device=DEV)
        tide.tide_log_probs_backward(x, dlogits=d, targets=t, dlogp=g, entropy=entropy, dentropy=h, **source)
        return d

    want = grad(g, h)
    assert want.isfinite().all() and (want[[0, 3]] == 0).all()
    odd_g, odd_h = g.clone(), h.clone()
    odd_g[[0, 2, 3]] = given  # rows without a token, or with a target outside
    odd_h[[0, 3]] = given
    assert torch.equal(grad(odd_g, odd_h), want)
