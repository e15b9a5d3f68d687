"""Calls of the operators at the ends of a training step as programs make them: on other streams,
from several threads, captured and replayed, and beyond what 31 and 32 bits count."""

import concurrent.futures

import pytest
import torch

import fsdp_layout_aware_gb300 as tide
import lm_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def generator(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def randn(*shape, seed, dtype=BF):
    return torch.randn(*shape, generator=generator(seed), device=DEV).to(dtype)


def some_ids(n, vocab, seed):
    ids = torch.randint(-1, vocab, (n,), generator=generator(seed), device=DEV)
    ids[::3] = vocab // 2
    return ids


# Each: (inputs that may change, outputs, the call on a stream).

def embedding(seed):
    ids, w, out = some_ids(500, 300, seed), randn(300, 264, seed=seed + 1), torch.empty(500, 264, dtype=BF, device=DEV)
    return (ids, w), (out,), lambda stream: tide.tide_embedding(ids, w, out, scale=2.0, stream=stream)


def embedding_gradient(seed):
    """Sorted ids and long runs' parts in the workspace."""
    ids, dy, dw = some_ids(6000, 300, seed), randn(6000, 264, seed=seed + 1), torch.empty(300, 264, dtype=BF, device=DEV)
    return (ids, dy), (dw,), lambda stream: tide.tide_embedding_backward(ids, dy, dw, stream=stream)


def log_probs(seed):
    """A row on a cluster."""
    x, t = randn(3, 60000, seed=seed), some_ids(3, 60000, seed)
    out = [torch.empty(3, device=DEV) for _ in range(3)]
    best = torch.empty(3, 7, device=DEV), torch.empty(3, 7, dtype=torch.int32, device=DEV)
    return (x, t), (*out, *best), lambda stream: tide.tide_log_probs(x, t, out[0], lse=out[1], entropy=out[2], top=best,
                                                                     stream=stream)


def log_probs_gradient(seed):
    x, t, dx = randn(50, 1001, seed=seed), some_ids(50, 1001, seed), torch.empty(50, 1001, dtype=BF, device=DEV)
    lse, g = torch.logsumexp(x.float(), 1), randn(50, seed=seed + 1, dtype=torch.float32)
    return (x, t), (dx,), lambda stream: tide.tide_log_probs_backward(x, lse, dx, targets=t, dlogp=g, stream=stream)


def norm_and_clip(seed):
    """Partial sums in the workspace."""
    xs = [randn(n, seed=seed + n) for n in (3000001, 5, 700000)]
    outs, norm = [torch.empty_like(x) for x in xs], torch.empty(1, device=DEV)

    def run(stream):
        tide.tide_grad_norm(xs, norm, stream=stream)
        tide.tide_grad_clip(xs, norm, 1.0, out=outs, stream=stream)

    return xs, (norm, *outs), run


CALLS = [embedding, embedding_gradient, log_probs, log_probs_gradient, norm_and_clip]


@pytest.mark.parametrize("make", CALLS)
@pytest.mark.parametrize("as_handle", [False, True])
def test_a_call_on_another_stream_leaves_the_current_ones_memory_alone(make, as_handle):
    """A call on the current stream, waiting behind a long kernel, has let its workspace go when the same call with other
    inputs is made on a side stream, as has a tensor of the current stream: neither may be the second call's workspace."""
    side = torch.cuda.Stream()
    _, here, run_here = make(1)
    _, there, run_there = make(11)
    run_here(None)
    run_there(None)
    want = [t.clone() for t in here + there]
    for t in here + there:
        t.zero_()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms
    held = [torch.full((n << 20,), n, dtype=torch.uint8, device=DEV) for n in (1, 4, 8)]
    copies = [t.clone() for t in held]
    del held
    run_here(None)
    run_there(side.cuda_stream if as_handle else side)
    torch.cuda.synchronize()
    assert all(torch.equal(t, w) for t, w in zip(here + there, want))
    assert all((t == n).all() for t, n in zip(copies, (1, 4, 8)))


@pytest.mark.parametrize("make", CALLS)
def test_captured_and_replayed(make):
    """Two graphs of the same call on different inputs, replayed at once on two streams, and again after the first one's
    inputs changed, give what plain calls give."""
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    cases, graphs = [make(1), make(11)], []
    for (_, _, run), s in zip(cases, sides):
        run(None)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            run(None)
        graphs.append(g)
    for turn in range(3):
        if turn == 1:  # the second's inputs to the first
            for a, b in zip(cases[0][0], cases[1][0]):
                a.copy_(b)
        wants = []
        for _, outs, run in cases:
            run(None)
            wants.append([t.clone() for t in outs])
            for t in outs:
                t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, sides):
            with torch.cuda.stream(s):
                for _ in range(3):
                    g.replay()
        torch.cuda.synchronize()
        for (_, outs, _), want in zip(cases, wants):
            assert all(torch.equal(t, w) for t, w in zip(outs, want))


def test_from_several_threads():
    """Each thread on a stream of its own, all calls at once."""
    cases = [make(100 * i + j) for i in range(3) for j, make in enumerate(CALLS)]
    wants = []
    for _, outs, run in cases:
        run(None)
        wants.append([t.clone() for t in outs])
        for t in outs:
            t.zero_()
    torch.cuda.synchronize()

    def work(case):
        s = torch.cuda.Stream()
        for _ in range(5):
            case[2](s)
        s.synchronize()

    with concurrent.futures.ThreadPoolExecutor(len(cases)) as pool:
        list(pool.map(work, cases))
    for (_, outs, _), want in zip(cases, wants):
        assert all(torch.equal(t, w) for t, w in zip(outs, want))


# ---------------------------------------------------------------- beyond 2^31 elements

def test_embedding_of_a_table_beyond_31_bits():
    vocab, cols = 70001, 32776
    w = torch.zeros(vocab, cols, dtype=BF, device=DEV)
    ids = torch.tensor([vocab - 1, 0, 65535, vocab, vocab - 2], device=DEV)
    for i in (0, 65535, vocab - 2, vocab - 1):
        w[i] = randn(cols, seed=i)
    out = torch.empty(5, cols, dtype=BF, device=DEV)
    tide.tide_embedding(ids, w, out, scale=2.0)
    for r, i in enumerate(ids.tolist()):
        assert torch.equal(out[r], w[i] * 2 if i < vocab else torch.zeros_like(out[r]))
    # Its gradient: all but the rows named are zero, up to the last.
    dw = torch.full_like(w, 3.0)
    tide.tide_embedding_backward(ids, out, dw)
    for r, i in enumerate(ids.tolist()):
        if i < vocab:
            assert torch.equal(dw[i], out[r])
            dw[i] = 0
    assert not dw.any()


@pytest.mark.parametrize("cols", [32776, 32771])
def test_embedding_gradient_of_rows_beyond_31_bits(cols):
    """Small whole numbers, whose sums are exact."""
    n = 70001
    dy = torch.zeros(n, cols, dtype=BF, device=DEV)
    value = torch.arange(n, device=DEV) % 7 - 3
    dy += value[:, None].to(BF)
    ids = torch.arange(n, device=DEV) % 3 * 2
    ids[-1] = 5
    dw = torch.empty(6, cols, device=DEV, dtype=BF)
    tide.tide_embedding_backward(ids, dy, dw)
    want = torch.zeros(6, dtype=torch.float64, device=DEV).index_add_(0, ids, value.double())
    assert torch.equal(dw, want.to(BF)[:, None].expand_as(dw))


@pytest.mark.parametrize("rows,vocab", [(16500, 131077), (17000, 131072)])
def test_log_probs_beyond_31_bits(rows, vocab):
    x = torch.zeros(rows, vocab, dtype=BF, device=DEV)
    ends = torch.tensor([0, 1, rows - 2, rows - 1])
    for i in ends.tolist():
        x[i] = randn(vocab, seed=i) * 3
    t = torch.randint(0, vocab, (rows,), generator=generator(5), device=DEV)
    t[-1] = vocab - 1
    lse, logp, entropy = (torch.empty(rows, device=DEV) for _ in range(3))
    best = torch.empty(rows, 4, device=DEV), torch.empty(rows, 4, dtype=torch.int32, device=DEV)
    tide.tide_log_probs(x, t, logp, lse=lse, entropy=entropy)
    want, tol = R.log_probs(x[ends].cpu(), t[ends].cpu(), 1.0, 4)
    for k, v in (("lse", lse), ("logp", logp), ("entropy", entropy)):
        R.check(v[ends], want[k], tol[k], k)
    tide.tide_log_probs(x[rows - 40:], top=(best[0][rows - 40:], best[1][rows - 40:]))
    assert torch.equal(best[1][ends[2:]].cpu().long(), want["top_tokens"][2:])
    g = randn(rows, seed=3, dtype=torch.float32)
    kept = x[ends].cpu()
    tide.tide_log_probs_backward(x, lse, x, targets=t, dlogp=g)
    want, tol = R.log_probs_grad(kept, lse[ends].cpu(), t[ends].cpu(), g[ends].cpu(), None, None, 1.0)
    R.check(x[ends], want, tol, "dlogits")
    # A row of zeros between: -g / vocab, and g more at the target.
    i = rows // 2
    row = torch.full((vocab,), -1.0 / vocab, dtype=torch.float64)
    row[t[i].item()] += 1.0
    row *= g[i].double().item()
    R.check(x[i], row, 2.0 ** -8 * row.abs() * 1.01, "a row between")


def test_norm_and_clip_beyond_31_bits():
    n = (1 << 31) + 1001
    x = torch.ones(n, dtype=BF, device=DEV)
    y = torch.full((3,), 2.0, device=DEV)
    norm = torch.empty(1, device=DEV)
    tide.tide_grad_norm([x, y], norm)
    want = (n + 12.0) ** 0.5
    assert abs(norm.item() - want) <= 12 * R.U * want
    tide.tide_grad_clip([x, y], norm, want / 4, eps=0.0)  # a quarter, but for roundings
    assert (x[-2000:].float() - 0.25).abs().max() <= 2.0 ** -10 and (x[:2000].float() - 0.25).abs().max() <= 2.0 ** -10
    assert bool((x == x[0]).all()) and (y - 0.5).abs().max() <= 4 * R.U


def test_more_rows_than_one_launch_takes():
    """Rows of one column, on both sides of the place where the second launch begins."""
    rows = (1 << 31) - 1
    at = torch.tensor([0, 1, rows // 2, rows - 300, rows - 257, rows - 256, rows - 255, rows - 2, rows - 1], device=DEV)
    ids = torch.zeros(rows, dtype=torch.int32, device=DEV)
    w = torch.tensor([[1.5], [-2.0], [7.0]], dtype=BF, device=DEV)
    want = torch.tensor([0, 1, 2, 1, 2, 0, 1, 2, 1], dtype=torch.int32, device=DEV)
    ids[at] = want
    x = torch.empty(rows, 1, dtype=BF, device=DEV)
    tide.tide_embedding(ids, w, x)
    assert torch.equal(x[at], w[want.long()])
    x[at] = 1.5
    assert bool((x == 1.5).all())
    # One logit a row, x, and an lse of x + 1: p = 1 / e, so that the gradient is g (1 - 1 / e), and 0 where the target is
    # outside.
    lse = torch.full((rows,), 2.5, device=DEV)
    g = torch.full((rows,), 1.0, device=DEV)
    g[at] = torch.arange(1.0, 10.0, device=DEV)
    tide.tide_log_probs_backward(x, lse, x, targets=ids, dlogp=g)
    p = 2.718281828459045 ** -1
    got = x[at].double().cpu()[:, 0]
    exact = torch.arange(1.0, 10.0, dtype=torch.float64) * torch.where(want.cpu() == 0, 1 - p, 0.0)
    assert ((got - exact).abs() <= 2.0 ** -8 * 1.01 * exact.abs()).all()
    x[at] = x[5000].clone()
    assert bool((x == x[5000]).all()) and abs(x[5000].item() - (1 - p)) <= 2.0 ** -8
