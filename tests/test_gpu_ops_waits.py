"""Bounded waits of the training-block operators that run out: what is reported,
and that the calls after it are right."""

import concurrent.futures

import pytest
import torch

import fsdp_layout_aware_gb300 as tide

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


class options:
    """A wait limit (ns) and a withheld load for the calls within."""

    def __init__(self, limit, drop=-1):
        self.limit, self.drop = limit, drop

    def __enter__(self):
        tide.tide_ops_set_option(tide.TIDE_OPS_OPT_WAIT_LIMIT_NS, self.limit)
        tide.tide_ops_set_option(tide.TIDE_OPS_OPT_TEST_DROP_LOAD, self.drop)

    def __exit__(self, *_):
        tide.tide_ops_set_option(tide.TIDE_OPS_OPT_TEST_DROP_LOAD, -1)
        tide.tide_ops_set_option(tide.TIDE_OPS_OPT_WAIT_LIMIT_NS, 2_000_000_000)


def randn(*shape, seed, dtype=BF):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def norm_gradient(rows, cols, kept):
    h, dy, w = randn(rows, cols, seed=1), randn(rows, cols, seed=2), randn(cols, seed=3)
    rstd, dx, dw = torch.ones(rows, device=DEV), torch.empty_like(dy), torch.empty_like(w)
    if kept:
        ck = tide.Checkpoint8.empty(rows, cols)
        tide.tide_checkpoint_store(h, ck)
        h = ck
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    return (dx, dw), lambda: tide.tide_rms_norm_backward(dy, h, w, rstd, dx, dweight=dw, workspace=ws)


SHAPES = [(1, 4096, False), (3, 512, True), (152, 8192, False), (700, 2047, False), (608, 5120, True), (40, 16384, True)]


@pytest.mark.parametrize("rows,cols,kept", SHAPES)
def test_a_copy_withheld_where_nothing_is_handed_back(rows, cols, kept):
    """The first rows' copies: with so few turns a block that the warp that copies waits for no slot before it is done."""
    outs, run = norm_gradient(rows, cols, kept)
    run()
    tide.tide_ops_check()
    want = [t.clone() for t in outs]
    with options(20_000_000, 0):
        run()
        with pytest.raises(tide.TideError) as e:
            tide.tide_ops_check()
        assert e.value.status == 8
    for t in outs:
        t.zero_()
    run()
    tide.tide_ops_check()
    assert all(torch.equal(t, w) for t, w in zip(outs, want))


@pytest.mark.parametrize("rows,cols,kept", SHAPES)
def test_a_limit_that_no_copy_meets(rows, cols, kept):
    """Waits of a nanosecond: given up or not, copies land before their block leaves, and what runs next is right."""
    outs, run = norm_gradient(rows, cols, kept)
    run()
    tide.tide_ops_check()
    want = [t.clone() for t in outs]
    for _ in range(5):
        with options(1):
            run()
        for t in outs:
            t.zero_()
        run()
        try:
            tide.tide_ops_check()
        except tide.TideError as e:
            assert e.status == 8
        assert all(torch.equal(t, w) for t, w in zip(outs, want))


def product():
    x, w, y = randn(64, 4096, seed=1), randn(256, 4096, seed=2), torch.empty(64, 256, dtype=BF, device=DEV)
    return lambda: tide.tide_linear(x, w, y)


def status_of(f):
    try:
        f()
    except tide.TideError as e:
        return e.status
    return 0


@pytest.mark.parametrize("first", ["caller", "other"])
def test_every_thread_that_checks_learns_of_a_timeout(first):
    """Whichever checks first, the thread that made the call or another, takes no report from the other."""
    run = product()

    def withheld():
        with options(20_000_000, 2):
            run()

    with concurrent.futures.ThreadPoolExecutor(1) as pool:
        def other():
            return pool.submit(status_of, tide.tide_ops_check).result()

        other(), status_of(tide.tide_ops_check)  # what earlier calls left
        assert (other(), status_of(tide.tide_ops_check)) == (0, 0)
        withheld()
        if first == "caller":
            got = [status_of(tide.tide_ops_check), other()]
        else:
            got = [other(), status_of(tide.tide_ops_check)]
        assert got == [8, 8]
        assert (other(), status_of(tide.tide_ops_check)) == (0, 0)
        pool.submit(withheld).result()
        assert (status_of(tide.tide_ops_check), other()) == (8, 8)
        run()
        assert (status_of(tide.tide_ops_check), other()) == (0, 0)


def test_a_withheld_load_is_the_calling_threads_own():
    """The test hook set in one thread leaves another thread's products and norms alone."""
    outs, run = norm_gradient(700, 2048, False)
    run()
    product()()
    status_of(tide.tide_ops_check)
    with concurrent.futures.ThreadPoolExecutor(1) as pool, options(20_000_000, 1):
        pool.submit(run).result()
        pool.submit(product()).result()
        assert status_of(tide.tide_ops_check) == 0
        product()()
        assert status_of(tide.tide_ops_check) == 8
