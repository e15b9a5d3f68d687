"""The sizes that the operators at the ends of a training step refuse, beside the last ones that they take, as
include/tide_lm_ops.h has them.  No call here reaches the GPU."""

import pytest

from test_lm_ops_host import INVALID, OK, UNIMPLEMENTED, clip, embed, embed_grad, lib, norm, probs, probs_grad

TOKENS, VOCAB, COLS, ROWS, LOGITS, ELEMENTS = (1 << 31) - 1, (1 << 31) - 2, 1 << 24, (1 << 31) - 1, (1 << 31) - 17, 1 << 40


# An accepted size ends at a later check of the same call: a missing output, or nothing to do.
@pytest.mark.parametrize("call,size,last,other,then", [
    (embed, "tokens", TOKENS, dict(out=None), INVALID),
    (embed, "vocab", VOCAB, dict(tokens=0), OK),
    (embed, "cols", COLS, dict(tokens=0), OK),
    (embed_grad, "tokens", TOKENS, dict(dw=None), INVALID),
    (embed_grad, "vocab", VOCAB, dict(tokens=0, add=1), OK),
    (embed_grad, "cols", COLS, dict(tokens=0, add=1), OK),
    (probs, "rows", ROWS, dict(logp=None, t=None), OK),
    (probs, "vocab", LOGITS, dict(rows=0, ldz=LOGITS + 1), OK),
    (probs_grad, "rows", ROWS, dict(out=None), INVALID),
    (probs_grad, "vocab", LOGITS, dict(rows=0, ldz=LOGITS + 1), OK),
    (norm, "numels", ELEMENTS, dict(out=None), INVALID),
    (clip, "numels", ELEMENTS, dict(norm=None), INVALID),
])
def test_the_last_size_taken_and_the_first_refused(call, size, last, other, then):
    def at(n):
        return call(**{size: (8, n) if size == "numels" else n, **other})

    assert at(last) == then, lib().tide_last_error()
    assert at(last + 1) == UNIMPLEMENTED
    assert lib().tide_last_error()


@pytest.mark.parametrize("call", [probs, probs_grad])
def test_scales_that_are_taken(call):
    for scale in (2.0 ** -120, 1.0, 2.0 ** 64):
        assert call(scale=scale, rows=0) == OK
    for scale in (2.0 ** -121, 1e-40, 2.0 ** 65):
        assert call(scale=scale, rows=0) == INVALID
