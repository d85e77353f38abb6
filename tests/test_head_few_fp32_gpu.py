"""Log probabilities and gradients of few fp32 rows over a head of 2^23 elements and more,
whose terms are made on the way into the tensor cores, and at the sizes where that begins
(definitions and tolerances: test_head_gpu.py)."""
import math

import pytest
import torch
from test_head_gpu import DEV, F32, Exact, check, check_grad, inputs, poison

from checkpoint_averaging_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    yield
    torch.cuda.synchronize()
    assert B.operators_status() == 0


SIZES = [(1, 50304, 200), (2, 70001, 131), (3, 400, 20011), (5, 16500, 515), (16, 30011, 300), (64, 20011, 424),
         (65, 16411, 520), (127, 16500, 513), (128, 9000, 1000), (100, 513, 16384),
         # either side of the elements, the rows and the width that decide
         (7, 16384, 512), (7, 16383, 512), (64, 32768, 256), (65, 32768, 256), (128, 16384, 512),
         (128, 16384, 513), (129, 16384, 513)]


@pytest.mark.parametrize("rows,vocab,width", SIZES)
def test_sizes(rows, vocab, width):
    hidden, head, tokens = inputs(rows, vocab, width, F32)
    e = Exact(hidden, head, tokens)
    a, b = check(hidden, head, tokens, e=e), B.head_logprobs(hidden, head, tokens)
    for u, v in zip(a, b):
        assert u is None or torch.equal(u, v)
    x, y = check_grad(hidden, head, tokens, e=e), check_grad(hidden, head, tokens, e=e)
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    check_grad(hidden, head, tokens, with_h=False, e=e)
    only = check_grad(hidden, head, tokens, need_head=False, e=e)
    assert only[1] is None and torch.equal(only[0], x[0])
    only = check_grad(hidden, head, tokens, need_hidden=False, e=e)
    assert only[0] is None and torch.equal(only[1], x[1])


@pytest.mark.parametrize("rows", [7, 100])
@pytest.mark.parametrize("width", [516, 518, 519])
@pytest.mark.parametrize("pad, offset", [(0, 0), (0, 1), (1, 0), (2, 0), (4, 0), (4, 2), (8, 4), (3, 2)])
def test_strides_and_what_lies_beside(rows, width, pad, offset):
    vocab = 16411
    hidden, head, tokens = inputs(rows, vocab, width, F32)
    want, grads = check(hidden, head, tokens), check_grad(hidden, head, tokens)
    a = torch.full((rows + 1, width + pad + offset), math.nan, device=DEV)
    w = torch.full((vocab + 1, width + pad + offset), math.nan, device=DEV)
    a[:rows, offset:offset + width], w[:vocab, offset:offset + width] = hidden, head
    a, w = a[:rows, offset:offset + width], w[:vocab, offset:offset + width]
    poison()
    for u, v in zip(want, B.head_logprobs(a, w, tokens)):
        assert u is None or torch.equal(u, v)
    poison()
    got = check_grad(a, w, tokens)
    assert torch.equal(got[0], grads[0]) and torch.equal(got[1], grads[1])


@pytest.mark.parametrize("rows", [7, 100])
def test_rows_that_are_broken(rows):
    hidden, head, tokens = inputs(rows, 16411, 520, F32)
    good = B.head_logprobs(hidden, head, tokens)
    hidden[0, 3], hidden[2, 519], hidden[4, 0] = math.nan, math.inf, -math.inf
    r = B.head_logprobs(hidden, head, tokens)
    bad = torch.zeros(rows, dtype=torch.bool, device=DEV)
    bad[[0, 2, 4]] = True
    for u, v in zip(r, good):
        if u is not None:
            assert torch.isnan(u[bad]).all() and torch.equal(u[~bad], v[~bad])
    # without a gradient they reach nothing, whether by theirs or by their token's id
    g = torch.full((rows,), -1.0, device=DEV)
    for t, gt in ((tokens, g.masked_fill(bad, 0.0)), (tokens.masked_fill(bad, -5), g)):
        gx, gw = B.head_logprobs_backward(hidden, head, t, r.lse, r.entropy, gt, None, lse_lo=r.lse_lo)
        assert (gx[bad] == 0).all() and torch.isfinite(gx).all() and torch.isfinite(gw).all()
    gx, gw = B.head_logprobs_backward(hidden, head, tokens, r.lse, r.entropy, g, None)
    assert torch.isnan(gx[bad]).all() and torch.isfinite(gx[~bad]).all() and torch.isnan(gw).all()


@pytest.mark.parametrize("rows", [7, 100])
def test_large_logits_and_equal_ones(rows):
    hidden, head, tokens = inputs(rows, 16411, 520, F32, spread=400.0)
    check(hidden, head, tokens)
    check_grad(hidden, head, tokens)
    head[5] = head[6]
    check(hidden, head, tokens)
    r = B.head_logprobs(torch.zeros_like(hidden), head, tokens)
    known = tokens >= 0
    assert (r.logp[known] + math.log(16411)).abs().max() < 1e-5
    assert (r.entropy - math.log(16411)).abs().max() < 1e-5
