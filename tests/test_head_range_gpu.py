"""A head's log probabilities and gradients where logits are far from zero, and the
exponential of the gradients, on the GPU against 64 bits.

The gradient's p = exp(x - lse): 2^-22 of itself for the exponential (the accuracy that PTX
gives for ex2.approx), 2^-24 for each of its correction and the product with g, and G's three bf16
terms and their sum 2 * 2^-23: 2^-20 together for fp32. lse of the forward call is off by
2^-22 + 70 * 2^-24 < 2^-17 (exponentials, sums of 32, two roundings for each of 32 joins): with
it p is off by 2^-16 at most.
"""
import math

import pytest
import torch
from test_head_masks_gpu import with_masks

from checkpoint_averaging_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    yield
    torch.cuda.synchronize()
    assert B.operators_status() == 0


def apart(logits, base, dtype):
    """Hidden states and head of these logits [rows, vocab] plus base: the head's gradient then
    has G^T in its first columns."""
    rows, vocab = logits.shape
    hidden = torch.cat([torch.eye(rows), torch.ones(rows, 1)], 1)
    head = torch.cat([logits.t(), torch.full((vocab, 1), float(base))], 1)
    return hidden.to(dtype).to(DEV), head.to(dtype).to(DEV)


@pytest.mark.parametrize("rows,vocab", [(5, 3000), (64, 1 << 17), (100, 2000), (300, 1000)])
def test_exponentials_of_the_gradients(rows, vocab):
    gen = torch.Generator().manual_seed(rows)
    logits = torch.rand(rows, vocab, generator=gen) * 80 - 60
    hidden, head = apart(logits, 0.0, F32)
    lse = (torch.rand(rows, generator=gen) * 30 - 10).to(DEV)
    lo = lse * 2.0 ** -25
    x = logits.to(DEV).double()
    tokens = torch.zeros(rows, dtype=torch.int64, device=DEV)
    g = torch.full((rows,), -1.0, device=DEV)
    _, got = B.head_logprobs_backward(hidden, head, tokens, lse, lse, g, lse_lo=lo, need_hidden=False)
    want = (x - lse.double()[:, None] - lo.double()[:, None]).exp()
    G = got.double().t()[:rows]
    off = ((G - want).abs() / want)[:, 1:]
    fine = want[:, 1:] > 2.0 ** -100  # (smaller ones have fewer bits in three bf16 terms)
    assert float(off[fine].max()) <= 2.0 ** -20


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,vocab", [(5, 300), (64, 1 << 17), (100, 700), (300, 600)])
@pytest.mark.parametrize("power", [10, 17, 20, 22, 23])
def test_gradients_of_logits_beyond_their_fraction(rows, vocab, power, dtype):
    # lse rounded to binary32 leaves up to 2^(power - 24) in lse_lo: a half at 2^23
    gen = torch.Generator().manual_seed(rows + power)
    logits = torch.randint(0, 9, (rows, vocab), generator=gen).float()
    hidden, head = apart(logits, 2.0 ** power, dtype)
    x = logits.to(DEV).double() + 2.0 ** power
    lse = torch.logsumexp(x, 1)
    p = (x - lse[:, None]).exp()
    tokens = torch.randint(0, vocab, (rows,), generator=gen).to(DEV)
    r = B.head_logprobs(hidden, head, tokens)
    at = (torch.arange(rows, device=DEV), tokens)
    assert ((r.lse.double() + r.lse_lo.double() - lse).abs() <= 2.0 ** -17).all()
    assert ((r.logp.double() - (x - lse[:, None])[at]).abs() <= 2.0 ** -16).all()
    g = torch.full((rows,), -1.0, device=DEV)
    _, got = B.head_logprobs_backward(hidden, head, tokens, r.lse, r.entropy, g, lse_lo=r.lse_lo,
                                      need_hidden=False)
    G = p.clone()
    G[at] -= 1.0
    # bf16: G in one or two terms and the result's rounding
    rel = 2.0 ** -16 + (2.0 ** -7 if dtype == BF16 else 0.0)
    off = (got.double().t()[:rows] - G).abs() / G.abs()
    assert float(off.max()) <= rel


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [5, 100, 300])
def test_rows_whose_mask_leaves_nothing(rows, dtype):
    """Every id masked: the logits are equal, so is every p."""
    vocab, width = 901, 40
    hidden, head, _, _ = with_masks(rows, vocab, width, dtype, [0])
    head[:, -1] = torch.finfo(dtype).min
    tokens = torch.arange(rows, device=DEV) % vocab
    r = B.head_logprobs(hidden, head, tokens)
    assert (r.lse == torch.finfo(dtype).min).all()
    assert ((r.logp.double() + math.log(vocab)).abs() <= 2.0 ** -16 * math.log(vocab)).all()
    assert ((r.entropy.double() - math.log(vocab)).abs() <= 2.0 ** -16 * math.log(vocab)).all()
    g = torch.full((rows,), -1.0, device=DEV)
    G = torch.full((rows, vocab), 1.0 / vocab, device=DEV, dtype=torch.float64)
    G.scatter_add_(1, tokens[:, None], torch.full((rows, 1), -1.0, device=DEV).double())
    # (the head's other columns: its bias times G is of no use)
    dx, dw = B.head_logprobs_backward(hidden, head, tokens, r.lse, r.entropy, g, lse_lo=r.lse_lo)
    a = hidden.double()
    want, scale = G.t() @ a, G.abs().t() @ a.abs()
    rel = 2.0 ** -15 + (2.0 ** -8 if dtype == BF16 else 0.0)
    tol = rel * scale + (2.0 ** -8 * want.abs() if dtype == BF16 else 0.0)
    assert ((dw.double() - want).abs() <= tol).all()
    w = head[:, :-1].double()
    want, scale = G @ w, G.abs() @ w.abs()
    tol = rel * scale + (2.0 ** -8 * want.abs() if dtype == BF16 else 0.0)
    assert ((dx[:, :-1].double() - want).abs() <= tol).all()
