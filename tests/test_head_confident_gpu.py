"""Gradients of rows that are sure of their token, by the log sum that the forward call left,
against 64 bits. The gradient of the token's logit is g (1 - p), so what the two calls' sums
of one logit differ by shows as a multiple of itself where p is near 1.

Tolerances. A logit is summed on the tensor cores in runs of 256 terms for fp32 and 768 for
bf16 inputs, whose sums are added in fp32. Per 16 terms of a run two roundings of at most 2^-23 of
A = sum |hidden_i head_i|, per run one of 2^-24 of it, and for fp32 2^-22 A for the products of
terms that are left out (the small products of a run are summed first, at 2^-8 of A at most:
another eighth): off = (2.25 run / 16 + width / run / 2 + 2) 2^-23 max A, whatever the width but
for its share of 2^-24 per run. Every p but the token's is then off by r = 2 off + 2^-16 of itself (2^-16: the
exponential, the sums over the vocabulary and lse's two parts, test_head_range_gpu.py), and so is
1 - p, their sum; G of the token as g (1 - p), the others as g p. With the entropy's gradient h,
G = -h p (log p + H) moves by (|log p| + H + 1) r of h p, and at the token, where log p and H are of
the size of 1 - p, by 4 r (|log p| + H) of h p (H moves by r (H + (1 - p)) at most).
What the products add is in test_head_gpu.py.
"""
import math

import pytest
import torch

from checkpoint_averaging_gb300 import binding as B
from checkpoint_averaging_gb300 import probe as P

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


def confident(rows, vocab, width, dtype, seed=1):
    """Dense rows and head, a token of its own for each row, whose logit leads by so much that
    1 - p runs from some 1e-2 to 1e-8."""
    gen = torch.Generator().manual_seed(seed + rows + vocab + width)
    head = torch.randn(vocab, width, generator=gen) * (2.5 / math.sqrt(width))
    tokens = torch.randperm(vocab, generator=gen)[:rows]
    lead = math.log(vocab) + torch.linspace(4.6, 18.4, rows)
    mine = head[tokens]
    hidden = mine * (lead / (mine * mine).sum(1))[:, None]
    return hidden.to(dtype).to(DEV), head.to(dtype).to(DEV), tokens.to(DEV)


class Exact:
    def __init__(self, hidden, head, tokens):
        self.a, self.w, self.tokens = hidden.double(), head.double(), tokens
        self.rows = torch.arange(len(tokens), device=DEV)
        x = self.a @ self.w.t()
        d = x - x[self.rows, tokens][:, None]  # relative to the token's
        e = d.exp()
        e[self.rows, tokens] = 0.0
        rest = e.sum(1)
        self.mine = -torch.log1p(rest)
        self.p = e / (1 + rest)[:, None]  # (0 at the token)
        self.miss = rest / (1 + rest)  # 1 - p of the token
        self.own = 1 / (1 + rest)
        self.logp = d + self.mine[:, None]
        self.H = (torch.special.entr(self.p)).sum(1) - self.own * self.mine
        run = 256 if hidden.dtype == F32 else 768
        A = (self.a.abs() @ self.w.abs().t()).amax(1)
        self.r = 2 * (2.25 * run / 16 + hidden.shape[1] / run / 2 + 2) * 2.0 ** -23 * A + 2.0 ** -16

    def gradient(self, g, h):
        """G, and how far it may be off."""
        c, k, r = g.double()[:, None], h.double()[:, None], self.r[:, None]
        H, at = self.H[:, None], (self.rows, self.tokens)
        G = -self.p * (c + k * (self.logp + H))
        G[at] = g.double() * self.miss - h.double() * self.own * (self.mine + self.H)
        dG = self.p * (c.abs() + k.abs() * (self.logp.abs() + H + 1)) * r
        dG[at] = self.r * (g.double().abs() * self.miss
                           + h.double().abs() * 4 * (self.mine.abs() + self.H))
        return G, dG


SIZES = [(9, 500, 2048), (9, 4200, 2048), (100, 4200, 2048), (100, 700, 4096), (300, 900, 4096), (300, 4200, 2048),
         (9, 300, 16384), (140, 300, 16384)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,vocab,width", SIZES)
@pytest.mark.parametrize("entropy", [False, True])
def test_gradients_by_the_forward_calls_lse(rows, vocab, width, dtype, entropy):
    hidden, head, tokens = confident(rows, vocab, width, dtype)
    e = Exact(hidden, head, tokens)
    r = B.head_logprobs(hidden, head, tokens)
    assert ((r.logp.double() - e.mine).abs() <= (e.r + 2e-5) * e.mine.abs()).all()
    gen = torch.Generator().manual_seed(rows)
    g = -(torch.rand(rows, generator=gen) + 0.5).to(DEV)
    h = torch.randn(rows, generator=gen).to(DEV) * 0.1 if entropy else torch.zeros(rows, device=DEV)
    got = B.head_logprobs_backward(hidden, head, tokens, r.lse, r.entropy, g, h if entropy else None,
                                   lse_lo=r.lse_lo)
    G, dG = e.gradient(g, h)
    dG = dG + (2.0 ** -8 if dtype == BF16 else 2.0 ** -23) * G.abs()
    for out, other, dGo, Go, n in ((got[0], e.w, dG, G, vocab), (got[1], e.a, dG.t(), G.t(), rows)):
        want = Go @ other
        # (sums over the vocabulary in runs of 8,192 terms at most)
        tol = dGo @ other.abs() + (2 * min(n, 8192) / 16 + 64) * 2.0 ** -23 * (Go.abs() @ other.abs())
        if dtype == BF16:
            tol += 2.0 ** -8 * want.abs()
        off = (out.double() - want).abs()
        assert (off <= tol + 1e-37).all(), (float((off / (tol + 1e-37)).max()), int((off > tol).sum()))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,vocab,width", SIZES)
@pytest.mark.parametrize("given", ["none", "negative", "another"])
def test_entropy_gradients_of_rows_sure_of_another_id(rows, vocab, width, dtype, given):
    """The id that has nearly all of the probability is not the row's token: log p + H of it is of
    the size of 1 - p all the same."""
    hidden, head, sure = confident(rows, vocab, width, dtype)
    e = Exact(hidden, head, sure)
    tokens = {"none": None, "negative": torch.full_like(sure, -1), "another": (sure + 1) % vocab}[given]
    r = B.head_logprobs(hidden, head, tokens)
    gen = torch.Generator().manual_seed(rows)
    h = (torch.rand(rows, generator=gen) + 0.5).to(DEV)
    zero = torch.zeros(rows, device=DEV)
    got = B.head_logprobs_backward(hidden, head, tokens, r.lse, r.entropy, zero if given == "another" else None, h,
                                   lse_lo=r.lse_lo)
    G, dG = e.gradient(zero, h)
    dG = dG + (2.0 ** -8 if dtype == BF16 else 2.0 ** -23) * G.abs()
    for out, other, dGo, Go, n in ((got[0], e.w, dG, G, vocab), (got[1], e.a, dG.t(), G.t(), rows)):
        want = Go @ other
        tol = dGo @ other.abs() + (2 * min(n, 8192) / 16 + 64) * 2.0 ** -23 * (Go.abs() @ other.abs())
        if dtype == BF16:
            tol += 2.0 ** -8 * want.abs()
        off = (out.double() - want).abs()
        assert (off <= tol + 1e-37).all(), (float((off / (tol + 1e-37)).max()), int((off > tol).sum()))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,vocab,width", [(9, 4200, 2048), (300, 900, 4096)])
def test_rows_push_along_their_token(rows, vocab, width, dtype):
    """Through autograd: a row's gradient pushes it along its token's row of the head, by
    1 - p, however small."""
    hidden, head, tokens = confident(rows, vocab, width, dtype)
    e = Exact(hidden, head, tokens)
    a, w = hidden.clone().requires_grad_(True), head.clone().requires_grad_(True)
    (-P.differentiable_head_logprobs(a, w, tokens)[0].sum()).backward()
    assert torch.isfinite(w.grad).all()
    mine = e.w[tokens]
    size = (mine * mine).sum(1)
    G, _ = e.gradient(torch.full((rows,), -1.0, device=DEV), torch.zeros(rows, device=DEV))
    along, want = (a.grad.double() * mine).sum(1) / size, ((G @ e.w) * mine).sum(1) / size
    assert (want < 0).all() and (along < 0).all()
    rel = e.r + (3 * 2.0 ** -8 if dtype == BF16 else 2.0 ** -10)  # (sums over the vocabulary)
    tol = rel * ((G.abs() @ e.w.abs()) * mine.abs()).sum(1) / size
    assert ((along - want).abs() <= tol).all(), float(((along - want).abs() / tol).max())
