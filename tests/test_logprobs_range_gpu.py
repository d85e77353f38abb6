"""Log probabilities and their gradient where the arithmetic's range decides:
masked logits under large gradients, and logits far from 0, on the GPU against
the definitions in 64 bits with the largest logit subtracted first.

Tolerances, absolute, from the derivations in test_logprobs_gpu.py with the
magnitude of the logits taken out: x - M is exact where it matters, so log p
keeps 2e-5 + 2^-22 |log p| however large M is.
"""
import math

import pytest
import torch

from checkpoint_averaging_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = math.inf


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    yield
    torch.cuda.synchronize()


def distribution(x):
    """In 64 bits: M, log s (lse = M + log s), log p, p and the entropy."""
    x = x.double()
    M = x.amax(1, keepdim=True)
    d = x - M
    e = d.exp()
    s = e.sum(1, keepdim=True)
    log_s = s.log()
    H = log_s - (e * d.masked_fill(e == 0, 0.0)).sum(1, keepdim=True) / s
    return M, log_s, d - log_s, e / s, H


def gradient(x, tokens, g, h):
    """The formula, and what rounding may add: 1e-4 p (|g| + |h| (|log p| + H)) + 2^-22 |g|,
    and 2^-8 of a bf16 result."""
    _, _, logp, p, H = distribution(x)
    g, h = g.double()[:, None], h.double()[:, None]
    known = (tokens >= 0)[:, None]
    one = torch.zeros_like(p).scatter_(1, tokens.clamp(min=0)[:, None], 1.0)
    lp = logp.masked_fill(p == 0, 0.0)
    want = g * known * (one - p) - h * p * (lp + H)
    tol = 1e-4 * p * (g.abs() + h.abs() * (lp.abs() + H)) + 2.0 ** -22 * g.abs()
    if x.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs()
    return want, tol


def statistics(x):
    """(lse, what its rounding left out, entropy) as the forward call would give them, from 64 bits."""
    M, log_s, _, _, H = distribution(x)
    lse = (M + log_s).float()
    return lse[:, 0], ((M - lse.double()) + log_s).float()[:, 0], H.float()[:, 0]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [40, 3001, 50304])
@pytest.mark.parametrize("at", [0, 1, 3])
def test_masked_logits_under_large_entropy_gradients(vocab, at, dtype):
    # a masked logit's gradient is 0 whatever h is: p is 0 there, and its factor has to stay finite
    hs = [2.0, -5.0, 1e3, 65536.0, 1e6, -1e10, 1e20, 0.3]
    gen = torch.Generator().manual_seed(vocab + at)
    wide = torch.randn(2 * len(hs), vocab + 8, generator=gen) * 2.5
    x = wide.to(dtype).to(DEV)[:, at:at + vocab]
    for r in range(len(x)):
        mask = -INF if r % 2 else torch.finfo(dtype).min
        x[r, r % 3::3] = mask
        x[r, vocab // 4:vocab // 2] = mask
        if r in (4, 5):
            x[r, 9:] = mask
    h = torch.tensor([v for v in hs for _ in range(2)], device=DEV)
    g = torch.full((len(x),), -0.5, device=DEV)
    tokens = (torch.arange(len(x), device=DEV) * 5 + 1) % vocab
    tokens[3] = -1
    lse, lo, H = statistics(x)
    out = torch.empty_like(wide, dtype=dtype, device=DEV)[:, at:at + vocab]
    B.token_logprobs_backward(x, tokens, lse, H, g, h, lse_lo=lo, out=out)
    want, tol = gradient(x, tokens, g, h)
    assert ((out.double() - want).abs() <= tol).all()
    assert torch.equal(out, B.token_logprobs_backward(x, tokens, lse, H, g, h, lse_lo=lo, out=x))


FAR = [1e6, 1.6e7, 2e7, 1e9, 3e9, 1e10, 1e11, 1e12, 1e15, 1e25, 1e30, 9e35, 1e37]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [300, 9000, 50304])
@pytest.mark.parametrize("sign", [1, -1])
def test_gradient_of_rows_far_from_0(vocab, sign, dtype):
    # a row of equal logits (a mask of a finite value left nothing else), two tied logits above the
    # rest, masks beside them, and rows where such a value masks all but a few
    gen = torch.Generator().manual_seed(vocab)
    x = (torch.randn(5 * len(FAR), vocab, generator=gen) * 2.5).to(dtype).to(DEV)
    for i, c in enumerate(FAR):
        c = torch.tensor(sign * c).to(dtype).item()
        x[5 * i] = c
        x[5 * i + 1] = min(2 * c, c / 2)
        x[5 * i + 1, 5::vocab // 2] = c
        x[5 * i + 2] = c
        x[5 * i + 2, 1::2] = -INF
        x[5 * i + 3, 20:] = -abs(c)
        x[5 * i + 4, ::2] = -abs(c)
    g = torch.linspace(-1, 1, len(x)).to(DEV)
    h = torch.linspace(0.5, -3, len(x)).to(DEV)
    tokens = (torch.arange(len(x), device=DEV) * 7 + 5) % vocab
    tokens[::6] = -1
    lse, lo, H = statistics(x)
    got = B.token_logprobs_backward(x, tokens, lse, H, g, h, lse_lo=lo)
    want, tol = gradient(x, tokens, g, h)
    assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab,top", [
    (170, 40000, 3), (1300, 33001, 0), (8, 73760, 12), (2, 300001, 5), (400, 9000, 4)])
@pytest.mark.parametrize("sign", [1, -1])
def test_log_probabilities_far_from_0(rows, vocab, top, sign, dtype):
    # rows of equal logits, a few tied ones above the rest, masks beside them, rows where such a
    # value masks all but a few or a run of the vocabulary, and one logit far above ordinary ones;
    # in sizes that stream, that a cluster shares and that a block holds
    gen = torch.Generator().manual_seed(vocab)
    for first in range(0, 7 * len(FAR), rows):
        x = (torch.randn(min(rows, 200), vocab, generator=gen) * 2.5).to(dtype).to(DEV)
        if rows > 200:
            x = x.repeat(-(-rows // 200), 1)[:rows]
        for r in range(rows):
            c, kind = FAR[(first + r) // 7 % len(FAR)], (first + r) % 7
            c = torch.tensor(sign * c).to(dtype).item()
            if kind == 0:
                x[r] = c
            elif kind == 1:
                x[r] = min(2 * c, c / 2)
                x[r, 5::vocab // 3] = c
            elif kind == 2:
                x[r] = c
                x[r, 1::2] = -INF
            elif kind == 3:
                x[r, 20:] = -abs(c)
            elif kind == 4:
                x[r, vocab // 3:] = -abs(c)
            elif kind == 5:
                x[r] = c
                x[r, vocab // 2] = c / 2 if c < 0 else c * 2
            else:
                x[r, vocab - 7] = abs(c)
        tokens = (torch.arange(rows, device=DEV) * 7 + 5) % vocab
        got = B.token_logprobs(x, tokens, top=top)
        for at in range(0, rows, 100):
            s = slice(at, min(rows, at + 100))
            M, log_s, logp, p, H = distribution(x[s])
            mine = logp.gather(1, tokens[s, None])[:, 0]
            tol = 2e-5 + 2.0 ** -22 * mine.abs()
            assert torch.equal(torch.isinf(got.logp[s]), torch.isinf(mine))
            fine = torch.isfinite(mine)
            assert ((got.logp[s].double() - mine).abs() <= tol)[fine].all()
            lse = (M + log_s)[:, 0]
            assert ((got.lse[s].double() - lse).abs() <= 2e-5 + 2.0 ** -23 * lse.abs()).all()
            # lse and what it left out, together
            both = (got.lse[s].double() - M[:, 0]) + got.lse_lo[s].double()
            assert ((both - log_s[:, 0]).abs() <= 2e-5 + 2.0 ** -22 * log_s[:, 0]).all()
            # a streamed row's terms have exponents of up to 64 in common, in sums of at most 200
            # additions in a row: 64 * 200 * 2^-24 < 8e-4 on the entropy
            assert ((got.entropy[s].double() - H[:, 0]).abs() <= 8e-4 + 2e-5 * H[:, 0]).all()
            if top:
                ids = torch.sort(x[s].double(), dim=1, descending=True, stable=True).indices[:, :top]
                assert torch.equal(got.top_ids[s], ids)
                best = logp.gather(1, ids)
                ok = torch.isfinite(best)
                off = (got.top_logp[s].double() - best).abs() - (2e-5 + 2.0 ** -22 * best.abs())
                assert torch.equal(ok, torch.isfinite(got.top_logp[s])) and (off[ok] <= 0).all()
        if rows >= 7 * len(FAR):
            break
