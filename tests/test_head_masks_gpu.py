"""A head's log probabilities and gradients where logits hold masks (a bias column of the head
that is the type's lowest value for ids that cannot occur), on the GPU against 64 bits, at
the tolerances of test_head_gpu.py.
"""
import math

import pytest
import torch
from test_head_gpu import Exact

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


def with_masks(rows, vocab, width, dtype, masked, seed=0):
    gen = torch.Generator().manual_seed(seed + rows + vocab)
    head = torch.randn(vocab, width, generator=gen) * (2.0 / math.sqrt(width))
    hidden = torch.randn(rows, width, generator=gen)
    hidden[:, -1] = 1.0
    head[masked, -1] = torch.finfo(dtype).min
    keep = torch.ones(vocab, dtype=torch.bool)
    keep[masked] = False
    tokens = keep.nonzero()[:, 0][torch.randint(0, int(keep.sum()), (rows,), generator=gen)]
    return hidden.to(dtype).to(DEV), head.to(dtype).to(DEV), tokens.to(DEV), keep.to(DEV)


MASKS = {"one": [7], "some": list(range(3, 900, 17)), "first": list(range(70)), "tile": list(range(256, 600)),
         "last": list(range(640, 901)), "most": [j for j in range(901) if j % 300 != 5]}

CASES = [(rows, 901, 40, dtype, MASKS[m]) for m in MASKS for rows in (5, 100, 300) for dtype in (F32, BF16)]
# (few fp32 rows over 2^23 elements: a kernel of their own)
CASES += [(rows, 14001, 600, F32, list(range(9000, 13000)) + [5, 6, 7]) for rows in (9, 100)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}-{str(c[3])[6:]}-{len(c[4])}")
def test_log_probabilities_with_masks(case):
    """As of the ids that can occur alone."""
    hidden, head, tokens, keep = with_masks(*case)
    rows, dtype = len(tokens), hidden.dtype
    new_id = keep.cumsum(0) - 1
    e = Exact(hidden, head[keep], new_id[tokens])
    r = B.head_logprobs(hidden, head, tokens)
    off = e.off.amax(1)
    base = 2e-5 + 2.0 ** -22 * e.L
    assert ((r.lse.double() - e.lse).abs() <= base + off).all()
    assert ((r.logp.double() - e.mine).abs() <= base + 2 * off).all()
    assert ((r.entropy.double() - e.H).abs() <= base + (4 * off + 2e-5) * e.H).all()
    # a masked token's own log probability
    ids = (~keep).nonzero()[:, 0]
    t = ids[torch.arange(rows, device=DEV) % len(ids)]
    low = B.head_logprobs(hidden, head, t).logp.double()
    assert ((low / torch.finfo(dtype).min - 1).abs() <= 2.0 ** -20).all()


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}-{str(c[3])[6:]}-{len(c[4])}")
def test_gradients_with_masks(case):
    """Ids that cannot occur give and get nothing; the others are as without them."""
    hidden, head, tokens, keep = with_masks(*case)
    new_id = keep.cumsum(0) - 1
    rows, dtype = len(tokens), hidden.dtype
    e = Exact(hidden, head[keep], new_id[tokens])
    r = B.head_logprobs(hidden, head, tokens)
    off = e.off.amax(1)
    base = 2e-5 + 2.0 ** -22 * e.L
    # gradients, the entropy's large enough to pass the type's range with a masked logit
    gen = torch.Generator().manual_seed(rows)
    g = -(torch.rand(rows, generator=gen) + 0.5).to(DEV)
    for h in (None, torch.full((rows,), 3.0, device=DEV)):
        dx, dw = B.head_logprobs_backward(hidden, head, tokens, r.lse, r.entropy, g, h, lse_lo=r.lse_lo)
        assert (dw[~keep] == 0).all()
        c = g.double()[:, None]
        k = torch.zeros_like(c) if h is None else h.double()[:, None]
        spread = e.logp.abs() + e.H[:, None]
        G = -c * e.p - k * e.p * (e.logp + e.H[:, None])
        G.scatter_add_(1, new_id[tokens][:, None], c)
        # (test_head_gpu.py; the forward call's entropy may be off as above)
        p_off = 2 * e.off + (e.logp.abs() + 4 + e.L[:, None]) * 2.0 ** -22 + 2.0 ** -16
        H_off = (base + (4 * off + 2e-5) * e.H)[:, None]
        dG = c.abs() * e.p * p_off + k.abs() * e.p * ((spread + 1) * p_off + H_off + 2.0 ** -20 * spread)
        dG.scatter_add_(1, new_id[tokens][:, None], c.abs() * (p_off.amax(1, keepdim=True) + 2.0 ** -22))
        dG += (2.0 ** -8 if dtype == BF16 else 2.0 ** -23) * G.abs()
        for got, other, dGo, Go, n in ((dx, e.w, dG, G, len(e.w)), (dw[keep], e.a, dG.t(), G.t(), rows)):
            want = Go @ other
            tol = dGo @ other.abs() + (12 * n / 16 + 64) * 2.0 ** -23 * (Go.abs() @ other.abs())
            if dtype == BF16:
                tol += 2.0 ** -8 * want.abs()
            assert torch.isfinite(got).all()
            assert ((got.double() - want).abs() <= tol + 1e-37).all()
