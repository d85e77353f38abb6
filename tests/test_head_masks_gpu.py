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
