"""The operators together (checkpoint_averaging_gb300.probe): a merged global
published in 4 bits, answered from, probed, and trained on from there."""
import pytest
import torch

from checkpoint_averaging_gb300 import binding as B
from checkpoint_averaging_gb300 import probe as P

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    yield
    torch.cuda.synchronize()


def test_the_example_runs_and_its_heads_agree():
    found, losses = P.main(vocab=2000, width=320, rows=9)
    assert losses[1] < losses[0]
    for a in ("global", "EMA"):
        full, four = found[a], found[a + ", 4 bits"]
        # a logit moves by sum (step / 2) |x| at most, step = the group's scale; every log
        # probability by twice that
        bound = 2 * 320 * (0.05 * 6 / 7 / 2) * (6 * 0.05 * 6)
        assert (full.logp - four.logp).abs().max() < bound
        assert full.logp[-1] == 0 and four.logp[-1] == 0
        assert full.top_ids.shape == (9, 5)
        # the leading token has a margin that 4 bits do not close
        assert torch.equal(full.top_ids[:-1, 0], four.top_ids[:-1, 0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_loss_through_autograd(dtype):
    gen = torch.Generator().manual_seed(4)
    x = (torch.randn(7, 3001, generator=gen) * 2).to(dtype)
    tokens = torch.randint(0, 3001, (7,), generator=gen)
    want_x = x.double().requires_grad_(True)
    logp = torch.log_softmax(want_x, 1)
    entropy = -(logp.exp() * logp).sum(1)
    want = -logp[torch.arange(7), tokens].mean() + 0.1 * entropy.sum()
    want.backward()
    got_x = x.cuda().requires_grad_(True)
    lp, h = P.differentiable_logprobs(got_x, tokens.cuda())
    got = -lp.mean() + 0.1 * h.sum()
    got.backward()
    # 2e-5 on each row's log probability and entropy (test_logprobs_gpu.py), entropies near 6
    assert abs(float(got.detach()) - float(want.detach())) < 2e-5 * (1 + 0.1 * 7 * 8)
    # 1e-4 of p (|g| + |h| (|log p| + H)) and the result's own rounding
    p = logp.detach().exp()
    scale = 1e-4 * p * (1 / 7 + 0.1 * (logp.detach().abs() + entropy.detach()[:, None]))
    scale += 2.0 ** -22 / 7 + (2.0 ** -8 * want_x.grad.abs() if dtype == torch.bfloat16 else 0)
    assert got_x.grad.dtype == dtype
    assert ((got_x.grad.cpu().double() - want_x.grad).abs() <= scale).all()
    # a loss that leaves one of the two out
    only = x.cuda().requires_grad_(True)
    P.differentiable_logprobs(only, tokens.cuda())[1].sum().backward()
    assert torch.isfinite(only.grad).all() and float(only.grad.abs().max()) > 0


def test_probe_takes_either_head():
    gen = torch.Generator().manual_seed(1)
    w = torch.randn(500, 64, generator=gen).cuda()
    x = torch.randn(3, 64, generator=gen).cuda()
    tokens = torch.tensor([1, 2, 3]).cuda()
    packed = B.pack4(w, 32)
    a = P.probe(x, B.unpack4(packed), tokens, top=3)
    b = P.probe(x, packed, tokens, top=3)
    assert torch.equal(a.top_ids, b.top_ids)
    assert abs(float(a.loss) - float(b.loss)) < 1e-3


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab,width", [(9, 2000, 320), (1, 8192, 512), (40, 3001, 130)])
def test_a_published_head_is_probed_as_its_values(rows, vocab, width, dtype):
    gen = torch.Generator().manual_seed(vocab)
    w = torch.randn(vocab, width, generator=gen) * 0.05
    x = (torch.randn(rows, width, generator=gen) * 2).to(dtype).cuda()
    tokens = torch.randint(0, vocab, (rows,), generator=gen).cuda()
    tokens[-1] = -1 if rows > 1 else tokens[-1]
    packed = B.pack4(w.cuda(), 64)
    got = P.probe(x, packed, tokens, top=5)
    value = B.unpack4(packed).double()
    logits = x.double() @ value.t()
    logp = torch.log_softmax(logits, 1)
    entropy = -(logp.exp() * logp).sum(1)
    # a product is off by (width / 32 + 96) 2^-22 sum |s q x| and 2^-8 of itself in bf16
    # (test_pack4_gemv4_gpu.py), a log probability by twice its row's largest and by
    # 2e-5 + 2^-22 of the largest logit (test_logprobs_gpu.py)
    mag = x.double().abs() @ value.abs().t()
    off = ((width / 32 + 96) * 2.0 ** -22 * mag).amax(1)
    if dtype == torch.bfloat16:
        off += 2.0 ** -8 * logits.abs().amax(1)
    tol = 2 * off + 2e-5 + 2.0 ** -22 * logits.abs().amax(1)
    known = tokens >= 0
    mine = logp.gather(1, tokens.clamp(min=0)[:, None])[:, 0] * known
    assert ((got.logp.double() - mine).abs() <= tol).all()
    assert abs(float(got.loss) + float(mine.sum() / known.sum())) <= float(tol.max()) * 1.01
    assert ((got.top_logp.double() - logp.gather(1, got.top_ids)).abs() <= tol[:, None]).all()
    assert ((got.top_logp.double() - logp.topk(5, 1).values).abs() <= tol[:, None]).all()
    # |dH| <= sum |dp| (|log p| + H) with |dp| <= 2 off p: at most 4 off H
    assert (got.entropy.double() - entropy.mean()).abs() <= (tol + 4 * off * entropy + 2e-5 * entropy).max()
