"""The example for whole contexts (probe.main_contexts) against 64 bits: its loss without
logits, its probe of the 8-bit head, and its step along the gradients."""
import torch
import pytest

from checkpoint_averaging_gb300 import binding as B
from checkpoint_averaging_gb300 import probe as P

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    yield
    torch.cuda.synchronize()
    assert B.operators_status() == 0


def inputs(vocab, width, rows, seed):
    """The example's, from its seed."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    head = torch.empty(vocab, width, device="cuda").normal_(0.0, 0.05, generator=gen)
    tokens = torch.randint(0, vocab, (rows,), device="cuda", generator=gen)
    hidden = head[tokens] * 3.0 + torch.empty(rows, width, device="cuda").normal_(0.0, 0.3, generator=gen)
    tokens[::10] = -1
    return hidden, head, tokens


def mine(logits, tokens):
    logp = torch.log_softmax(logits, 1)
    return logp, logp.gather(1, tokens.clamp(min=0)[:, None])[:, 0] * (tokens >= 0)


@pytest.mark.parametrize("vocab,width,rows,seed", [(3001, 160, 250, 0), (1000, 512, 40, 7)])
def test_the_example_against_64_bits(vocab, width, rows, seed):
    eight, full, losses = P.main_contexts(vocab, width, rows, seed)
    hidden, head, tokens = inputs(vocab, width, rows, seed)
    # without logits, bf16 inputs: test_head_gpu.py
    a, w = hidden.bfloat16().double(), head.bfloat16().double()
    x, size = a @ w.t(), a.abs() @ w.abs().t()
    off = ((12 * width / 16 + 16) * 2.0 ** -23 * size).amax(1)
    logp = mine(x, tokens)[1]
    assert ((full.logp.double() - logp).abs() <= 2e-5 + 2.0 ** -22 * x.abs().amax(1) + 2 * off).all()
    # in 8 bits: weights and hidden states are off by 2^-4 of themselves and by 2^-10 of their
    # block's scale, at most 2^-17 of its largest value (2^-10 * 2^e, the largest above 224 * 2^e);
    # the weights are packed from fp32, the others' bf16 ones are 2^-8 off; the logits are
    # rounded to bf16, and a log probability is off by twice its row's largest
    rel = (1 + 2.0 ** -4) ** 2 * (1 + 2.0 ** -8) - 1
    small = 2.0 ** -17 * 1.1 * (a.abs().amax(1) * w.abs().sum(1).max() + a.abs().sum(1) * w.abs().max())
    logit = (rel * size).amax(1) + small
    logit = logit + 2.0 ** -8 * (x.abs().amax(1) + logit)
    assert ((eight.logp.double() - logp).abs() <= 2 * logit + 2e-5 + 2.0 ** -22 * x.abs().amax(1)).all()
    # the fp32 step
    s, v = hidden.double().requires_grad_(True), head.double().requires_grad_(True)
    want = []
    for _ in range(2):
        lp, own = mine(s @ v.t(), tokens)
        entropy = -(lp.exp() * lp).sum(1)
        loss = -own.sum() / (tokens >= 0).sum() + 0.01 * entropy.mean()
        want.append(float(loss.detach()))
        if len(want) == 1:
            loss.backward()
            s, v = (s - 0.5 * s.grad).detach(), (v - 0.5 * v.grad).detach()
    off = ((12 * width / 16 + 16) * 2.0 ** -23 * (s.abs() @ v.abs().t())).amax()
    tol = float(2e-5 + 2.0 ** -22 * (s @ v.t()).abs().max() + 2 * off) + 0.01 * float(5 * off + 2e-5) * 10
    # (the gradients of the step are off by 1e-4 of themselves, test_contexts_autograd_gpu.py, the
    # loss after it by that times the squared length of the step's gradient)
    assert abs(losses[0] - want[0]) <= tol
    assert abs(losses[1] - want[1]) <= tol + 1e-4 * abs(want[0] - want[1]) * 2
