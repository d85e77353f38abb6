"""The operators for whole contexts together, as a user runs them: a merged global
published in 8 bits and probed, its loss without the logits, and the gradients through
autograd, against 64 bits (tolerances: test_head_gpu.py and test_pack8_gpu.py)."""
import pytest
import torch

from checkpoint_averaging_gb300 import binding as B
from checkpoint_averaging_gb300 import probe as P

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    yield
    torch.cuda.synchronize()
    assert B.operators_status() == 0


def inputs(rows, vocab, width, dtype, seed=3):
    gen = torch.Generator().manual_seed(seed)
    head = torch.randn(vocab, width, generator=gen) * 2.0 / width ** 0.5
    hidden = torch.randn(rows, width, generator=gen)
    tokens = torch.randint(0, vocab, (rows,), generator=gen)
    tokens[0] = -1
    return hidden.to(dtype).to(DEV), head.to(dtype).to(DEV), tokens.to(DEV)


def test_the_example_runs():
    eight, full, losses = P.main_contexts(vocab=3001, width=160, rows=250)
    assert len(losses) == 2 and all(x == x for x in losses)
    # a weight and a hidden state are off by 2^-4 of themselves (8 bits), a logit by
    # 2 * 2^-4 sum |x w| at most and by 2^-8 of itself in bf16, a log probability by twice its
    # row's largest
    assert eight.logp.shape == full.logp.shape == (250,)
    assert torch.isfinite(eight.logp).all() and torch.isfinite(full.logp).all()
    assert ((eight.logp == 0) == (full.logp == 0)).all()


def test_a_round_published_and_probed():
    """Merge, publish in 8 bits, probe a context by both forms of the new global."""
    vocab, width, rows = 2500, 192, 300
    hidden, head, tokens = inputs(rows, vocab, width, torch.float32)
    theta = [head.clone()]
    m = B.Merger(theta, quorum=2)
    rd = m.begin(0)
    for scale in (0.01, -0.02):
        rd.accumulate([head + scale * head.flip(0)], 1000)
    rd.finalize(B.MEAN_REPLACE)
    rd.commit()
    w8 = B.pack8(theta[0])
    got = P.probe(hidden, w8, tokens, top=3)
    a, w = B.unpack8(B.pack8(hidden)).double(), B.unpack8(w8).double()
    x = a @ w.t()
    logp = torch.log_softmax(x, 1)
    off = (2 * width / 32 + 16) * 2.0 ** -23 * (a.abs() @ w.abs().t()).amax(1)
    tol = 2 * off + 2e-5 + 2.0 ** -22 * x.abs().amax(1)
    mine = logp.gather(1, tokens.clamp(min=0)[:, None])[:, 0] * (tokens >= 0)
    assert ((got.logp.double() - mine).abs() <= tol).all()
    assert ((got.top_logp.double() - logp.topk(3, 1).values).abs() <= tol[:, None]).all()
    full = P.context_loss(hidden, theta[0], tokens)
    x = hidden.double() @ theta[0].double().t()
    off = (12 * width / 16 + 16) * 2.0 ** -23 * (hidden.double().abs() @ theta[0].double().abs().t()).amax(1)
    tol = 2 * off + 2e-5 + 2.0 ** -22 * x.abs().amax(1)
    mine = torch.log_softmax(x, 1).gather(1, tokens.clamp(min=0)[:, None])[:, 0] * (tokens >= 0)
    assert ((full.logp.double() - mine).abs() <= tol).all()
    assert abs(float(full.loss) + float(mine.sum() / (tokens >= 0).sum())) <= float(tol.max()) * 1.01
    m.close()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [9, 200])
def test_a_loss_through_autograd(rows, dtype):
    hidden, head, tokens = inputs(rows, 1500, 96, dtype)
    want_a, want_w = hidden.double().requires_grad_(True), head.double().requires_grad_(True)
    logp = torch.log_softmax(want_a @ want_w.t(), 1)
    entropy = -(logp.exp() * logp).sum(1)
    mine = logp.gather(1, tokens.clamp(min=0)[:, None])[:, 0] * (tokens >= 0)
    (-mine.mean() + 0.1 * entropy.sum()).backward()
    a, w = hidden.clone().requires_grad_(True), head.clone().requires_grad_(True)
    lp, h = P.differentiable_head_logprobs(a, w, tokens)
    (-lp.mean() + 0.1 * h.sum()).backward()
    # |G| is off by (1e-4 + its rounding) of itself and of p (|g| + |h| (|log p| + H + 1)), the
    # result by that through |head| or |hidden| and by its own rounding (test_head_gpu.py)
    p = logp.detach().exp()
    scale = p * (1 / rows + 0.1 * (logp.detach().abs() + entropy.detach()[:, None] + 1))
    scale.scatter_add_(1, tokens.clamp(min=0)[:, None], torch.full((rows, 1), 1 / rows, device=DEV).double())
    rel = 2.0 ** -8 + 1e-4 if dtype == torch.bfloat16 else 1e-4
    for got, want, off in ((a, want_a, scale @ head.double().abs()), (w, want_w, scale.t() @ hidden.double().abs())):
        tol = rel * off + (2.0 ** -8 * want.grad.abs() if dtype == torch.bfloat16 else 0)
        assert got.grad.dtype == dtype
        assert ((got.grad.double() - want.grad).abs() <= tol).all()
    # what requires no gradient gets none, and the other is the same
    only = hidden.clone().requires_grad_(True)
    lp, h = P.differentiable_head_logprobs(only, head, tokens)
    (-lp.mean() + 0.1 * h.sum()).backward()
    assert torch.equal(only.grad, a.grad) and head.grad is None
    # a loss that leaves one of the two out
    only = head.clone().requires_grad_(True)
    P.differentiable_head_logprobs(hidden, only, tokens)[1].sum().backward()
    assert torch.isfinite(only.grad).all() and float(only.grad.abs().max()) > 0


@pytest.mark.parametrize("which", ["logp", "entropy", "square"])
def test_second_derivatives_are_refused(which):
    hidden, head, tokens = inputs(5, 300, 64, torch.float32)
    hidden.requires_grad_(True)
    head.requires_grad_(True)

    def loss():
        logp, entropy = P.differentiable_head_logprobs(hidden, head, tokens)
        return {"logp": -logp.mean(), "entropy": entropy.sum(), "square": (logp * logp).sum()}[which]

    once = torch.autograd.grad(loss(), (hidden, head))
    first = torch.autograd.grad(loss(), (hidden, head), create_graph=True)
    assert all(torch.equal(x, y.detach()) for x, y in zip(once, first))
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad((first[0] * first[0]).sum(), hidden)
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(first[1].sum(), head)


def test_a_captured_step():
    hidden, head, tokens = inputs(150, 900, 96, torch.bfloat16)
    a, w = hidden.clone().requires_grad_(True), head.clone().requires_grad_(True)

    def step():
        logp, entropy = P.differentiable_head_logprobs(a, w, tokens)
        return torch.autograd.grad(-logp.mean() + 0.1 * entropy.mean(), (a, w))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    with torch.no_grad():
        a.copy_(hidden.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    want = step()
    assert all(torch.equal(x, y) for x, y in zip(out, want))


def test_an_8_bit_head_refuses_hidden_states_that_require_a_gradient():
    hidden, head, tokens = inputs(5, 300, 64, torch.float32)
    w8 = B.pack8(head)
    want = P.probe(hidden, w8, tokens, top=2)
    hidden.requires_grad_(True)
    with pytest.raises(ValueError, match="gradient"):
        P.probe(hidden, w8, tokens, top=2)
    with torch.no_grad():
        assert torch.equal(P.probe(hidden, w8, tokens, top=2).logp, want.logp)
    with pytest.raises(ValueError, match="differentiable_head_logprobs"):
        P.context_loss(hidden, head, tokens)
