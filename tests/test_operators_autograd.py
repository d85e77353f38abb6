"""Where gradients end at the operators beside the merge: said by an error, never
by a gradient that lacks a part. On the host with stand-ins for CUDA tensors and
kernels, and on the GPU."""
import pytest
import torch

from checkpoint_averaging_gb300 import binding as B
from checkpoint_averaging_gb300 import build as cam_build

gpu = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")


@pytest.fixture(scope="module", autouse=True)
def built():
    cam_build.build()


class OnGpu:
    """A host tensor that says it is a CUDA tensor."""

    def __init__(self, t):
        self.t = t

    is_cuda = True

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return 0

    def unsqueeze(self, dim):
        return OnGpu(self.t.unsqueeze(dim))


@pytest.fixture
def products(monkeypatch):
    """gemv4 without a GPU: how often the library was called."""
    from checkpoint_averaging_gb300 import operators as O

    made = []
    monkeypatch.setattr(O, "_current_stream", lambda device: 0)
    monkeypatch.setattr(O, "_current_device", lambda: 0)
    monkeypatch.setattr(O, "_empty", lambda shape, dtype, device: torch.empty(shape, dtype=dtype))
    monkeypatch.setattr(O, "_gemv4", lambda *args: made.append(args) or 0)
    data = OnGpu(torch.empty(B.pack4_bytes(20, 130, 64) + 16, dtype=torch.uint8))
    data.t = data.t[-data.t.data_ptr() % 16:][:B.pack4_bytes(20, 130, 64)]
    return B.Packed4(data, 20, 130, 64), made


@pytest.mark.parametrize("shape", [(130,), (1, 130), (3, 130)])
@pytest.mark.parametrize("more", [{}, {"out_dtype": torch.bfloat16}])
def test_products_refuse_an_x_that_requires_a_gradient(products, shape, more):
    w4, made = products
    x = OnGpu(torch.zeros(shape, requires_grad=True))
    with pytest.raises(ValueError, match="gradient"):
        B.gemv4(x, w4, **more)
    assert not made
    with torch.no_grad():
        assert B.gemv4(x, w4, **more).shape == (*shape[:-1], 20)
    assert B.gemv4(OnGpu(x.t.detach()), w4, **more).shape == (*shape[:-1], 20)
    assert len(made) == 2


@gpu
@needs_gpu
def test_a_4_bit_head_refuses_hidden_states_that_require_a_gradient():
    from checkpoint_averaging_gb300 import probe as P

    w = torch.randn(500, 64, generator=torch.Generator().manual_seed(1)).cuda()
    x = torch.randn(3, 64, generator=torch.Generator().manual_seed(2)).cuda()
    w4, tokens = B.pack4(w, 32), torch.tensor([1, 2, 3]).cuda()
    want = P.probe(x, w4, tokens, top=3)
    x.requires_grad_(True)
    with pytest.raises(ValueError, match="gradient"):
        P.probe(x, w4, tokens, top=3)
    with torch.no_grad():
        got = P.probe(x, w4, tokens, top=3)
    assert torch.equal(got.logp, want.logp) and torch.equal(got.top_ids, want.top_ids)
    assert P.head_logits(x, w).requires_grad


@pytest.fixture
def plain_kernels(monkeypatch):
    """The probe on the host: log probabilities and their gradient by torch, without a graph."""
    from types import SimpleNamespace

    from checkpoint_averaging_gb300 import probe as P

    def forward(logits, tokens):
        logp = torch.log_softmax(logits.detach(), 1)
        lse = torch.logsumexp(logits.detach(), 1)
        entropy = -(logp.exp() * logp).sum(1)
        return SimpleNamespace(logp=logp.gather(1, tokens[:, None])[:, 0], entropy=entropy, lse=lse,
                               lse_lo=torch.zeros_like(lse))

    def backward(logits, tokens, lse, entropy, g, h, *, lse_lo):
        with torch.no_grad():
            logp = logits - lse[:, None]
            p = logp.exp()
            out = torch.zeros_like(p)
            if g is not None:
                out -= g[:, None] * p
                out.scatter_add_(1, tokens[:, None], g[:, None])
            if h is not None:
                out -= h[:, None] * p * (logp + entropy[:, None])
            return out

    monkeypatch.setattr(P, "B", SimpleNamespace(token_logprobs=forward,
                                                token_logprobs_backward=backward))


def losses(logits, tokens, which):
    from checkpoint_averaging_gb300 import probe as P

    logp, entropy = P.differentiable_logprobs(logits, tokens)
    return {"logp": -logp.mean(), "entropy": entropy.sum(), "both": -logp.mean() + 0.1 * entropy.sum(),
            "square": (logp * logp).sum(), "other": -logp.mean() + (logits ** 3).sum()}[which]


def second_derivatives_are_refused(which, device):
    gen = torch.Generator().manual_seed(3)
    logits = torch.randn(4, 11, generator=gen).to(device).requires_grad_(True)
    tokens = torch.tensor([1, 5, 2, 9], device=device)
    once, = torch.autograd.grad(losses(logits, tokens, which), logits)
    assert not once.requires_grad
    first, = torch.autograd.grad(losses(logits, tokens, which), logits, create_graph=True)
    assert torch.equal(first.detach(), once)
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad((first * first).sum(), logits)
    with pytest.raises(RuntimeError, match="second derivative"):
        (losses(logits, tokens, which) + torch.autograd.grad(
            losses(logits, tokens, which), logits, create_graph=True)[0].norm()).backward()


@pytest.mark.parametrize("which", ["logp", "entropy", "both", "square", "other"])
def test_second_derivatives_are_refused(plain_kernels, which):
    second_derivatives_are_refused(which, "cpu")


@gpu
@needs_gpu
@pytest.mark.parametrize("which", ["logp", "entropy", "both", "square", "other"])
def test_second_derivatives_are_refused_on_the_gpu(which):
    second_derivatives_are_refused(which, "cuda")
