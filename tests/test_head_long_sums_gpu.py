"""The head's gradient as a sum over very many rows, on the GPU against 64 bits."""
import pytest
import torch

from checkpoint_averaging_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    yield
    torch.cuda.synchronize()
    assert B.operators_status() == 0
    torch.cuda.empty_cache()


def test_sums_over_many_rows_do_not_lean():
    """A head of zeros: p = 1 / vocab and G = 1 / vocab for a g of -1, exactly, so that the
    head's gradient is a sum of positive bf16 numbers. The tensor core's additions lean to zero;
    the results' mean is off by what they lose, the results' own roundings (2^-8 of
    each at most, either way) average out: 4 sigma of 2^-8 / sqrt(3) per result, which are columns of different scales. The sums are
    cut into runs of at most 8,192 terms, 512 additions of at most 2^-23 of what has been summed,
    a half of the whole in the mean."""
    rows, width, vocab = 1 << 19, 8192, 512
    gen = torch.Generator(device=DEV).manual_seed(rows)
    hidden = torch.empty(rows, width, dtype=torch.bfloat16, device=DEV)
    # (scales of the columns that are not bf16 numbers: else the results, 1,024 times the scale and
    # a little, would all lie at one place between two bf16 numbers, and round one way)
    scale = 1 + torch.arange(width, device=DEV) / width
    for part in hidden.split(1 << 14):
        part.copy_(torch.empty(part.shape, device=DEV).uniform_(0.5, 1.5, generator=gen) * scale)
    head = torch.zeros(vocab, width, dtype=torch.bfloat16, device=DEV)
    tokens = torch.zeros(rows, dtype=torch.int64, device=DEV)
    r = B.head_logprobs(hidden, head, tokens)
    g = torch.full((rows,), -1.0, device=DEV)
    _, got = B.head_logprobs_backward(hidden, head, tokens, r.lse, r.entropy, g, lse_lo=r.lse_lo,
                                      need_hidden=False)
    want = torch.zeros(width, dtype=torch.float64, device=DEV)
    for part in hidden.split(1 << 14):
        want += part.double().sum(0)
    want /= vocab
    rel = (got[1:].double() / want - 1).mean(0)  # (every id's gradient is the same sum)
    lean = float(rel.mean())
    assert abs(lean) <= 256 * 2.0 ** -23 + 4 * 2.0 ** -8 / 3 ** 0.5 / width ** 0.5, lean
