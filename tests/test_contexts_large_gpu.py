"""The operators for whole contexts where offsets pass 32 bits, with long rows, large
vocabularies, and a first call while a graph is captured."""
import subprocess
import sys

import pytest
import torch

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
    torch.cuda.empty_cache()


def randn(rows, cols, dtype, seed, scale=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.empty(rows, cols, device=DEV, dtype=dtype).normal_(0.0, scale, generator=gen)


@pytest.mark.parametrize("rows", [70016, 70013])  # rows of results that TMA stores, and others
def test_products_of_more_than_2_to_the_32_bytes(rows):
    tokens, cols = 33000, 64  # 2.3e9 results
    x, w = randn(tokens, cols, BF16, 1), randn(rows, cols, BF16, 2)
    w8 = B.pack8(w)
    y = B.matmul8(x, w8)
    last = slice(tokens - 700, tokens)
    assert torch.equal(y[last], B.matmul8(x[last], w8))  # a row's result is its own
    assert torch.equal(y[:300], B.matmul8(x[:300], w8))
    short = B.pack8(w[rows - 192 * 2:])
    assert torch.equal(y[last, rows - 384:], B.matmul8(x[last], short))


def test_matrices_of_more_than_2_to_the_32_bytes():
    rows, cols = 2_200_000, 1000
    w = randn(rows, cols, BF16, 3)
    w8 = B.pack8(w)
    back = B.unpack8(w8, BF16)
    for at in (0, 1_073_741, 2_147_483, rows - 1000):
        part = B.unpack8(B.pack8(w[at:at + 1000]), BF16)
        assert torch.equal(back[at:at + 1000], part)


@pytest.mark.parametrize("dtype,rows", [(BF16, 3), (BF16, 300), (F32, 3)])
def test_heads_of_more_than_2_to_the_32_bytes(dtype, rows):
    vocab, width = (1_100_000, 2048) if dtype == BF16 else (1_100_000, 1024)
    head = randn(vocab, width, dtype, 4, 2.0 / width ** 0.5)
    hidden = randn(rows, width, dtype, 5)
    tokens = torch.arange(rows, device=DEV) * 3000 + (vocab - 1 - 3000 * rows)
    r = B.head_logprobs(hidden, head, tokens)
    cut = 600_000
    a = B.head_logprobs(hidden, head[:cut], tokens.where(tokens < cut, -1))
    b = B.head_logprobs(hidden, head[cut:], tokens - cut)  # (a token of the first part is none of the second)
    lse = torch.logaddexp(a.lse.double() + a.lse_lo, b.lse.double() + b.lse_lo)
    # two sums of the same products, each within 2e-5 + 2^-22 of the logits (test_head_gpu.py)
    assert (r.lse.double() + r.lse_lo - lse).abs().max() < 1e-4
    mine = torch.where(tokens < cut, a.logp.double() + a.lse.double() + a.lse_lo,
                       b.logp.double() + b.lse.double() + b.lse_lo)
    assert (r.logp.double() - (mine - lse)).abs().max() < 1e-4
    g = torch.full((rows,), -1.0, device=DEV)
    gx, gw = B.head_logprobs_backward(hidden, head, tokens, r.lse, r.entropy, g, lse_lo=r.lse_lo)
    # the rows of the head near its end, from their logits alone
    at = vocab - 5000
    p = (hidden.double() @ head[at:].double().t() - lse[:, None]).exp()
    G = p.clone()
    known = tokens >= at
    G[known, (tokens - at)[known]] -= 1.0
    want = G.t() @ hidden.double()
    size = G.abs().t() @ hidden.double().abs()
    rel = 2.0 ** -7 if dtype == BF16 else 1e-4
    assert ((gw[at:].double() - want).abs() <= rel * size + 1e-30).all()
    assert torch.isfinite(gx).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,vocab,width", [(3, 500, 20011), (150, 300, 20000), (2, 300_001, 70), (5000, 70, 64)])
def test_long_rows_and_large_vocabularies(rows, vocab, width, dtype):
    from test_head_gpu import Exact, check, check_grad, inputs

    hidden, head, tokens = inputs(rows, vocab, width, dtype)
    e = Exact(hidden, head, tokens)
    check(hidden, head, tokens, e=e)
    check_grad(hidden, head, tokens, e=e)


@pytest.mark.parametrize("rows", [5, 100, 300])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_a_first_call_while_a_graph_is_captured(rows, dtype):
    code = f"""
import torch
from checkpoint_averaging_gb300 import binding as B
gen = torch.Generator().manual_seed(1)
hidden = torch.randn({rows}, 96, generator=gen).to(torch.{dtype}).cuda()
head = torch.randn(700, 96, generator=gen).to(torch.{dtype}).cuda() * 0.2
tokens = torch.arange({rows}).cuda()
g = torch.full(({rows},), -1.0).cuda()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
def step():
    r = B.head_logprobs(hidden, head, tokens)
    return (r._stats, *B.head_logprobs_backward(hidden, head, tokens, r.lse, r.entropy, g, lse_lo=r.lse_lo),
            B.matmul8(hidden, B.pack8(head)))
with torch.cuda.graph(graph):
    out = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(out, step()))
assert B.operators_status() == 0
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
