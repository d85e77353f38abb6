"""Log probabilities of given tokens, their entropy and top alternatives, and
the gradient, on the GPU against the definitions in 64 bits (include/cam.h).

Tolerances, absolute, with x the row's finite logits and L the largest of
|x| and |lse|. Forward: a term exp(x - M) has a relative error of at most
2^-22 (the exponential) + |x - M| 2^-22 (its argument); the terms that matter
have |x - M| < 32, and sums of 512 threads' fp32 partial sums add 2^-24 for
each of at most 200 additions in a row: 33 2^-22 + 200 2^-24 < 2e-5 relative
on s and t, so 2e-5 on log s, 2e-5 (1 + H) on the entropy with t / s <= H, and
the last subtractions round by 2^-23 L each. Backward: p = exp(x - lse) has
(1 + |x - lse| + L) 2^-22 < 1e-4 relative with |x - lse|, L < 300, so
1e-4 p (|g| + |h| (|log p| + H)) + 2^-22 |g|, and a bf16 result 2^-8 of itself.
Ids are exact: logits are compared as they are given.
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


def definition(x, tokens, top):
    """In 64 bits on the CPU: logp, entropy, lse, top_logp, top_ids."""
    x = x.double().cpu()
    R, V = x.shape
    bad = torch.isnan(x).any(1) | (x == INF).any(1)
    dead = (x == -INF).all(1)
    lse = torch.logsumexp(x, 1)
    logp = x - lse[:, None]
    H = torch.special.entr(logp.exp()).sum(1)
    logp[dead] = -INF
    H[dead] = 0.0
    for v in (lse, H):
        v[bad] = math.nan
    logp[bad] = math.nan
    ids = None
    best = None
    if top:
        # torch's stable descending sort puts NaN first and equals in the order of their ids
        ids = torch.sort(x + 0.0, dim=1, descending=True, stable=True).indices[:, :top]
        best = torch.gather(logp, 1, ids)
    mine = None
    if tokens is not None:
        tokens = tokens.cpu()
        mine = logp[torch.arange(R), tokens.clamp(0, V - 1)]
        mine = torch.where(tokens < 0, 0.0, torch.where(tokens >= V, math.nan, mine))
    return mine, H, lse, best, ids


def close(got, want, tol):
    got = got.cpu().double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)])
    off = (got - want).abs()[fine] - (tol if not torch.is_tensor(tol) else tol.expand_as(want)[fine])
    assert not off.numel() or off.max() <= 0, off.max()


def check(x, tokens, top):
    r = B.token_logprobs(x, tokens, top=top)
    mine, H, lse, best, ids = definition(x, tokens, top)
    finite = x.float().cpu().masked_fill(~torch.isfinite(x.float().cpu()), 0.0)
    L = torch.maximum(finite.abs().amax(1).double(), lse.abs().nan_to_num(0.0, 0.0, 0.0))
    base = 2e-5 + 2.0 ** -22 * L
    if tokens is None:
        assert r.logp is None
    else:
        close(r.logp, mine, base)
    close(r.entropy, H, base + 2e-5 * H.nan_to_num(0.0))
    close(r.lse, lse, base)
    if top:
        assert r.top_ids.dtype == torch.int64
        assert torch.equal(r.top_ids.cpu(), ids)
        close(r.top_logp, best, base[:, None])
    else:
        assert r.top_ids is None and r.top_logp is None
    return r


def logits(rows, vocab, seed, dtype=torch.float32, spread=2.5):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, vocab, generator=g) * spread).to(dtype)
    return x.to(DEV), torch.randint(0, vocab, (rows,), generator=g).to(DEV)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab,top", [
    (1, 1, 1), (3, 2, 2), (5, 7, 3), (4, 33, 32), (2, 100, 0), (7, 129, 5), (3, 1000, 20),
    (2, 4095, 1), (2, 4097, 32), (1, 50304, 5), (5, 50257, 10), (160, 20481, 3), (2, 73760, 32),
    (300, 2049, 7), (1, 131071, 10), (2, 300001, 10)])
def test_log_probabilities(rows, vocab, top, dtype):
    x, tokens = logits(rows, vocab, rows + vocab, dtype)
    if rows > 2:
        tokens[1] = -1
    a = check(x, tokens, top)
    b = B.token_logprobs(x, tokens, top=top)
    for u, v in zip(a, b):
        assert u is None or torch.equal(u, v)  # the same bits again


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab,top", [
    (3000, 1001, 20), (2700, 4003, 5), (1300, 9001, 32), (1300, 16385, 1), (700, 33001, 10)])
def test_many_rows_of_every_kind(rows, vocab, top, dtype):
    # rows enough that a block takes several, or that each is held by as few threads as can
    x, tokens = logits(rows, vocab, vocab, dtype)
    k = torch.arange(rows, device=DEV) % 16
    x[k == 1, vocab // 2] = 60.0                 # confident
    x[k == 2, vocab - 1] = 90.0
    x[k == 3, 1:] = -INF                         # one token left
    x[k == 4] = -INF
    x[k == 5, vocab // 3] = math.nan
    x[k == 6, 0] = INF
    x[k == 7] = 1.25                             # all equal
    x[k == 8] = torch.floor(x[k == 8])           # many equal
    x[k == 9, ::3] = torch.finfo(dtype).min
    x[k == 10] *= 1e37
    x[k == 11] = torch.finfo(dtype).min
    x[k == 12, 40:] = -INF
    tokens[k == 13] = -1
    tokens[k == 14] = vocab
    r = B.token_logprobs(x, tokens, top=top)
    at = torch.cat([torch.arange(48), torch.arange(48, rows, 61), torch.arange(rows - 16, rows)])
    mine, H, lse, best, ids = definition(x[at.to(DEV)], tokens[at.to(DEV)], top)
    finite = x[at.to(DEV)].float().cpu().masked_fill(~torch.isfinite(x[at.to(DEV)].float().cpu()), 0.0)
    L = torch.maximum(finite.abs().amax(1).double(), lse.abs().nan_to_num(0.0, 0.0, 0.0))
    base = 2e-5 + 2.0 ** -22 * L
    got = [v.cpu()[at] for v in (r.logp, r.entropy, r.lse, r.top_logp, r.top_ids)]
    close(got[0], mine, base)
    close(got[1], H, base + 2e-5 * H.nan_to_num(0.0))
    close(got[2], lse, base)
    assert torch.equal(got[4], ids)
    close(got[3], best, base[:, None])


def test_without_tokens_and_with_strides():
    x, tokens = logits(6, 5000, 1)
    check(x, None, 4)
    wide, _ = logits(6, 6100, 2, torch.bfloat16)
    for at in range(0, 9):
        check(wide[:, at:at + 5003], tokens, 5)
    wide, _ = logits(6, 5101, 3)
    for at in range(0, 5):
        check(wide[:, at:at + 4000 + at], tokens.clamp(max=3999), 5)
    assert B.token_logprobs(x[:0], tokens[:0], top=3).top_ids.shape == (0, 3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [50, 9000, 73760])
def test_masked_rows(vocab, dtype):
    x, tokens = logits(8, vocab, 11, dtype)
    x[0] = -INF                                  # nothing left
    x[1, :] = -INF
    x[1, vocab // 2] = 3.0                       # one token left
    x[2, : vocab - 3] = -INF
    x[3, 1::2] = -INF
    tokens[3] = 1                                # a masked token: logp = -inf
    x[4] = torch.finfo(dtype).min                # masked by the type's lowest value alone
    x[5] = torch.finfo(dtype).min
    x[5, 7] = 0.0
    x[6] = torch.finfo(dtype).max
    tokens[1] = vocab // 2
    r = check(x, tokens, 12)
    assert r.logp[0] == -INF and r.entropy[0] == 0 and r.lse[0] == -INF
    assert r.top_ids[0].tolist() == list(range(12))
    assert r.logp[1] == 0 and r.entropy[1] == 0 and r.lse[1] == 3 and r.logp[3] == -INF
    assert abs(r.entropy[4].item() - math.log(vocab)) < 1e-4


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [40, 9000, 73760])
def test_rows_with_nan_and_infinities(vocab, dtype):
    x, tokens = logits(6, vocab, 12, dtype)
    x[0, vocab - 1] = math.nan
    x[1, 5] = -math.nan
    x[1, 30] = INF
    x[2, 17] = INF
    x[3, :] = math.nan
    x[4, 20] = INF
    x[4, 3] = -INF
    x[4, 0] = INF
    tokens[4] = 20
    check(x, tokens, 9)


@pytest.mark.parametrize("vocab", [64, 5000, 50304])
def test_equal_logits_come_in_the_order_of_their_ids(vocab):
    x = torch.zeros(5, vocab)
    x[0, 1::2] = -0.0                            # -0 is 0
    x[1] = 2.5
    x[2] = torch.arange(vocab) % 3
    x[3] = torch.arange(vocab).float()           # ascending
    x[4] = -torch.arange(vocab).float()          # descending
    tokens = torch.arange(5)
    for dtype in (torch.float32, torch.bfloat16):
        for top in (1, 20, 32):
            check(x.to(dtype).to(DEV), tokens.to(DEV), top)


def test_tokens_outside_the_vocabulary():
    x, tokens = logits(5, 300, 4)
    tokens[:] = torch.tensor([0, 299, 300, -100, 1 << 40])
    r = check(x, tokens, 0)
    assert torch.isnan(r.logp[[2, 4]]).all() and r.logp[3] == 0


def test_a_confident_row_keeps_its_small_loss():
    # log s = log(1 + r) with r far below 2^-24: s itself would round to 1
    x = torch.full((1, 1000), -40.0)
    x[0, 3] = 0.0
    r = B.token_logprobs(x.to(DEV), torch.tensor([3], device=DEV))
    want = -math.log1p(999 * math.exp(-40.0))
    assert abs(r.logp.item() - want) <= 1e-5 * abs(want)
    want_h = 999 * math.exp(-40.0) * 40.0 + 999 * math.exp(-40.0)
    assert abs(r.entropy.item() - want_h) <= 1e-5 * want_h


def gradient(x, tokens, g, h):
    x = x.double().cpu()
    R, V = x.shape
    tokens = None if tokens is None else tokens.cpu()
    logp = torch.log_softmax(x, 1)
    p = logp.exp()
    out = torch.zeros_like(x)
    scale = torch.zeros_like(x)
    if g is not None:
        g = g.double().cpu() * (tokens >= 0)
        out -= g[:, None] * p
        out[torch.arange(R), tokens.clamp(min=0)] += g
        scale += 1e-4 * p * g.abs()[:, None] + 2.0 ** -22 * g.abs()[:, None]
    if h is not None:
        h = h.double().cpu()
        H = torch.special.entr(p).sum(1, keepdim=True)
        out -= h[:, None] * (p * H - torch.special.entr(p))
        scale += 1e-4 * h.abs()[:, None] * (p * H + torch.special.entr(p).abs())
    return out, scale


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (2, 3), (5, 7), (4, 1000), (3, 8193), (16, 50304),
                                        (2, 50257), (3, 131071)])
@pytest.mark.parametrize("which", ["logp", "entropy", "both"])
def test_gradient_is_the_formula(rows, vocab, dtype, which):
    x, tokens = logits(rows, vocab, 3 * rows + vocab, dtype)
    x[0, vocab // 2:vocab // 2 + 1] += 9.0
    if rows > 1:
        tokens[1] = -1
        if vocab > 4:
            x[1, 2:4] = -INF
    gen = torch.Generator().manual_seed(1)
    g = torch.randn(rows, generator=gen).to(DEV) if which != "entropy" else None
    h = torch.randn(rows, generator=gen).to(DEV) if which != "logp" else None
    r = B.token_logprobs(x, tokens)
    got = B.token_logprobs_backward(x, tokens, r.lse, r.entropy, g, h, lse_lo=r.lse_lo)
    want, tol = gradient(x, tokens, g, h)
    assert got.dtype == dtype
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs()
    assert ((got.cpu().double() - want).abs() <= tol + 1e-12).all()
    assert torch.equal(got, B.token_logprobs_backward(x, tokens, r.lse, r.entropy, g, h, lse_lo=r.lse_lo))
    same = x.clone()
    assert B.token_logprobs_backward(same, tokens, r.lse, r.entropy, g, h, lse_lo=r.lse_lo, out=same) is same
    assert torch.equal(same, got)


def test_gradient_is_the_difference_quotient():
    # central differences of g logp + h H in 64 bits: their error is about
    # step^2 times the third derivative (below 10 here) + 1e-16 / step
    x, tokens = logits(3, 11, 8)
    gen = torch.Generator().manual_seed(2)
    g, h = torch.randn(3, generator=gen), torch.randn(3, generator=gen)
    r = B.token_logprobs(x, tokens)
    got = B.token_logprobs_backward(x, tokens, r.lse, r.entropy, g.to(DEV), h.to(DEV),
                                    lse_lo=r.lse_lo).cpu().double()

    def f(z):
        mine, H, _, _, _ = definition(z, tokens, 0)
        return g.double() * mine + h.double() * H

    step = 1e-4
    base = x.cpu().double()
    for j in range(11):
        e = torch.zeros_like(base)
        e[:, j] = step
        want = (f(base + e) - f(base - e)) / (2 * step)
        assert ((got[:, j] - want).abs() <= 1e-6 + 1e-4 * want.abs()).all()


def test_gradient_of_rows_without_one():
    x, tokens = logits(7, 900, 6)
    x[0] = -INF
    x[1, 5] = math.nan
    x[2, 5] = math.nan
    x[4, 800] = INF
    tokens[3] = -1
    tokens[5] = 900
    g = torch.ones(7, device=DEV)
    g[2] = 0.0
    r = B.token_logprobs(x, tokens)
    got = B.token_logprobs_backward(x, tokens, r.lse, r.entropy, g)
    assert (got[[0, 2, 3]] == 0).all()
    assert torch.isnan(got[[1, 4, 5]]).all()
    assert torch.isfinite(got[6]).all()
    h = torch.zeros(7, device=DEV)
    h[3] = 1.0
    got = B.token_logprobs_backward(x, None, r.lse, r.entropy, None, h)
    assert (got[[0, 1, 2, 4, 5, 6]] == 0).all()
    want, tol = gradient(x[3:4], None, None, h[3:4])
    assert ((got[3:4].cpu().double() - want).abs() <= tol + 1e-12).all()


def test_gradient_strides_and_alignments():
    wide, tokens = logits(5, 4200, 9, torch.bfloat16)
    g = torch.ones(5, device=DEV)
    for at, to in ((0, 0), (1, 1), (3, 3), (1, 2), (0, 5)):
        x = wide[:, at:at + 4003]
        tk = tokens.clamp(max=4002)
        r = B.token_logprobs(x, tk)
        room = torch.full((5, 4111), 7.0, dtype=torch.bfloat16, device=DEV)
        out = room[:, to:to + 4003]
        B.token_logprobs_backward(x, tk, r.lse, r.entropy, g, out=out)
        want, tol = gradient(x, tk, g, None)
        assert ((out.cpu().double() - want).abs() <= tol + 2.0 ** -8 * want.abs()).all()
        assert (room[:, :to] == 7).all() and (room[:, to + 4003:] == 7).all()
    assert B.token_logprobs_backward(wide[:0], tokens[:0], g[:0], g[:0], g[:0]).shape == (0, 4200)


def test_offsets_past_32_bits():
    ld = 600_000_000
    flat = torch.empty(5 * ld, dtype=torch.bfloat16, device=DEV)  # 6 GB, sparsely used
    x = flat.as_strided((5, 3001), (ld, 1))
    small, tokens = logits(5, 3001, 10, torch.bfloat16)
    x.copy_(small)
    r = check(x, tokens, 5)
    g = torch.ones(5, device=DEV)
    want, tol = gradient(small, tokens, g, None)
    B.token_logprobs_backward(x, tokens, r.lse, r.entropy, g, lse_lo=r.lse_lo, out=x)
    assert ((x.cpu().double() - want).abs() <= tol + 2.0 ** -8 * want.abs()).all()


def test_another_stream_and_graph_capture():
    x, tokens = logits(40, 9000, 13)
    want = B.token_logprobs(x, tokens, top=4)
    g = torch.ones(40, device=DEV)
    grad = B.token_logprobs_backward(x, tokens, want.lse, want.entropy, g)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = B.token_logprobs(x, tokens, top=4, stream=s)
    got_grad = B.token_logprobs_backward(x, tokens, got.lse, got.entropy, g, stream=s)
    s.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want)) and torch.equal(got_grad, grad)
    out = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = B.token_logprobs(x, tokens, top=4)
        B.token_logprobs_backward(x, tokens, r.lse, r.entropy, g, out=out)
    x.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    again = B.token_logprobs(x, tokens, top=4)
    assert all(torch.equal(u, v) for u, v in zip(r, again))
    assert torch.equal(out, B.token_logprobs_backward(x, tokens, again.lse, again.entropy, g))


def test_binding_refusals():
    x, tokens = logits(4, 50, 1)
    r = B.token_logprobs(x, tokens)
    with pytest.raises(ValueError, match="fp32 or bf16"):
        B.token_logprobs(x.half(), tokens)
    with pytest.raises(ValueError, match="int64"):
        B.token_logprobs(x, tokens.int())
    with pytest.raises(ValueError, match="int64"):
        B.token_logprobs(x, tokens[:3])
    with pytest.raises(ValueError, match="top"):
        B.token_logprobs(x, tokens, top=33)
    with pytest.raises(B.ArgError, match="top"):
        B.token_logprobs(x[:, :5], tokens.clamp(max=4), top=6)
    with pytest.raises(ValueError, match="contiguous rows"):
        B.token_logprobs(x.t(), None)
    with pytest.raises(ValueError, match="one CUDA device"):
        B.token_logprobs(x, tokens.cpu())
    with pytest.raises(B.ArgError, match="both NULL"):
        B.token_logprobs_backward(x, tokens, r.lse, r.entropy)
    with pytest.raises(ValueError, match="fp32"):
        B.token_logprobs_backward(x, tokens, r.lse.double(), r.entropy, r.lse)
    with pytest.raises(B.ArgError, match="lse"):
        B.token_logprobs_backward(x, tokens, None, r.entropy, r.lse)
    with pytest.raises(B.ArgError, match="entropy"):
        B.token_logprobs_backward(x, tokens, r.lse, None, r.lse, r.lse)
