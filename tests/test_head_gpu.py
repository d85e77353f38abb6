"""Log probabilities of a head's tokens without its logits, and the gradients, on the
GPU against the definitions in 64 bits (include/cam.h).

Tolerances. A logit is a sum of `width` products, exact each for bf16 inputs, on the
tensor cores: per step of 16 terms two roundings of at most 2^-23 of
A = sum |hidden_i head_i|, and for fp32 inputs six such sums and 2^-22 A for the
products of terms that are left out: off = (12 width / 16 + 16) 2^-23 A at most for
either (for bf16 a sixth of it would do). lse moves by at most a row's largest off,
log p by twice it; their own arithmetic is that of token_logprobs
(test_logprobs_gpu.py): base = 2e-5 + 2^-22 L with L the largest |logit|. The entropy
moves by |dH| <= sum |dp| (|log p| + H) with |dp| <= 2 off p: at most 4 off H, and
2e-5 (1 + H).

The gradient: p = exp(x - lse) is off by r p, r = 2 off + (|x - lse| + 4) 2^-22
+ 2^-22 L, so G by |g| p r + |h| p ((|log p| + H + 1) r + 2^-20 (|log p| + H)) and
2^-22 |g| at the token, and for bf16 inputs by its rounding, 2^-8 |G|, for fp32 ones by 2^-23 |G|.
The products with the head and with hidden pass that on, |dG| |head| and |dG|^T |hidden|,
and add (12 K / 16 + 64) 2^-23 of |G| |head| (K = vocab) and |G|^T |hidden| (K = rows);
a bf16 result rounds by 2^-8 of itself.
"""
import ctypes
import math

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


def inputs(rows, vocab, width, dtype, seed=0, spread=2.5):
    g = torch.Generator().manual_seed(seed + rows + vocab + width)
    head = torch.randn(vocab, width, generator=g) * (spread / math.sqrt(width))
    tokens = torch.randint(0, vocab, (rows,), generator=g)
    hidden = torch.randn(rows, width, generator=g)
    hidden += head[tokens] * (torch.rand(rows, 1, generator=g) * 14 / spread ** 2)
    if rows > 2:
        tokens[1] = -1
    return hidden.to(dtype).to(DEV), head.to(dtype).to(DEV), tokens.to(DEV)


class Exact:
    """The definitions in 64 bits, and how far a logit may be off."""

    def __init__(self, hidden, head, tokens):
        self.a, self.w = hidden.double(), head.double()
        x = self.a @ self.w.t()
        self.lse = torch.logsumexp(x, 1)
        self.logp = x - self.lse[:, None]
        self.p = self.logp.exp()
        self.H = torch.special.entr(self.p).sum(1)
        self.tokens = tokens
        mine = self.logp.gather(1, tokens.clamp(0, len(self.w) - 1)[:, None])[:, 0]
        self.mine = mine.masked_fill(tokens < 0, 0.0)
        self.off = (12 * hidden.shape[1] / 16 + 16) * 2.0 ** -23 * (self.a.abs() @ self.w.abs().t())
        self.L = x.abs().amax(1)


def check(hidden, head, tokens, e=None):
    e = e or Exact(hidden, head, tokens)
    r = B.head_logprobs(hidden, head, tokens)
    off = e.off.amax(1)
    base = 2e-5 + 2.0 ** -22 * e.L
    assert ((r.lse.double() - e.lse).abs() <= base + off).all()
    assert ((r.lse.double() + r.lse_lo.double() - e.lse).abs() <= base + off).all()
    assert (r.lse_lo.abs() <= 2.0 ** -24 * r.lse.abs() + 1e-30).all()
    assert ((r.logp.double() - e.mine).abs() <= base + 2 * off).all()
    assert (r.logp[tokens < 0] == 0).all()
    assert ((r.entropy.double() - e.H).abs() <= base + (4 * off + 2e-5) * e.H).all()
    assert r.top_logp is None and r.top_ids is None
    return r


def check_grad(hidden, head, tokens, with_g=True, with_h=True, lo=True, e=None, **more):
    e = e or Exact(hidden, head, tokens)
    rows = len(tokens)
    gen = torch.Generator().manual_seed(rows)
    g = -(torch.rand(rows, generator=gen) + 0.5).to(DEV) / rows if with_g else None
    h = (torch.randn(rows, generator=gen) * 0.1).to(DEV) / rows if with_h else None
    lse = e.lse.float()
    got = B.head_logprobs_backward(hidden, head, tokens, lse, e.H.float(), g, h,
                                   lse_lo=(e.lse - lse.double()).float() if lo else None, **more)
    c = torch.zeros(rows, 1, device=DEV, dtype=torch.float64) if g is None \
        else (g.double() * (tokens >= 0))[:, None]
    k = torch.zeros_like(c) if h is None else h.double()[:, None]
    spread = e.logp.abs() + e.H[:, None]
    G = -c * e.p - k * e.p * (e.logp + e.H[:, None])
    G.scatter_add_(1, tokens.clamp(min=0)[:, None], c)
    r = 2 * e.off + (e.logp.abs() + 4 + e.L[:, None]) * 2.0 ** -22 + (0 if lo else 1) * 2.0 ** -23 * e.L[:, None]
    dG = c.abs() * e.p * r + k.abs() * e.p * ((spread + 1) * r + 2.0 ** -20 * spread)
    dG.scatter_add_(1, tokens.clamp(min=0)[:, None], 2.0 ** -22 * c.abs())
    dG += (2.0 ** -8 if hidden.dtype == BF16 else 2.0 ** -23) * G.abs()
    for out, other, dGo, Go, n in ((got[0], e.w, dG, G, e.w.shape[0]), (got[1], e.a, dG.t(), G.t(), rows)):
        if out is None:
            continue
        want = Go @ other
        tol = dGo @ other.abs() + (12 * n / 16 + 64) * 2.0 ** -23 * (Go.abs() @ other.abs())
        if out.dtype == BF16:
            tol += 2.0 ** -8 * want.abs()
        assert out.dtype == hidden.dtype and out.shape == want.shape
        off = (out.double() - want).abs() - tol - 1e-37
        assert off.max() <= 0, (off.max(), int((off > 0).sum()))
    return got


SIZES = [(1, 1, 1), (1, 2, 3), (3, 100, 64), (2, 257, 65), (5, 1000, 8), (16, 5000, 128), (127, 300, 100),
         (128, 513, 200), (129, 129, 64), (130, 1000, 129), (256, 255, 72), (257, 2049, 300), (300, 777, 512),
         (1000, 3001, 130), (1, 50304, 128), (40, 20011, 257)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,vocab,width", SIZES)
def test_log_probabilities(rows, vocab, width, dtype):
    hidden, head, tokens = inputs(rows, vocab, width, dtype)
    a = check(hidden, head, tokens)
    b = B.head_logprobs(hidden, head, tokens)
    for u, v in zip(a, b):
        assert u is None or torch.equal(u, v)  # the same bits again
    none = B.head_logprobs(hidden, head)
    assert none.logp is None and torch.equal(none.lse, a.lse) and torch.equal(none.entropy, a.entropy)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,vocab,width", SIZES)
def test_gradients(rows, vocab, width, dtype):
    hidden, head, tokens = inputs(rows, vocab, width, dtype)
    e = Exact(hidden, head, tokens)
    a = check_grad(hidden, head, tokens, e=e)
    b = check_grad(hidden, head, tokens, e=e)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check_grad(hidden, head, tokens, with_h=False, e=e)
    check_grad(hidden, head, tokens, with_g=False, lo=False, e=e)
    only = check_grad(hidden, head, tokens, need_head=False, e=e)
    assert only[1] is None and torch.equal(only[0], a[0])
    only = check_grad(hidden, head, tokens, need_hidden=False, e=e)
    assert only[0] is None and torch.equal(only[1], a[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [7, 200])
def test_strides_and_alignment(rows, dtype):
    hidden, head, tokens = inputs(rows, 600, 136, dtype)
    want, grads = check(hidden, head, tokens), check_grad(hidden, head, tokens)
    for pad, offset in ((1, 0), (3, 2), (8, 0), (8, 1), (16, 8)):
        a = torch.full((rows, 136 + pad + offset), math.nan, dtype=dtype, device=DEV)
        w = torch.full((600, 136 + pad + offset), math.nan, dtype=dtype, device=DEV)
        a[:, offset:offset + 136], w[:, offset:offset + 136] = hidden, head
        a, w = a[:, offset:offset + 136], w[:, offset:offset + 136]
        for u, v in zip(want, B.head_logprobs(a, w, tokens)):
            assert u is None or torch.equal(u, v)
        got = check_grad(a, w, tokens)
        assert torch.equal(got[0], grads[0]) and torch.equal(got[1], grads[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_confident_rows_keep_their_loss(dtype):
    # one logit at 20 to 58 above the rest: losses down to 1e-23
    width, vocab = 64, 500
    head = torch.eye(vocab, width)
    hidden = torch.zeros(20, width)
    tokens = torch.arange(20)
    hidden[torch.arange(20), tokens] = torch.arange(20) * 2.0 + 20.0
    hidden, head, tokens = hidden.to(dtype).to(DEV), head.to(dtype).to(DEV), tokens.to(DEV)
    r = B.head_logprobs(hidden, head, tokens)
    top = torch.arange(20, device=DEV).double() * 2 + 20
    want = -torch.log1p((vocab - 1) * torch.exp(-top))
    assert ((r.logp.double() - want).abs() <= 1e-5 * want.abs()).all()
    p = torch.exp(-top) / (1 + (vocab - 1) * torch.exp(-top))
    H = -want + (vocab - 1) * p * top
    assert ((r.entropy.double() - H).abs() <= 1e-5 * H).all()
    g = torch.full((20,), -1.0, device=DEV)
    grad, _ = B.head_logprobs_backward(hidden, head, tokens, r.lse, r.entropy, g, lse_lo=r.lse_lo)
    mine = grad.double()[torch.arange(20), tokens]  # -(1 - p) of the token
    tol = 1e-5 + (2.0 ** -7 if dtype == BF16 else 0)
    assert ((mine + (vocab - 1) * p).abs() <= tol * (vocab - 1) * p + 1e-37).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_equal_logits(dtype):
    hidden = torch.zeros(130, 64, dtype=dtype, device=DEV)
    head = torch.ones(1000, 64, dtype=dtype, device=DEV)
    hidden[::2] = 0.5
    tokens = torch.arange(130, device=DEV)
    r = B.head_logprobs(hidden, head, tokens)
    assert (r.logp + math.log(1000)).abs().max() < 1e-6
    assert (r.entropy - math.log(1000)).abs().max() < 1e-6


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [5, 150])
def test_rows_that_are_broken(rows, dtype):
    hidden, head, tokens = inputs(rows, 700, 96, dtype)
    good = B.head_logprobs(hidden, head, tokens)
    hidden[0, 3], hidden[2, 95], hidden[4, 0] = math.nan, math.inf, -math.inf
    r = B.head_logprobs(hidden, head, tokens)
    bad = torch.zeros(rows, dtype=torch.bool, device=DEV)
    bad[[0, 2, 4]] = True
    for u, v in zip(r, good):
        if u is not None:
            assert torch.isnan(u[bad]).all() and torch.equal(u[~bad], v[~bad])
    # a broken row without a gradient reaches nothing
    g = torch.full((rows,), -1.0, device=DEV)
    g[bad] = 0.0
    h = torch.zeros(rows, device=DEV)
    a = B.head_logprobs_backward(hidden, head, tokens, r.lse, r.entropy, g, h, lse_lo=r.lse_lo)
    clean = hidden.clone()
    clean[bad] = 0.0
    lse = r.lse.masked_fill(bad, 1.0)
    b = B.head_logprobs_backward(clean, head, tokens, lse, r.entropy.masked_fill(bad, 1.0), g, h,
                                 lse_lo=r.lse_lo.masked_fill(bad, 0.0))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert (a[0][bad] == 0).all() and torch.isfinite(a[1]).all()
    # nor does one whose token id is negative
    t = tokens.masked_fill(bad, -5)
    c = B.head_logprobs_backward(hidden, head, t, r.lse, r.entropy, g.masked_fill(bad, -1.0), None,
                                 lse_lo=r.lse_lo)
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
    # with a gradient it breaks its own and the head's
    d = B.head_logprobs_backward(hidden, head, tokens, r.lse, r.entropy, g - 1, None)
    assert torch.isnan(d[0][bad]).all() and torch.isfinite(d[0][~bad]).all() and torch.isnan(d[1]).all()


def test_token_ids_outside():
    hidden, head, tokens = inputs(150, 700, 96, BF16)
    good = B.head_logprobs(hidden, head, tokens)
    t = tokens.clone()
    t[3], t[4], t[140] = 700, 1 << 40, -(1 << 40)
    r = B.head_logprobs(hidden, head, t)
    assert torch.isnan(r.logp[3]) and torch.isnan(r.logp[4]) and r.logp[140] == 0
    keep = torch.ones(150, dtype=torch.bool, device=DEV)
    keep[[3, 4, 140]] = False
    assert torch.equal(r.logp[keep], good.logp[keep]) and torch.equal(r.lse, good.lse)
    g = torch.full((150,), -1.0, device=DEV)
    a = B.head_logprobs_backward(hidden, head, t, r.lse, r.entropy, g)
    assert torch.isnan(a[0][[3, 4]]).all() and torch.isfinite(a[0][keep]).all() and (a[0][140] == 0).all()
    g[[3, 4]] = 0.0
    a = B.head_logprobs_backward(hidden, head, t, r.lse, r.entropy, g)
    assert torch.isfinite(a[0]).all() and torch.isfinite(a[1]).all() and (a[0][[3, 4]] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_logits(dtype):
    # logits up to some thousands: one token has all of the probability, or shares it with an equal
    hidden, head, tokens = inputs(140, 900, 64, dtype, spread=400.0)
    check(hidden, head, tokens)
    check_grad(hidden, head, tokens)
    head[5] = head[6]
    check(hidden, head, tokens)


def test_no_rows():
    head = torch.ones(300, 64, device=DEV)
    hidden = torch.empty(0, 64, device=DEV)
    tokens = torch.empty(0, dtype=torch.int64, device=DEV)
    r = B.head_logprobs(hidden, head, tokens)
    assert r.logp.shape == (0,)
    none = torch.empty(0, device=DEV)
    gx, gw = B.head_logprobs_backward(hidden, head, tokens, none, none, none)
    assert gx.shape == (0, 64) and torch.equal(gw, torch.zeros_like(head))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_several_pieces_of_the_vocabulary(dtype):
    # G of all the vocabulary would be over the piece's bytes: several pieces, the last ragged
    rows, vocab, width = (9001, 20011, 64) if dtype == F32 else (9001, 30011, 64)
    hidden, head, tokens = inputs(rows, vocab, width, dtype)
    check(hidden, head, tokens)
    check_grad(hidden, head, tokens)


def test_differences():
    """The gradients against differences of the forward call itself, fp32."""
    hidden, head, tokens = inputs(9, 400, 80, F32)
    gen = torch.Generator().manual_seed(5)
    g, h = torch.randn(9, generator=gen).to(DEV), torch.randn(9, generator=gen).to(DEV)
    r = B.head_logprobs(hidden, head, tokens)
    gx, gw = B.head_logprobs_backward(hidden, head, tokens, r.lse, r.entropy, g, h, lse_lo=r.lse_lo)

    def loss(a, w):
        s = B.head_logprobs(a, w, tokens)
        return float((s.logp.double() * g.double()).sum() + (s.entropy.double() * h.double()).sum())

    for _ in range(4):
        da = torch.randn(9, 80, generator=gen).to(DEV)
        dw = torch.randn(400, 80, generator=gen).to(DEV) * 0.1
        t = 2.0 ** -7
        slope = (loss(hidden + t * da, head + t * dw) - loss(hidden - t * da, head - t * dw)) / (2 * t)
        want = float((gx.double() * da).sum() + (gw.double() * dw).sum())
        # forward values of ~1e2 rounded to 2^-22 over 2 t, and t^2 / 6 of third derivatives
        assert abs(slope - want) <= 2e-2 * (1 + abs(want))


def test_refusals():
    hidden, head, tokens = inputs(5, 300, 64, F32)
    r = B.head_logprobs(hidden, head, tokens)
    with pytest.raises(ValueError, match="one dtype"):
        B.head_logprobs(hidden.bfloat16(), head, tokens)
    with pytest.raises(ValueError, match="columns"):
        B.head_logprobs(hidden[:, :63], head, tokens)
    with pytest.raises(ValueError, match="tokens"):
        B.head_logprobs(hidden, head, tokens[:4])
    with pytest.raises(ValueError, match="tokens"):
        B.head_logprobs(hidden, head, tokens.int())
    with pytest.raises(ValueError, match="contiguous rows"):
        B.head_logprobs(hidden, head.t().contiguous().t(), tokens)
    with pytest.raises(ValueError, match="gradient"):
        B.head_logprobs(hidden, head.clone().requires_grad_(True), tokens)
    with pytest.raises(ValueError, match="one per row"):
        B.head_logprobs_backward(hidden, head, tokens, r.lse[:4], r.entropy, r.lse)
    with pytest.raises(B.ArgError, match="both NULL"):
        B.head_logprobs_backward(hidden, head, tokens, r.lse, r.entropy)
    with pytest.raises(B.ArgError, match="tokens"):
        B.head_logprobs_backward(hidden, head, None, r.lse, r.entropy, r.lse)
    assert B.head_logprobs_backward(hidden, head, tokens, r.lse, r.entropy, r.lse, need_hidden=False,
                                    need_head=False) == (None, None)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_other_streams_and_graphs(dtype):
    hidden, head, tokens = inputs(200, 1500, 96, dtype)
    g = torch.full((200,), -0.01, device=DEV)

    def both(a):
        r = B.head_logprobs(a, head, tokens)
        return r._stats, *B.head_logprobs_backward(a, head, tokens, r.lse, r.entropy, g, lse_lo=r.lse_lo)

    want = both(hidden)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r = B.head_logprobs(hidden, head, tokens, stream=s)
    with torch.cuda.stream(s):
        lse, entropy, lo = r.lse, r.entropy, r.lse_lo
    grads = B.head_logprobs_backward(hidden, head, tokens, lse, entropy, g, lse_lo=lo, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for u, v in zip((r._stats, *grads), want):
        assert torch.equal(u, v)
    # two graphs replayed at once
    other = hidden.flip(0).contiguous()
    graphs, outs, ins = [], [], [hidden.clone(), hidden.clone()]
    for a in ins:
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            outs.append(both(a))
        graphs.append(graph)
    ins[1].copy_(other)
    want2 = both(other)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for got, ref in zip(outs, (want, want2)):
        for u, v in zip(got, ref):
            assert torch.equal(u, v)


@pytest.mark.parametrize("rows", [9, 150])
def test_logits_far_from_zero(rows):
    """bf16 logits of 1e5 and more, all of a row near its largest: p keeps what the logits say."""
    gen = torch.Generator().manual_seed(rows)
    hidden = torch.zeros(rows, 64)
    hidden[:, 0] = 2.0 ** 17
    hidden[:, 1:4] = torch.randn(rows, 3, generator=gen)
    head = torch.zeros(300, 64)
    head[:, 0] = 1.0
    head[:, 1:4] = torch.randn(300, 3, generator=gen)
    tokens = torch.randint(0, 300, (rows,), generator=gen).to(DEV)
    hidden, head = hidden.to(BF16).to(DEV), head.to(BF16).to(DEV)
    x = hidden.double() @ head.double().t()
    lse = torch.logsumexp(x, 1)
    p = (x - lse[:, None]).exp()
    top = lse.float()
    g = torch.full((rows,), -1.0, device=DEV)
    _, gw = B.head_logprobs_backward(hidden, head, tokens, top, torch.zeros_like(top), g,
                                     lse_lo=(lse - top.double()).float())
    # logits are sums rounded at 2^17: 64 / 16 steps and a sum of fp32 lose 2 * 2^-6 each at most
    off = 10 * 2.0 ** -6
    G = p.clone()
    G.scatter_add_(1, tokens[:, None], torch.full((rows, 1), -1.0, device=DEV).double())
    dG = p * (math.exp(off) - 1) + 2.0 ** -8 * G.abs()
    assert ((gw.double() - G.t() @ hidden.double()).abs()
            <= dG.t() @ hidden.double().abs() * 1.01 + 2.0 ** -8 * (G.t() @ hidden.double()).abs() + 1e-6).all()


def poison(size=1 << 27):
    """Leaves NaN in the allocator's free memory, where workspaces come from."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.full((n // 4,), math.nan, device=DEV) for n in (size, 1 << 20, 1 << 16, 4096)]
    torch.cuda.synchronize()
    del blocks


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [7, 120, 200, 300])
@pytest.mark.parametrize("more", range(1, 8))
def test_what_lies_beside_the_rows_is_not_read(rows, more, dtype):
    # rows that start on 16 bytes and end anywhere, NaN behind them and in the workspaces
    width, vocab = 128 + more, 600 + more
    hidden, head, tokens = inputs(rows, vocab, width, dtype)
    want, grads = check(hidden, head, tokens), check_grad(hidden, head, tokens)
    a = torch.full((rows + 1, 144), math.nan, dtype=dtype, device=DEV)
    w = torch.full((vocab + 1, 144), math.nan, dtype=dtype, device=DEV)
    a[:rows, :width], w[:vocab, :width] = hidden, head
    a, w = a[:rows, :width], w[:vocab, :width]
    poison()
    for u, v in zip(want, B.head_logprobs(a, w, tokens)):
        assert u is None or torch.equal(u, v)
    poison()
    got = check_grad(a, w, tokens)
    assert torch.equal(got[0], grads[0]) and torch.equal(got[1], grads[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [7, 120, 200, 300])
@pytest.mark.parametrize("width", range(129, 137))
def test_what_lies_beside_the_gradients_stays(rows, width, dtype):
    hidden, head, tokens = inputs(rows, 601, width, dtype)
    e = Exact(hidden, head, tokens)
    want = check_grad(hidden, head, tokens, with_h=False, e=e)
    gen = torch.Generator().manual_seed(rows)
    g = -(torch.rand(rows, generator=gen) + 0.5).to(DEV) / rows
    L, code = B.lib(), B.F32 if dtype is F32 else B.BF16
    lse, H = e.lse.float(), e.H.float()
    lo = (e.lse - lse.double()).float()
    size = ctypes.c_int64()
    args = (rows, 601, width)
    assert L.cam_head_logprobs_backward_workspace(*args, head.data_ptr(), width, code,
                                                  ctypes.byref(size)) == 0
    space = torch.empty(size.value, dtype=torch.uint8, device=DEV)
    dx = torch.full((rows + 1, 144), 9.0, dtype=dtype, device=DEV)
    dw = torch.full((602, 144), 9.0, dtype=dtype, device=DEV)
    stream = torch.cuda.current_stream().cuda_stream
    assert L.cam_head_logprobs_backward(
        *args, hidden.data_ptr(), width, head.data_ptr(), width, code, tokens.data_ptr(),
        lse.data_ptr(), lo.data_ptr(), H.data_ptr(), g.data_ptr(), None, dx.data_ptr(), 144,
        dw.data_ptr(), 144, space.data_ptr(), size.value, stream) == 0
    torch.cuda.synchronize()
    for got, room, n in ((want[0], dx, rows), (want[1], dw, 601)):
        assert torch.equal(room[:n, :width], got)
        assert (room[:n, width:] == 9).all() and (room[n] == 9).all()
