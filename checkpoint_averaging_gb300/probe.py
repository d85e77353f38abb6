"""A merged global after its round: published in 4 or 8 bits, answered from for
a few tokens or whole contexts, probed on given tokens, and trained on from there.

The DiffuRefill-1B run probed every published global on held-out tokens and
chose between the global, its EMA and running averages by their losses
("DiffuRefill-1B" technical report, section 5.4, Table 5); a decoder picks by
each position's confidence and alternatives (model card, decoding). This
module runs the operators together as such a user would:

    python -m checkpoint_averaging_gb300.probe

merges a round of synthetic workers, publishes the tied embedding of the new
global and of its EMA, computes the logits of a few positions from the 4-bit
form, and reports each head's loss, entropy and alternatives, then takes one
gradient step of the positions' hidden states; after that it does the same with
whole contexts: the 8-bit form, and losses and gradients without the logits.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import binding as B


class _TokenLogprobsGrad(torch.autograd.Function):
    """The gradient, as a step of the graph under create_graph=True, so that a second
    derivative is refused. (once_differentiable would refuse it only where the gradients
    that arrive require one: a loss linear in its log probabilities lost this term.)"""

    @staticmethod
    def forward(ctx, logits, tokens, lse, lse_lo, entropy, g, h):
        return B.token_logprobs_backward(logits, tokens, lse, entropy, g, h, lse_lo=lse_lo)

    @staticmethod
    def backward(ctx, grad):
        raise RuntimeError("token log probabilities have no second derivative")


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens):
        r = B.token_logprobs(logits, tokens)
        ctx.save_for_backward(logits, tokens, r.lse, r.lse_lo, r.entropy)
        ctx.set_materialize_grads(False)
        return r.logp.clone(), r.entropy.clone()

    @staticmethod
    def backward(ctx, grad_logp, grad_entropy):
        logits, tokens, lse, lse_lo, entropy = ctx.saved_tensors
        if grad_logp is None and grad_entropy is None:
            return None, None
        # (the gradient of a sum or mean is one value expanded over the rows)
        g = None if grad_logp is None else grad_logp.contiguous()
        h = None if grad_entropy is None else grad_entropy.contiguous()
        return _TokenLogprobsGrad.apply(logits, tokens, lse, lse_lo, entropy, g, h), None


def differentiable_logprobs(logits, tokens):
    """(log probabilities of the tokens, entropies) of rows of logits, for a loss:
    gradients reach the logits through cam_token_logprobs_backward. A second
    derivative is refused."""
    return _TokenLogprobs.apply(logits, tokens)


class _HeadLogprobsGrad(torch.autograd.Function):
    """The gradients, as a step of the graph under create_graph=True, so that a second
    derivative is refused (see _TokenLogprobsGrad)."""

    @staticmethod
    def forward(ctx, hidden, head, tokens, lse, lse_lo, entropy, g, h, need_hidden, need_head):
        return B.head_logprobs_backward(hidden, head, tokens, lse, entropy, g, h, lse_lo=lse_lo,
                                        need_hidden=need_hidden, need_head=need_head)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("token log probabilities have no second derivative")


class _HeadLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, head, tokens):
        r = B.head_logprobs(hidden, head, tokens)
        ctx.save_for_backward(hidden, head, tokens, r.lse, r.lse_lo, r.entropy)
        ctx.set_materialize_grads(False)
        return r.logp.clone(), r.entropy.clone()

    @staticmethod
    def backward(ctx, grad_logp, grad_entropy):
        if grad_logp is None and grad_entropy is None:
            return None, None, None
        g = None if grad_logp is None else grad_logp.contiguous()
        h = None if grad_entropy is None else grad_entropy.contiguous()
        hidden, head, tokens, lse, lse_lo, entropy = ctx.saved_tensors
        grads = _HeadLogprobsGrad.apply(hidden, head, tokens, lse, lse_lo, entropy, g, h,
                                        *ctx.needs_input_grad[:2])
        return *grads, None


def differentiable_head_logprobs(hidden, head, tokens):
    """(log probabilities of the tokens, entropies) of the logits hidden head^T, which are
    not stored, for a loss: gradients reach hidden and head through
    cam_head_logprobs_backward, the one that requires none is not computed. A second
    derivative is refused."""
    return _HeadLogprobs.apply(hidden, head, tokens)


class Probe(NamedTuple):
    """What probe found of a head on given tokens."""
    loss: torch.Tensor        # mean of -log p over the rows with a token
    entropy: torch.Tensor     # mean over all rows
    logp: torch.Tensor        # [rows]
    top_logp: torch.Tensor    # [rows, top]
    top_ids: torch.Tensor


def head_logits(hidden, head):
    """The logits of hidden states [rows, width]: `head` is a [vocab, width]
    matrix, or its 4-bit form (Packed4) for the few rows of a decoding step, or its
    8-bit form (Packed8) for whole contexts; no gradient flows through those
    (hidden states that require one are refused)."""
    if isinstance(head, B.Packed4):
        return B.gemv4(hidden, head)
    if isinstance(head, B.Packed8):
        return B.matmul8(hidden, head)
    return hidden @ head.to(hidden.dtype).t()


def probe(hidden, head, tokens, top: int = 5) -> Probe:
    """Probes a head: loss and entropy on given tokens (a negative id is no
    token) and the `top` alternatives of every row."""
    r = B.token_logprobs(head_logits(hidden, head), tokens, top=top)
    known = (tokens >= 0).sum().clamp(min=1)
    return Probe(-r.logp.sum() / known, r.entropy.mean(), r.logp, r.top_logp, r.top_ids)


class ContextLoss(NamedTuple):
    """What context_loss found of a head on given tokens."""
    loss: torch.Tensor        # mean of -log p over the rows with a token
    entropy: torch.Tensor     # mean over all rows
    logp: torch.Tensor        # [rows]


def context_loss(hidden, head, tokens) -> ContextLoss:
    """probe's loss and entropy of whole contexts, for a [vocab, width] head of
    hidden's dtype: the logits are neither stored nor rounded to it (and there are no
    alternatives)."""
    r = B.head_logprobs(hidden, head, tokens)
    known = (tokens >= 0).sum().clamp(min=1)
    return ContextLoss(-r.logp.sum() / known, r.entropy.mean(), r.logp)


def main(vocab: int = 8192, width: int = 512, rows: int = 16, workers: int = 3, seed: int = 0):
    """One round, as described at the top; returns {head: Probe} and the losses
    before and after the gradient step."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale):
        return torch.empty(*shape, device="cuda").normal_(0.0, scale, generator=gen)

    # a round: three workers' copies of a tied embedding and a block matrix
    shapes = [(vocab, width), (width, width)]
    theta = [normal(*s, scale=0.05) for s in shapes]
    ema = [t.clone() for t in theta]
    m = B.Merger(theta, ema=ema, quorum=workers)
    rd = m.begin(0)
    for _ in range(workers):
        rd.accumulate([t + normal(*t.shape, scale=0.01) for t in theta], 100_000)
    rd.finalize(B.MEAN_REPLACE)
    rd.ema_update(0.9)
    rd.commit()

    # published: half a byte and a share of a scale per weight
    heads = {"global": theta[0], "global, 4 bits": B.pack4(theta[0], group=64),
             "EMA": ema[0], "EMA, 4 bits": B.pack4(ema[0], group=64)}

    # positions whose hidden states lean to their token's embedding
    tokens = torch.randint(0, vocab, (rows,), device="cuda", generator=gen)
    hidden = theta[0][tokens] * 6.0 + normal(rows, width, scale=0.3)
    tokens[-1] = -1
    found = {name: probe(hidden, head, tokens) for name, head in heads.items()}

    # one gradient step of the hidden states on the full-precision head
    state = hidden.clone().requires_grad_(True)
    losses = []
    for _ in range(2):
        logp, entropy = differentiable_logprobs(state @ theta[0].t(), tokens)
        loss = -logp.sum() / (rows - 1) + 0.01 * entropy.mean()
        losses.append(float(loss.detach()))
        if len(losses) == 1:
            loss.backward()
            state = (state - 0.5 * state.grad).detach()
    m.close()
    return found, losses


def main_contexts(vocab: int = 8192, width: int = 512, rows: int = 1000, seed: int = 0):
    """A head probed on a whole context and trained with it: the loss by the 8-bit
    form's logits and without any, in bf16, and the losses before and after one gradient
    step of the hidden states and the head in fp32."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale):
        return torch.empty(*shape, device="cuda").normal_(0.0, scale, generator=gen)

    head = normal(vocab, width, scale=0.05)
    tokens = torch.randint(0, vocab, (rows,), device="cuda", generator=gen)
    hidden = head[tokens] * 3.0 + normal(rows, width, scale=0.3)
    tokens[::10] = -1
    short, short_head = hidden.bfloat16(), head.bfloat16()
    eight = probe(short, B.pack8(head), tokens, top=1)
    full = context_loss(short, short_head, tokens)

    state, weight = hidden.clone().requires_grad_(True), head.clone().requires_grad_(True)
    losses = []
    for _ in range(2):
        logp, entropy = differentiable_head_logprobs(state, weight, tokens)
        loss = -logp.sum() / (tokens >= 0).sum() + 0.01 * entropy.mean()
        losses.append(float(loss.detach()))
        if len(losses) == 1:
            loss.backward()
            state = (state - 0.5 * state.grad).detach()
            weight = (weight - 0.5 * weight.grad).detach()
    if B.operators_status() != 0:  # (then results are undefined, and no call has said so)
        raise RuntimeError("an operator gave up waiting on a barrier")
    return eight, full, losses


if __name__ == "__main__":
    probes, steps = main()
    for name, p in probes.items():
        print(f"{name:15s} loss {float(p.loss):.4f}  entropy {float(p.entropy):.4f}  "
              f"first row's alternatives {p.top_ids[0].tolist()}")
    print(f"loss with entropy term: {steps[0]:.4f}, after one step {steps[1]:.4f}")
    eight, full, steps = main_contexts()
    print(f"a context: loss {float(full.loss):.4f} without logits, {float(eight.loss):.4f} in 8 bits; "
          f"with entropy term {steps[0]:.4f}, after one step of hidden states and head {steps[1]:.4f}")
