"""The operators beside the merge, as cases to measure: a merged global
published in 4 bits (``pack4`` / ``unpack4``), the products that answer from
it for a few tokens (``gemv4``), and the probe of a global on held-out text,
the log probabilities of its tokens with entropy and top alternatives
(``token_logprobs``) and their gradient (``token_logprobs_backward``).

``run`` computes each operator in elementary torch operations in 32 bits, or,
with ``own`` set, through the library. ``exact`` computes it in 64 bits.

The 4-bit form. A row of a matrix is cut into groups of G columns (the last
may be short). Group scale s = max|w| / 7, its low 16 bits cleared (a bf16,
rounded toward zero), 0 when that is below 2^-126; q = w * (1 / s) rounded to
the nearest integer (ties to even) and held to [-7, 7]; the value is q * s. A
group that holds a NaN or an infinity stands for NaN.

Log probabilities. For a row x of logits over V tokens: lse = log sum exp x,
log p = x - lse, H = -sum p log p. The probe gives log p of the row's token
(0 for a negative token id), H, lse and the `top` largest log p with their
ids (ties: the lowest id). A row of -inf alone has lse = log p = -inf, H = 0.
With g and h the gradients of log p[token] and of H, the logits' gradient is
g * (1[j = token] - p_j) - h * p_j * (log p_j + H).
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # publishing: one square attention matrix of the 512-wide stand, where the calls themselves count
        {"name": "pack_attention_512", "op": "pack4", "rows": 512, "cols": 512, "group": 64, "dtype": "f32", "values": "f32"},
        # publishing: the tied embedding of the 1.08B model from the fp32 master weights, the largest tensor of the list
        {"name": "pack_embedding_1b", "op": "pack4", "rows": 73760, "cols": 2048, "group": 64, "dtype": "f32", "values": "f32"},
        # answering: one token through the stand's down projection, 11 groups of 128 columns
        {"name": "gemv_down_stand", "op": "gemv4", "tokens": 1, "rows": 512, "cols": 1408, "group": 32, "dtype": "bf16"},
        # answering: one token through a gate or up projection of the 1.08B model
        {"name": "gemv_up_1b", "op": "gemv4", "tokens": 1, "rows": 5632, "cols": 2048, "group": 64, "dtype": "bf16"},
        # answering: one token's logits, the product that decoding waits for at every step
        {"name": "gemv_head_1b", "op": "gemv4", "tokens": 1, "rows": 73760, "cols": 2048, "group": 64, "dtype": "bf16"},
        # answering: a batch of 32 streams in fp32, the same head
        {"name": "gemv_head_1b_batch", "op": "gemv4", "tokens": 32, "rows": 73760, "cols": 2048, "group": 128, "dtype": "f32"},
        # decoding: one position's confidence, entropy and alternatives
        {"name": "logprobs_one_row", "op": "logprobs", "rows": 1, "vocab": 50304, "top": 5, "dtype": "bf16"},
        # the probe of a round: one context of 2,048 held-out tokens of the 1.08B model with 10 alternatives
        {"name": "logprobs_probe_1b", "op": "logprobs", "rows": 2048, "vocab": 73760, "top": 10, "dtype": "bf16"},
        # a probe in fp32 over an odd vocabulary, rows that no vector load is aligned to
        {"name": "logprobs_odd_f32", "op": "logprobs", "rows": 4096, "vocab": 50257, "top": 1, "dtype": "f32"},
        # training: the loss's gradient for a few positions
        {"name": "grad_few_rows", "op": "grad", "rows": 16, "vocab": 50304, "entropy": False, "dtype": "bf16"},
        # training: a worker's microbatch of two contexts, with an entropy term
        {"name": "grad_microbatch_1b", "op": "grad", "rows": 4096, "vocab": 73760, "entropy": True, "dtype": "bf16"},
        # training in fp32 over an odd vocabulary
        {"name": "grad_odd_f32", "op": "grad", "rows": 1000, "vocab": 50257, "entropy": True, "dtype": "f32"},
    ]


MOST_WEIGHTS = 73760 * 2048
MOST_LOGITS = 4096 * 50257


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("pack4", "gemv4", "gemv4", "logprobs", "logprobs", "grad"))
    dtype = rng.choice(("f32", "bf16"))
    while True:
        if op in ("pack4", "gemv4"):
            rows, cols = _spread(rng, 64, 80000), _spread(rng, 64, 16384)
            if rows * cols <= MOST_WEIGHTS:
                break
        else:
            rows, vocab = _spread(rng, 1, 8192), _spread(rng, 1000, 200000)
            if rows * vocab <= MOST_LOGITS:
                break
    if op == "pack4":
        return {"op": op, "rows": rows, "cols": cols, "group": rng.choice((32, 64, 128)), "dtype": dtype,
                "values": rng.choice(("f32", "bf16"))}
    if op == "gemv4":
        return {"op": op, "tokens": _spread(rng, 1, 32), "rows": rows, "cols": cols,
                "group": rng.choice((32, 64, 128)), "dtype": dtype}
    if op == "logprobs":
        return {"op": op, "rows": rows, "vocab": vocab, "top": rng.choice((0, 1, 5, 10, 20)), "dtype": dtype}
    return {"op": op, "rows": rows, "vocab": vocab, "entropy": rng.choice((False, True)), "dtype": dtype}


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _logits(case, gen):
    """Logits as a head gives them: a spread of a few units, the true token
    mostly well up, some tokens banned (-inf), as a decoder's bans or a padded
    vocabulary are; some positions carry no token (id -1)."""
    R, V = case["rows"], case["vocab"]
    x = torch.empty(R, V, device=DEV, dtype=torch.float32).normal_(0.0, 2.5, generator=gen)
    tokens = torch.randint(0, V, (R,), device=DEV, generator=gen)
    lift = torch.rand(R, 1, device=DEV, generator=gen) * 14.0
    x.scatter_add_(1, tokens[:, None], lift)
    banned = torch.randint(0, V, (R, 8), device=DEV, generator=gen)
    x.scatter_(1, banned.where(banned != tokens[:, None], (tokens[:, None] + 1) % V), -math.inf)
    tokens = tokens.masked_fill(torch.rand(R, device=DEV, generator=gen) < 0.1, -1)
    return x.to(TYPES[case["dtype"]]), tokens


def _weight(case, gen):
    return torch.empty(case["rows"], case["cols"], device=DEV, dtype=torch.float32).normal_(0.0, 0.02, generator=gen)


def _groups(w, group):
    """w in 32 bits as [rows, groups, group], a short last group filled with zeros."""
    w = w.float()
    short = -w.shape[1] % group
    if short:
        w = torch.nn.functional.pad(w, (0, short))
    return w.view(w.shape[0], -1, group)


def _quantised(w, group):
    """(q, s) of the 4-bit form, in 32 bits: q [rows, groups, group], s [rows, groups, 1]."""
    w = _groups(w, group)
    big = w.abs().amax(-1, keepdim=True)
    s = ((big / 7.0).view(torch.int32) & -65536).view(torch.float32)
    s = s.where(s >= 2.0 ** -126, torch.zeros_like(s))
    r = (1.0 / s).where(s > 0, torch.zeros_like(s))
    q = torch.round(w * r).clamp(-7.0, 7.0)
    fine = torch.isfinite(big)
    return q.where(fine, torch.zeros_like(q)), s.where(fine, torch.full_like(s, math.nan))


def prepare(case, seed):
    gen = _generator(seed)
    op = case["op"]
    if op == "pack4":
        return {"op": op, "case": case, "w": _weight(case, gen).to(TYPES[case["dtype"]])}
    if op == "gemv4":
        w = _weight(case, gen)
        x = torch.empty(case["tokens"], case["cols"], device=DEV, dtype=torch.float32).normal_(0.0, 1.0, generator=gen)
        x = x.to(TYPES[case["dtype"]])
        if own:
            from checkpoint_averaging_gb300 import binding as B

            return {"op": op, "case": case, "x": x, "w4": B.pack4(w, group=case["group"])}
        q, s = _quantised(w, case["group"])
        q = (q + 8.0).to(torch.uint8).view(q.shape[0], q.shape[1], q.shape[2] // 2, 2)
        return {"op": op, "case": case, "x": x, "q": q[..., 0] | (q[..., 1] << 4), "s": s.to(torch.bfloat16)}
    x, tokens = _logits(case, gen)
    state = {"op": op, "case": case, "x": x, "tokens": tokens}
    if op == "grad":
        # what the forward call left, and the gradients that reach it
        d = x.float()
        lse = torch.logsumexp(d, -1)
        d = d - lse[:, None]
        H = -(torch.exp(d) * d.clamp_min(-1e30)).sum(-1)
        R = case["rows"]
        state |= {"lse": lse, "H": H, "g": -(0.5 + torch.rand(R, device=DEV, generator=gen)) / R,
                  "h": torch.full((R,), -0.01 / R, device=DEV) if case["entropy"] else None}
    return state


def _plain_gemv(x, q, s, cols):
    v = torch.stack((q & 15, q >> 4), -1).flatten(2).float() - 8.0
    w = (v * s.float()).flatten(1)[:, :cols]
    return (x.float() @ w.t()).to(x.dtype)


def _plain_logprobs(x, tokens, top):
    x = x.float()
    m = x.amax(-1, keepdim=True)
    dead = m == -math.inf
    d = x - m.masked_fill(dead, 0.0)
    e = torch.exp(d)
    s = e.sum(-1, keepdim=True)
    log_s = torch.log(s)
    H = log_s - (e * d.masked_fill(e == 0, 0.0)).sum(-1, keepdim=True) / s
    logp = torch.gather(d, 1, tokens.clamp_min(0)[:, None]) - log_s
    out = {"logp": logp.masked_fill(dead, -math.inf)[:, 0].masked_fill(tokens < 0, 0.0),
           "entropy": H.masked_fill(dead, 0.0)[:, 0], "lse": (m + log_s)[:, 0]}
    if top:
        # one whole number for each logit, larger for a larger logit and, among equals, for a lower id
        bits = (x + 0.0).view(torch.int32)
        bits = bits ^ ((bits >> 31) & 0x7FFFFFFF)
        key = (bits.long() << 32) | (0x7FFFFFFF - torch.arange(x.shape[1], device=x.device))
        best = torch.topk(key, top, -1).values
        out["top_ids"] = 0x7FFFFFFF - (best & 0x7FFFFFFF)
        out["top_logp"] = (torch.gather(d, 1, out["top_ids"]) - log_s).masked_fill(dead, -math.inf)
    return out


def _plain_grad(x, tokens, lse, H, g, h):
    d = x.float() - lse[:, None]
    p = torch.exp(d)
    g = g.masked_fill(tokens < 0, 0.0)
    out = p * -g[:, None]
    if h is not None:
        out -= h[:, None] * p * (d.masked_fill(p == 0, 0.0) + H[:, None])
    out.scatter_add_(1, tokens.clamp_min(0)[:, None], g[:, None])
    return out.to(x.dtype)


def run(state):
    op, case = state["op"], state["case"]
    if own:
        from checkpoint_averaging_gb300 import binding as B

        if op == "pack4":
            return B.unpack4(B.pack4(state["w"], group=case["group"]), TYPES[case["values"]])
        if op == "gemv4":
            return B.gemv4(state["x"], state["w4"])
        if op == "logprobs":
            r = B.token_logprobs(state["x"], state["tokens"], top=case["top"])
            out = {"logp": r.logp, "entropy": r.entropy, "lse": r.lse}
            return out | {"top_ids": r.top_ids, "top_logp": r.top_logp} if case["top"] else out
        return B.token_logprobs_backward(state["x"], state["tokens"], state["lse"], state["H"], state["g"], state["h"])
    if op == "pack4":
        q, s = _quantised(state["w"], case["group"])
        return (q * s).flatten(1)[:, :case["cols"]].to(TYPES[case["values"]])
    if op == "gemv4":
        return _plain_gemv(state["x"], state["q"], state["s"], case["cols"])
    if op == "logprobs":
        return _plain_logprobs(state["x"], state["tokens"], case["top"])
    return _plain_grad(state["x"], state["tokens"], state["lse"], state["H"], state["g"], state["h"])


def work(case):
    op = case["op"]
    size = 4 if case["dtype"] == "f32" else 2
    if op in ("pack4", "gemv4"):
        N, K = case["rows"], case["cols"]
        packed = N * K // 2 + N * -(-K // case["group"]) * 2
        if op == "pack4":
            return {"bytes": N * K * (size + (4 if case["values"] == "f32" else 2)) + packed, "flops": 4 * N * K}
        M = case["tokens"]
        return {"bytes": packed + size * M * (N + K), "flops": 2 * M * N * K}
    R, V = case["rows"], case["vocab"]
    if op == "logprobs":
        return {"bytes": size * R * V + R * (8 + 12 + 12 * case["top"]), "flops": 5 * R * V}
    return {"bytes": 2 * size * R * V + R * (8 + 12 + (4 if case["entropy"] else 0)), "flops": (7 if case["entropy"] else 4) * R * V}


def exact(case, seed):
    op = case["op"]
    gen = _generator(seed)
    if op == "gemv4":
        # the weights are given in 4 bits: the product alone is the operator
        q, s = _quantised(_weight(case, gen), case["group"])
        x = torch.empty(case["tokens"], case["cols"], device=DEV, dtype=torch.float32).normal_(0.0, 1.0, generator=gen)
        value = (q.double() * s.double()).flatten(1)[:, :case["cols"]]
        return torch.matmul(x.to(TYPES[case["dtype"]]).double(), value.t())
    if op == "pack4":
        w = _weight(case, gen).to(TYPES[case["dtype"]])
        N, K, G = case["rows"], case["cols"], case["group"]
        n = -(-K // G)
        full = torch.zeros(N, n * G, device=DEV, dtype=torch.float64)
        full[:, :K] = w
        del w
        full = full.reshape(N * n, G)
        scale = full.abs().max(1).values / 7
        e = torch.floor(torch.log2(scale.clamp_min(1e-300)))
        e += (torch.exp2(e + 1) <= scale).double() - (torch.exp2(e) > scale).double()
        unit = torch.exp2(e - 7)
        scale = (torch.floor(scale / unit) * unit) * (scale >= 2.0 ** -126)
        full = torch.round(full / scale.clamp_min(1e-300)[:, None]).clamp(-7, 7) * scale[:, None]
        return full.reshape(N, n * G)[:, :K]
    x, tokens = _logits(case, gen)
    R, V = x.shape
    if op == "grad":
        g = -(0.5 + torch.rand(R, device=DEV, generator=gen)) / R
        grad = torch.empty(R, V, device=DEV, dtype=torch.float64)
    parts = []
    for at in range(0, R, 256):
        rows = slice(at, min(R, at + 256))
        logp = torch.log_softmax(x[rows].double(), -1)
        p = logp.exp()
        H = torch.special.entr(p).sum(-1)
        t = tokens[rows]
        if op == "grad":
            c = g[rows].double() * (t >= 0)
            part = -c[:, None] * p
            part[torch.arange(len(t), device=DEV), t.clamp_min(0)] += c
            if case["entropy"]:
                h = torch.full((len(t), 1), -0.01 / R, device=DEV).double()
                part += h * (torch.special.entr(p) - p * H[:, None])
            grad[rows] = part
            continue
        best = logp.topk(case["top"], -1).values if case["top"] else logp[:, :0]
        mine = logp[torch.arange(len(t), device=DEV), t.clamp_min(0)]
        parts.append((torch.where(t < 0, 0.0, mine), H, torch.logsumexp(x[rows].double(), -1), best))
    if op == "grad":
        return grad
    logp, H, lse, best = (torch.cat(v) for v in zip(*parts))
    out = {"logp": logp, "entropy": H, "lse": lse}
    return out | {"top_ids": None, "top_logp": best} if case["top"] else out
