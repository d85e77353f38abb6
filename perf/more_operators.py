"""More operators beside the merge, as cases to measure: a merged global
published in 8 bits (``pack8`` / ``unpack8``), its products with whole contexts
(``matmul8``), and the probe of a head on held-out text from hidden states,
whose logits are never kept (``head_logprobs``), with the gradients of the
hidden states and of the head (``head_logprobs_backward``).

``run`` computes each operator in elementary torch operations in 32 bits, or,
with ``own`` set, through the library. ``exact`` computes it in 64 bits.

The 8-bit form. A row of a matrix is cut into blocks of 128 columns (the last
may be short). Per block, e is the least integer, -126 or more, for which
max|w| <= 448 * 2^e; q is w * 2^-e rounded to the nearest e4m3 number (4
significant bits, steps of 2^-9 below 2^-6; ties to even); the value is
q * 2^e. A block that holds a NaN or an infinity stands for NaN. The product
takes a matrix in that form and rows x, which it brings into the same form.

Log probabilities of a head. x = hidden head^T is a row of logits over V
tokens: lse = log sum exp x, log p = x - lse, H = -sum p log p. The results are
log p of the row's token (0 for a negative id), H and lse. With g and h the
gradients of log p[token] and of H, G = g * (1[j = token] - p_j) -
h * p_j * (log p_j + H) is the logits' gradient, G head that of the hidden
states and G^T hidden that of the head.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BLOCK = 128


def listed():
    return [
        # publishing: one square attention matrix of the 512-wide stand, where the calls themselves count
        {"name": "pack8_attention_512", "op": "pack8", "rows": 512, "cols": 512, "dtype": "f32", "values": "bf16"},
        # publishing: the tied embedding of the 1.08B model from the fp32 master weights, the largest tensor of the list
        {"name": "pack8_embedding_1b", "op": "pack8", "rows": 73760, "cols": 2048, "dtype": "f32", "values": "bf16"},
        # answering: 16 positions through the stand's down projection, 11 blocks of columns
        {"name": "matmul8_down_stand", "op": "matmul8", "tokens": 16, "rows": 512, "cols": 1408, "dtype": "bf16"},
        # answering: a context of 2,048 positions through a gate or up projection of the 1.08B model
        {"name": "matmul8_up_1b", "op": "matmul8", "tokens": 2048, "rows": 5632, "cols": 2048, "dtype": "bf16"},
        # answering in fp32: odd numbers of positions, rows and columns, a short last block
        {"name": "matmul8_odd_f32", "op": "matmul8", "tokens": 1001, "rows": 5003, "cols": 1413, "dtype": "f32"},
        # answering: the logits of a whole context through the tied embedding of the 1.08B model
        {"name": "matmul8_head_1b", "op": "matmul8", "tokens": 2048, "rows": 73760, "cols": 2048, "dtype": "bf16"},
        # the probe: four positions of the Pythia-14M shape, where the calls themselves count
        {"name": "head_pythia_few", "op": "head", "rows": 4, "vocab": 50304, "width": 128, "dtype": "bf16"},
        # the probe in fp32: the stand's width over an odd vocabulary
        {"name": "head_stand_f32", "op": "head", "rows": 1000, "vocab": 50257, "width": 512, "dtype": "f32"},
        # the probe of a round: one context of 2,048 held-out tokens of the 1.08B model
        {"name": "head_probe_1b", "op": "head", "rows": 2048, "vocab": 73760, "width": 2048, "dtype": "bf16"},
        # training: the loss's gradients for a few positions of the stand
        {"name": "head_grad_few_stand", "op": "head_grad", "rows": 16, "vocab": 73760, "width": 512, "entropy": False, "dtype": "bf16"},
        # training in fp32: a batch of the Pythia-14M shape
        {"name": "head_grad_pythia_f32", "op": "head_grad", "rows": 1023, "vocab": 50304, "width": 128, "entropy": True, "dtype": "f32"},
        # training: a worker's microbatch of two contexts of the 1.08B model, with an entropy term
        {"name": "head_grad_microbatch_1b", "op": "head_grad", "rows": 4096, "vocab": 73760, "width": 2048, "entropy": True, "dtype": "bf16"},
    ]


MOST_WEIGHTS = 73760 * 2048
MOST_PRODUCTS = 2048 * 73760 * 2048
MOST_LOGITS = 4096 * 73760


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("pack8", "matmul8", "matmul8", "head", "head", "head_grad", "head_grad"))
    dtype = rng.choice(("f32", "bf16"))
    if op in ("pack8", "matmul8"):
        while True:
            rows, cols, tokens = _spread(rng, 64, 80000), _spread(rng, 64, 16384), _spread(rng, 1, 8192)
            if rows * cols <= MOST_WEIGHTS and (op == "pack8" or tokens * max(rows * cols, 1000 * (rows + cols)) <= MOST_PRODUCTS):
                break
        if op == "pack8":
            return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "values": rng.choice(("f32", "bf16"))}
        return {"op": op, "tokens": tokens, "rows": rows, "cols": cols, "dtype": dtype}
    while True:
        rows, vocab, width = _spread(rng, 1, 8192), _spread(rng, 1000, 200000), _spread(rng, 64, 4096)
        if rows * vocab <= MOST_LOGITS and vocab * width <= MOST_WEIGHTS and rows * vocab * width <= MOST_PRODUCTS:
            break
    if op == "head":
        return {"op": op, "rows": rows, "vocab": vocab, "width": width, "dtype": dtype}
    return {"op": op, "rows": rows, "vocab": vocab, "width": width, "entropy": rng.choice((False, True)), "dtype": dtype}


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(gen, rows, cols, scale):
    return torch.empty(rows, cols, device=DEV, dtype=torch.float32).normal_(0.0, scale, generator=gen)


def _probe_inputs(case, gen):
    """Hidden states and a head whose logits spread over a few units, the true
    token mostly well up; some positions carry no token (id -1)."""
    R, V, D = case["rows"], case["vocab"], case["width"]
    kind = TYPES[case["dtype"]]
    head = _normal(gen, V, D, 2.5 / math.sqrt(D))
    tokens = torch.randint(0, V, (R,), device=DEV, generator=gen)
    hidden = _normal(gen, R, D, 1.0)
    hidden += head[tokens] * (torch.rand(R, 1, device=DEV, generator=gen) * (14.0 / 6.25))
    tokens = tokens.masked_fill(torch.rand(R, device=DEV, generator=gen) < 0.1, -1)
    return hidden.to(kind), head.to(kind), tokens


def _quantised(w):
    """(q, e) of the 8-bit form, in 32 bits: q [rows, blocks, 128] as e4m3
    numbers, e [rows, blocks, 1] as int32; a short last block is filled with 0."""
    w = w.float()
    short = -w.shape[1] % BLOCK
    if short:
        w = torch.nn.functional.pad(w, (0, short))
    w = w.view(w.shape[0], -1, BLOCK)
    big = w.abs().amax(-1, keepdim=True)
    part, power = torch.frexp(big)  # big = part * 2^power, part in [0.5, 1)
    e = (power - 9 + (part > 0.875).int()).clamp_min(-126)
    fine = torch.isfinite(big)
    q = torch.ldexp(w, -e.where(fine, torch.zeros_like(e))).to(torch.float8_e4m3fn)
    if not bool(fine.all()):
        q = q.float().masked_fill(~fine, math.nan).to(torch.float8_e4m3fn)
    return q, e.where(fine, torch.zeros_like(e))


def _values(q, e, cols):
    return torch.ldexp(q.float(), e).flatten(1)[:, :cols]


def prepare(case, seed):
    gen = _generator(seed)
    op = case["op"]
    if op == "pack8":
        return {"op": op, "case": case, "w": _normal(gen, case["rows"], case["cols"], 0.02).to(TYPES[case["dtype"]])}
    if op == "matmul8":
        w = _normal(gen, case["rows"], case["cols"], 0.02)
        x = _normal(gen, case["tokens"], case["cols"], 1.0).to(TYPES[case["dtype"]])
        if own:
            from checkpoint_averaging_gb300 import binding as B

            return {"op": op, "case": case, "x": x, "w8": B.pack8(w)}
        q, e = _quantised(w)
        return {"op": op, "case": case, "x": x, "q": q, "e": e}
    hidden, head, tokens = _probe_inputs(case, gen)
    state = {"op": op, "case": case, "hidden": hidden, "head": head, "tokens": tokens}
    if op == "head_grad":
        # what the forward call left, and the gradients that reach it
        R = case["rows"]
        lse, H = [], []
        for at in range(0, R, 512):
            x = (hidden[at:at + 512].float() @ head.float().t()).double()
            lse.append(torch.logsumexp(x, -1))
            x -= lse[-1][:, None]
            H.append(-(torch.exp(x) * x).sum(-1))
            del x
        lse, H = torch.cat(lse), torch.cat(H).float()
        top = lse.float()
        state |= {"lse": top, "lse_lo": (lse - top.double()).float(), "H": H,
                  "g": -(0.5 + torch.rand(R, device=DEV, generator=gen)) / R,
                  "h": torch.full((R,), -0.01 / R, device=DEV) if case["entropy"] else None}
    return state


def _plain_head(hidden, head, tokens):
    x = hidden.float() @ head.float().t()
    m = x.amax(-1, keepdim=True)
    d = x - m
    del x
    e = torch.exp(d)
    s = e.sum(-1, keepdim=True)
    log_s = torch.log(s)
    mine = torch.gather(d, 1, tokens.clamp_min(0)[:, None])
    H = log_s - (e * d).sum(-1, keepdim=True) / s
    return {"logp": (mine - log_s)[:, 0].masked_fill(tokens < 0, 0.0), "entropy": H[:, 0], "lse": (m + log_s)[:, 0]}


def _plain_head_grad(hidden, head, tokens, lse, lse_lo, H, g, h):
    a, w = hidden.float(), head.float()
    d = a @ w.t()
    d -= lse[:, None]
    d -= lse_lo[:, None]
    p = torch.exp(d)
    g = g.masked_fill(tokens < 0, 0.0)
    G = p * -g[:, None]
    if h is not None:
        G -= h[:, None] * p * (d + H[:, None])
    del d, p
    G.scatter_add_(1, tokens.clamp_min(0)[:, None], g[:, None])
    return {"hidden": (G @ w).to(hidden.dtype), "head": (G.t() @ a).to(head.dtype)}


def run(state):
    op, case = state["op"], state["case"]
    if own:
        from checkpoint_averaging_gb300 import binding as B

        if op == "pack8":
            return B.unpack8(B.pack8(state["w"]), TYPES[case["values"]])
        if op == "matmul8":
            return B.matmul8(state["x"], state["w8"])
        if op == "head":
            r = B.head_logprobs(state["hidden"], state["head"], state["tokens"])
            return {"logp": r.logp, "entropy": r.entropy, "lse": r.lse}
        hidden, head = B.head_logprobs_backward(state["hidden"], state["head"], state["tokens"], state["lse"], state["H"],
                                                state["g"], state["h"], lse_lo=state["lse_lo"])
        return {"hidden": hidden, "head": head}
    if op == "pack8":
        return _values(*_quantised(state["w"]), case["cols"]).to(TYPES[case["values"]])
    if op == "matmul8":
        x = state["x"]
        a = _values(*_quantised(x), case["cols"])
        return (a @ _values(state["q"], state["e"], case["cols"]).t()).to(x.dtype)
    if op == "head":
        return _plain_head(state["hidden"], state["head"], state["tokens"])
    return _plain_head_grad(state["hidden"], state["head"], state["tokens"], state["lse"], state["lse_lo"], state["H"],
                            state["g"], state["h"])


def work(case):
    op = case["op"]
    size = 4 if case["dtype"] == "f32" else 2
    if op in ("pack8", "matmul8"):
        N, K = case["rows"], case["cols"]
        packed = N * K + N * -(-K // BLOCK)
        if op == "pack8":
            return {"bytes": N * K * (size + (4 if case["values"] == "f32" else 2)) + packed, "flops": 4 * N * K}
        M = case["tokens"]
        return {"bytes": packed + size * M * (N + K), "flops": 2 * M * N * K}
    R, V, D = case["rows"], case["vocab"], case["width"]
    if op == "head":
        return {"bytes": size * (R + V) * D + R * (8 + 12), "flops": 2 * R * V * D}
    return {"bytes": 2 * size * (R + V) * D + R * (8 + 16 + (4 if case["entropy"] else 0)), "flops": 6 * R * V * D}


def _exact_values(w):
    """The values of the 8-bit form, in 64 bits, by rows of blocks."""
    rows, cols = w.shape
    n = -(-cols // BLOCK)
    full = torch.zeros(rows, n * BLOCK, device=DEV, dtype=torch.float64)
    full[:, :cols] = w
    full = full.reshape(rows * n, BLOCK)
    big = full.abs().max(1, keepdim=True).values
    e = torch.ceil(torch.log2((big / 448).clamp_min(2.0 ** -126)))
    e += (448 * torch.exp2(e) < big).double()
    e -= ((448 * torch.exp2(e - 1) >= big) & (e > -126)).double()
    full *= torch.exp2(-e)
    size = full.abs()
    step = torch.floor(torch.log2(size.clamp_min(2.0 ** -6)))
    step += (torch.exp2(step + 1) <= size).double() - (torch.exp2(step) > size.clamp_min(2.0 ** -6)).double()
    step = torch.exp2(step - 3)
    full = torch.round(full / step) * step * torch.exp2(e)
    return full.reshape(rows, n * BLOCK)[:, :cols]


def exact(case, seed):
    op = case["op"]
    gen = _generator(seed)
    kind = TYPES[case["dtype"]]
    if op == "pack8":
        w = _normal(gen, case["rows"], case["cols"], 0.02).to(kind)
        return torch.cat([_exact_values(w[at:at + 8192]) for at in range(0, len(w), 8192)])
    if op == "matmul8":
        w = _normal(gen, case["rows"], case["cols"], 0.02)
        x = _exact_values(_normal(gen, case["tokens"], case["cols"], 1.0).to(kind))
        return torch.cat([torch.mm(x, _exact_values(w[at:at + 8192]).t()) for at in range(0, len(w), 8192)], 1)
    hidden, head, tokens = _probe_inputs(case, gen)
    R, V, D = case["rows"], case["vocab"], case["width"]
    w = head.double()
    if op == "head_grad":
        g = -(0.5 + torch.rand(R, device=DEV, generator=gen)) / R
        grad_hidden = torch.empty(R, D, device=DEV, dtype=torch.float64)
        grad_head = torch.zeros(V, D, device=DEV, dtype=torch.float64)
    parts = []
    for at in range(0, R, 1024):
        a, t = hidden[at:at + 1024].double(), tokens[at:at + 1024]
        x = torch.mm(a, w.t())
        lse = torch.logsumexp(x, -1)
        logp = x - lse[:, None]
        del x
        p = logp.exp()
        H = torch.special.entr(p).sum(-1)
        row = torch.arange(len(t), device=DEV)
        if op == "head":
            parts.append((torch.where(t < 0, 0.0, logp[row, t.clamp_min(0)]), H, lse))
            continue
        c = g[at:at + 1024].double() * (t >= 0)
        G = -c[:, None] * p
        G[row, t.clamp_min(0)] += c
        if case["entropy"]:
            h = torch.full((len(t), 1), -0.01 / R, device=DEV).double()
            G += h * (torch.special.entr(p) - p * H[:, None])
        del logp, p
        grad_hidden[at:at + 1024] = torch.mm(G, w)
        grad_head.addmm_(G.t(), a)
    if op == "head":
        logp, H, lse = (torch.cat(v) for v in zip(*parts))
        return {"logp": logp, "entropy": H, "lse": lse}
    return {"hidden": grad_hidden, "head": grad_head}
