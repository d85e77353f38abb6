"""The operators for whole contexts called by several host threads at once, each on a
stream of its own: the bits of the same calls one after another."""
import threading

import pytest
import torch

from checkpoint_averaging_gb300 import binding as B

pytestmark = pytest.mark.gpu


def _calls(seed, rows, vocab, width, dtype):
    gen = torch.Generator("cuda").manual_seed(seed)
    hidden = torch.randn(rows, width, device="cuda", generator=gen).to(dtype)
    head = (torch.randn(vocab, width, device="cuda", generator=gen) * 0.1).to(dtype)
    tokens = torch.randint(vocab, (rows,), device="cuda", generator=gen)
    g = torch.randn(rows, device="cuda", generator=gen)
    h = torch.randn(rows, device="cuda", generator=gen)

    def run():
        w8 = B.pack8(head)
        r = B.head_logprobs(hidden, head, tokens)
        dx, dw = B.head_logprobs_backward(hidden, head, tokens, r.lse, r.entropy, g, h,
                                          lse_lo=r.lse_lo)
        return [B.unpack8(w8), B.matmul8(hidden, w8), r.logp, r.entropy, r.lse, dx, dw]

    return run


def test_calls_by_several_threads():
    # sizes of both forms (few rows and many), both types
    cases = [(3, 1000, 131, torch.float32), (200, 2001, 96, torch.bfloat16),
             (40, 999, 72, torch.bfloat16), (300, 1500, 40, torch.float32)]
    runs = [_calls(i, *case) for i, case in enumerate(cases)]
    wanted = [run() for run in runs]
    torch.cuda.synchronize()
    got, errors = [[] for _ in runs], []
    start = threading.Barrier(len(runs))

    def work(i):
        try:
            stream = torch.cuda.Stream()
            start.wait(60)
            with torch.cuda.stream(stream):
                for _ in range(10):
                    got[i].append(runs[i]())
            stream.synchronize()
        except Exception as e:  # (an assertion of this thread would not reach the test)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(runs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not errors and not any(t.is_alive() for t in threads)
    for i, want in enumerate(wanted):
        assert len(got[i]) == 10
        for result in got[i]:
            for a, b in zip(want, result):
                assert torch.equal(a, b)
    assert B.operators_status() == 0
