"""Refusals of the calls for whole contexts (8-bit form, its products, a head's log
probabilities), on the host: arguments are checked before any CUDA call, so the
pointers below are never read."""
import ctypes

import pytest
import torch

from checkpoint_averaging_gb300 import binding as B
from checkpoint_averaging_gb300 import build as cam_build

P = 0x10000  # a pointer that is never read


@pytest.fixture(scope="module", autouse=True)
def built():
    cam_build.build()


def refused(rc, text):
    assert rc == B.E_ARG
    assert text in B.last_error()


@pytest.mark.parametrize("rows,cols,want", [
    (0, 0, 0), (0, 5, 0), (5, 0, 0), (1, 1, 512 + 512), (16, 128, 2048 + 512), (129, 129, 18944 + 4 * 512),
    (73760, 2048, 73760 * 2048 + 577 * 16 * 512)])
def test_bytes_of_the_form(rows, cols, want):
    assert B.pack8_bytes(rows, cols) == want


def test_bytes_refusals():
    out = ctypes.c_int64()
    refused(B.lib().cam_pack8_bytes(-1, 1, ctypes.byref(out)), "rows")
    refused(B.lib().cam_pack8_bytes((1 << 31) + 1, 1, ctypes.byref(out)), "rows")
    refused(B.lib().cam_pack8_bytes(1, (1 << 17) + 1, ctypes.byref(out)), "cols")
    refused(B.lib().cam_pack8_bytes(1, 1, None), "NULL")


@pytest.mark.parametrize("call", ["pack", "unpack"])
def test_pack_and_unpack_refusals(call):
    def f(rows=4, cols=8, m=P, ld=8, dt=B.F32, packed=P):
        if call == "pack":
            return B.lib().cam_pack8(rows, cols, m, ld, dt, packed, None)
        return B.lib().cam_unpack8(rows, cols, packed, m, ld, dt, None)

    refused(f(rows=-1), "rows")
    refused(f(cols=-1), "cols")
    refused(f(dt=7), "dtype")
    refused(f(m=None), "NULL")
    refused(f(packed=None), "NULL")
    refused(f(ld=7), "stride")
    refused(f(ld=1 << 60), "stride")
    refused(f(packed=P + 8), "16-byte")
    refused(f(m=P + 1), "aligned")
    refused(f(m=P + 1, dt=B.BF16), "aligned")
    assert f(rows=0, m=None, packed=None) == B.OK      # nothing to do
    assert f(cols=0, m=None, packed=None, ld=0) == B.OK


def test_matmul_refusals():
    def f(tokens=1, rows=4, cols=8, x=P, ldx=8, dx=B.F32, packed=P, y=P, ldy=4, dy=B.F32, ws=P,
          size=1 << 20):
        return B.lib().cam_matmul8(tokens, rows, cols, x, ldx, dx, packed, y, ldy, dy, ws, size, None)

    refused(f(tokens=-1), "tokens")
    refused(f(tokens=1 << 25), "tokens")
    refused(f(rows=-1), "rows")
    refused(f(rows=1 << 32, ldy=1 << 32), "rows")
    refused(f(tokens=1 << 24, rows=1 << 31, ldy=1 << 31), "tokens and rows")
    refused(f(cols=-1), "cols")
    refused(f(dx=2), "dtype")
    refused(f(dy=-1), "dtype")
    refused(f(x=None), "NULL")
    refused(f(packed=None), "NULL")
    refused(f(y=None), "NULL")
    refused(f(ldx=7), "stride")
    refused(f(ldy=3), "stride")
    refused(f(packed=P + 4), "16-byte")
    refused(f(x=P + 2), "aligned")
    refused(f(y=P + 1, dy=B.BF16), "aligned")
    refused(f(ws=None), "workspace")
    refused(f(ws=P + 16), "workspace")
    refused(f(size=1023), "workspace")
    assert f(tokens=0, x=None, packed=None, y=None, ws=None, size=0) == B.OK
    assert f(rows=0, x=None, packed=None, y=None, ldy=0, ws=None, size=0) == B.OK
    out = ctypes.c_int64()
    refused(B.lib().cam_matmul8_workspace(-1, 1, 1, ctypes.byref(out)), "tokens")
    refused(B.lib().cam_matmul8_workspace(1, 1, 1, None), "NULL")
    assert B.lib().cam_matmul8_workspace(1, 4, 8, ctypes.byref(out)) == B.OK and out.value == 1024


def head_workspace(rows=4, vocab=300, width=64, x=P, ldx=64, w=P, ldw=64, dt=B.BF16):
    out = ctypes.c_int64()
    rc = B.lib().cam_head_logprobs_workspace(rows, vocab, width, x, ldx, w, ldw, dt, ctypes.byref(out))
    assert rc == B.OK
    return out.value


def test_head_refusals():
    def f(rows=4, vocab=300, width=64, x=P, ldx=64, w=2 * P, ldw=64, dt=B.BF16, tokens=P, logp=P, ws=P,
          size=1 << 40):
        return B.lib().cam_head_logprobs(rows, vocab, width, x, ldx, w, ldw, dt, tokens, logp, P, P, P,
                                         ws, size, None)

    refused(f(rows=-1), "rows")
    refused(f(rows=(1 << 24) + 1), "rows")
    refused(f(vocab=0), "vocab")
    refused(f(vocab=(1 << 24) + 1), "vocab")
    refused(f(rows=1 << 24, vocab=1 << 24), "rows and vocab")
    refused(f(width=0), "width")
    refused(f(width=(1 << 17) + 1, ldx=1 << 18, ldw=1 << 18), "width")
    refused(f(dt=5), "dtype")
    refused(f(x=None), "NULL")
    refused(f(w=None), "NULL")
    refused(f(ldx=63), "stride")
    refused(f(ldw=63), "stride")
    refused(f(x=P + 1), "aligned")
    refused(f(w=P + 2, dt=B.F32), "aligned")
    refused(f(tokens=None), "tokens")
    refused(f(logp=None), "tokens")
    refused(f(ws=None), "workspace")
    refused(f(ws=P + 128), "workspace")
    refused(f(size=head_workspace() - 1), "workspace")
    assert f(rows=0, x=None, w=None, ws=None, size=0) == B.OK
    assert B.lib().cam_head_logprobs_workspace(1, 1, 1, P, 1, P, 1, B.F32, None) == B.E_ARG


def test_head_workspaces():
    # copies where rows do not start on 16 bytes, and of fp32 in three terms
    more = head_workspace(ldw=65) - head_workspace()
    assert more == 300 * 64 * 2
    assert head_workspace(x=P + 2) - head_workspace() == 512
    assert head_workspace(200, dt=B.F32) - head_workspace(200) == 3 * (300 + 200) * 64 * 2
    assert head_workspace(dt=B.F32) - head_workspace() == 3 * (300 + 4) * 64 * 2
    # few rows over 2^23 elements, above 64 rows of more than 512 each: the head as it is
    for rows, vocab, width, direct in ((4, 1 << 17, 64, True), (4, (1 << 17) - 1, 64, False), (64, 1 << 17, 64, True),
                                       (65, 1 << 17, 64, False), (65, 1 << 14, 512, False),
                                       (128, 1 << 14, 576, True), (129, 1 << 14, 576, False)):
        size = {"rows": rows, "vocab": vocab, "width": width, "ldx": width, "ldw": width}
        # (the statistics of `few` rows' calls are for 32 tokens each, of others for 256)
        parts = (vocab + 31) // 32 if direct or rows <= 64 else (vocab + 255) // 256
        padded = lambda n: (n + 511) // 512 * 512
        want = padded(3 * rows * width * 2) + padded(parts * rows * 16) + padded(rows * 4)
        if not direct:
            want += padded(3 * vocab * width * 2)
        assert head_workspace(dt=B.F32, **size) == want
    # a piece of the head, not all of it
    assert head_workspace(200, vocab=1 << 22, width=1024, ldx=1024, ldw=1024, dt=B.F32) < (1 << 29) + (1 << 20) \
        + (1 << 22) // 256 * 200 * 16


def test_head_backward_refusals():
    def f(rows=4, vocab=300, width=64, x=P, ldx=64, w=2 * P, ldw=64, dt=B.BF16, tokens=P, lse=P, ent=P,
          g=P, h=P, gx=3 * P, ldgx=64, gw=4 * P, ldgw=64, ws=P):
        return B.lib().cam_head_logprobs_backward(rows, vocab, width, x, ldx, w, ldw, dt, tokens, lse,
                                                  None, ent, g, h, gx, ldgx, gw, ldgw, ws, 0, None)

    refused(f(rows=-1), "rows")
    refused(f(vocab=0), "vocab")
    refused(f(width=0), "width")
    refused(f(dt=5), "dtype")
    refused(f(x=None), "NULL")
    refused(f(ldx=63), "stride")
    refused(f(ldgx=63), "stride")
    refused(f(ldgw=63), "stride")
    refused(f(g=None, h=None), "both NULL")
    refused(f(gx=None, gw=None), "both NULL")
    refused(f(lse=None), "lse")
    refused(f(tokens=None), "tokens")
    refused(f(ent=None), "entropy")
    refused(f(gx=3 * P + 1), "aligned")
    refused(f(gx=P), "place of an input")
    refused(f(gw=2 * P), "place of an input")
    refused(f(ws=None), "workspace")
    assert f(rows=0, x=None, w=None, lse=None, gw=None) == B.OK
    assert B.lib().cam_head_logprobs_backward_workspace(1, 1, 1, P, 1, B.F32, None) == B.E_ARG


def test_status_refusal():
    assert B.lib().cam_operators_status(None) == B.E_ARG


def test_the_binding_refuses_host_tensors():
    for call in (lambda: B.pack8(torch.zeros(4, 4)),
                 lambda: B.matmul8(torch.zeros(4, 4), None),
                 lambda: B.head_logprobs(torch.zeros(4, 4), torch.zeros(5, 4)),
                 lambda: B.head_logprobs_backward(torch.zeros(4, 4), torch.zeros(5, 4), None, None, None)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the GPU-less failure")
def test_no_gpu_fails_loudly():
    lib = B.lib()
    assert lib.cam_pack8(4, 8, P, 8, B.F32, P, None) == B.E_CUDA
    assert lib.cam_unpack8(4, 8, P, P, 8, B.F32, None) == B.E_CUDA
    assert lib.cam_matmul8(1, 4, 8, P, 8, B.F32, P, P, 4, B.F32, P, 1 << 20, None) == B.E_CUDA
    assert lib.cam_head_logprobs(4, 300, 64, P, 64, P, 64, B.BF16, P, P, P, P, P, P, 1 << 40, None) == B.E_CUDA
    assert lib.cam_head_logprobs_backward(4, 300, 64, P, 64, P, 64, B.BF16, P, P, None, P, P, P, 2 * P, 64,
                                          3 * P, 64, P, 1 << 40, None) == B.E_CUDA
    out = ctypes.c_int32()
    assert lib.cam_operators_status(ctypes.byref(out)) == B.E_CUDA
