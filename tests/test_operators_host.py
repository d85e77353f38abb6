"""Refusals of the calls beside the merge, on the host: arguments are checked
before any CUDA call, so the pointers below are never read."""
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


@pytest.mark.parametrize("group", [0, 16, 48, 256, -32])
def test_group_sizes(group):
    out = ctypes.c_int64()
    refused(B.lib().cam_pack4_bytes(1, 1, group, ctypes.byref(out)), "group")
    refused(B.lib().cam_pack4(1, 1, P, 1, B.F32, group, P, None), "group")
    refused(B.lib().cam_unpack4(1, 1, P, group, P, 1, B.F32, None), "group")
    refused(B.lib().cam_gemv4(1, 1, 1, P, 1, B.F32, P, group, P, 1, B.F32, None), "group")


@pytest.mark.parametrize("rows,cols,group,want", [
    (0, 0, 64, 0), (1, 1, 32, 1152), (16, 128, 64, 1088), (17, 129, 128, 4 * 1056),
    (73760, 2048, 64, 4610 * 16 * 1088)])
def test_bytes_of_the_form(rows, cols, group, want):
    assert B.pack4_bytes(rows, cols, group) == want


def test_bytes_refusals():
    out = ctypes.c_int64()
    refused(B.lib().cam_pack4_bytes(-1, 1, 32, ctypes.byref(out)), "rows")
    refused(B.lib().cam_pack4_bytes(1, (1 << 17) + 1, 32, ctypes.byref(out)), "cols")
    refused(B.lib().cam_pack4_bytes(1, 1, 32, None), "NULL")


@pytest.mark.parametrize("call", ["pack", "unpack"])
def test_pack_and_unpack_refusals(call):
    def f(rows=4, cols=8, m=P, ld=8, dt=B.F32, packed=P):
        if call == "pack":
            return B.lib().cam_pack4(rows, cols, m, ld, dt, 32, packed, None)
        return B.lib().cam_unpack4(rows, cols, packed, 32, m, ld, dt, None)

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


def test_gemv_refusals():
    def f(tokens=1, rows=4, cols=8, x=P, ldx=8, dx=B.F32, packed=P, y=P, ldy=4, dy=B.F32):
        return B.lib().cam_gemv4(tokens, rows, cols, x, ldx, dx, packed, 32, y, ldy, dy, None)

    refused(f(tokens=-1), "tokens")
    refused(f(tokens=1 << 19), "tokens")
    refused(f(rows=-1), "rows")
    refused(f(rows=1 << 32, ldy=1 << 32), "rows")
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
    assert f(tokens=0, x=None, packed=None, y=None) == B.OK
    assert f(rows=0, x=None, packed=None, y=None, ldy=0) == B.OK


def test_logprobs_refusals():
    def f(rows=4, vocab=8, x=P, ld=8, dt=B.F32, tokens=P, top=2, logp=P):
        return B.lib().cam_token_logprobs(rows, vocab, x, ld, dt, tokens, top, logp, P, P, P, P, P, None)

    refused(f(rows=-1), "rows")
    refused(f(vocab=0), "vocab")
    refused(f(vocab=(1 << 24) + 1, ld=1 << 25), "vocab")
    refused(f(dt=5), "dtype")
    refused(f(x=None), "logits")
    refused(f(ld=7), "stride")
    refused(f(x=P + 2), "aligned")
    refused(f(top=-1), "top")
    refused(f(top=9), "top")
    refused(f(top=33, vocab=64, ld=64), "top")
    refused(f(tokens=None), "tokens")
    assert f(rows=0, x=None) == B.OK


def test_logprobs_backward_refusals():
    def f(rows=4, vocab=8, x=P, ld=8, dt=B.F32, tokens=P, lse=P, ent=P, g=P, h=P, out=2 * P, ldo=8):
        return B.lib().cam_token_logprobs_backward(rows, vocab, x, ld, dt, tokens, lse, None, ent, g, h,
                                                   out, ldo, None)

    refused(f(rows=-1), "rows")
    refused(f(vocab=0), "vocab")
    refused(f(dt=5), "dtype")
    refused(f(x=None), "logits")
    refused(f(ld=7), "stride")
    refused(f(ldo=7), "grad_stride")
    refused(f(g=None, h=None), "both NULL")
    refused(f(lse=None), "lse")
    refused(f(out=None), "grad_logits")
    refused(f(tokens=None), "tokens")
    refused(f(ent=None), "entropy")
    refused(f(out=P + 1), "aligned")
    refused(f(out=P, ldo=16), "in place")
    assert f(rows=0, x=None, lse=None, out=None) == B.OK


def test_the_binding_refuses_host_tensors():
    with pytest.raises(ValueError, match="CUDA"):
        B.pack4(torch.zeros(4, 4))
    with pytest.raises(ValueError, match="CUDA"):
        B.token_logprobs(torch.zeros(4, 4))
    with pytest.raises(ValueError, match="CUDA"):
        B.token_logprobs_backward(torch.zeros(4, 4), None, None, None, torch.zeros(4))


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the GPU-less failure")
def test_no_gpu_fails_loudly():
    lib = B.lib()
    assert lib.cam_pack4(4, 8, P, 8, B.F32, 32, P, None) == B.E_CUDA
    assert lib.cam_gemv4(1, 4, 8, P, 8, B.F32, P, 32, P, 4, B.F32, None) == B.E_CUDA
    assert lib.cam_token_logprobs(4, 8, P, 8, B.F32, P, 0, P, P, P, None, None, None, None) == B.E_CUDA
    assert lib.cam_token_logprobs_backward(4, 8, P, 8, B.F32, P, P, None, P, P, P, P, 8, None) == B.E_CUDA
