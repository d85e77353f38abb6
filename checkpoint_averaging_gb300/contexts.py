"""Operators beside the merge for whole contexts, on the tensor cores: a merged
global published in 8 bits (``pack8``, ``unpack8``), its products with many
tokens (``matmul8``), and what a head says of given tokens from hidden states,
without the logits (``head_logprobs``), with the gradients of both
(``head_logprobs_backward``). All of them run in libcam's CUDA kernels
(declarations in include/cam.h); there is no fallback. They are also reached as
``binding.pack8`` and so on.

Inputs are CUDA tensors, fp32 or bf16, 2-D with contiguous rows (any row
stride). Work is queued on the current stream, or on ``stream``; tensors used
there are then recorded on it. Results are the same bits from call to call.
The calls' workspaces come from torch's allocator, for the call alone.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as _b
from . import operators as _o

_CODES, _empty, _FLOAT, _BYTE = _o._CODES, torch.empty, torch.float32, torch.uint8
_L = _b.lib()
_current_device, _current_stream = _o._current_device, _o._current_stream
_pack8, _unpack8, _matmul8 = _L.cam_pack8, _L.cam_unpack8, _L.cam_matmul8
_head, _head_backward = _L.cam_head_logprobs, _L.cam_head_logprobs_backward


# Workspaces by what decides their size (shapes, strides, dtypes, alignment): asking the library
# takes as long as an allocation.
_SIZES: dict = {}


def _workspace(key, query, *args):
    size = _SIZES.get(key)
    if size is None:
        if len(_SIZES) > 4096:
            _SIZES.clear()
        size = _SIZES[key] = _bytes(query, *args)
    return size


def _bytes(query, *args) -> int:
    out = ctypes.c_int64()
    _b._check(query(*args, ctypes.byref(out)))
    return out.value


def _no_gradient(what: str, instead: str, *tensors):
    if torch.is_grad_enabled() and any(t.requires_grad for t in tensors):
        raise ValueError(f"{what} has no gradient, and an input requires one: {instead}, or call "
                         "under torch.no_grad()")


def pack8_bytes(rows: int, cols: int) -> int:
    """The bytes of a rows x cols matrix in the 8-bit form (cam_pack8_bytes)."""
    return _bytes(_L.cam_pack8_bytes, rows, cols)


class Packed8:
    """A matrix in the 8-bit form (include/cam.h): ``data`` is its bytes (uint8,
    1-D, on the GPU), which may be saved and made a Packed8 of again, as may the
    Packed8 itself. The fields are read-only: the calls read as many bytes as
    they say."""

    __slots__ = ("_data", "_rows", "_cols", "_device", "_place")

    def __init__(self, data, rows: int, cols: int):
        if not data.is_cuda or data.dtype != torch.uint8 or not data.is_contiguous() \
                or data.data_ptr() % 16:
            raise ValueError("data must be a contiguous 16-byte aligned uint8 CUDA tensor")
        if data.numel() != pack8_bytes(rows, cols):
            raise ValueError(f"data must hold {pack8_bytes(rows, cols)} bytes")
        self._set(data, rows, cols, data.get_device())

    def _set(self, data, rows, cols, device):
        self._data, self._rows, self._cols = data, rows, cols
        self._device, self._place = device, data.device
        return self

    data = property(lambda self: self._data)
    rows = property(lambda self: self._rows)
    cols = property(lambda self: self._cols)
    shape = property(lambda self: (self._rows, self._cols))

    def __reduce__(self):  # (copies and saved files: of the bytes they come with)
        return Packed8, (self._data, self._rows, self._cols)


def pack8(weight, *, stream=None) -> Packed8:
    """The 8-bit form of a matrix (cam_pack8): a merged global's weight as it is
    published for products with whole contexts. 128 columns of a row share a
    power-of-two scale."""
    rows, cols, ld, code = _o._matrix(weight, "weight")
    device = weight.get_device()
    if stream is not None:
        return _o._on_stream(stream, device, lambda: pack8(weight), (weight,),
                             lambda packed: (packed.data,))
    if device != _current_device():
        with torch.cuda.device(device):
            return pack8(weight)
    size = _workspace((rows, cols), _L.cam_pack8_bytes, rows, cols)
    data = _empty(size, dtype=_BYTE, device=weight.device)
    rc = _pack8(rows, cols, weight.data_ptr(), ld, code, data.data_ptr(), _current_stream(device))
    if rc:
        _b._check(rc)
    return Packed8.__new__(Packed8)._set(data, rows, cols, device)


def unpack8(packed: Packed8, dtype=None, *, out=None, stream=None):
    """The values an 8-bit matrix stands for (cam_unpack8), as a new tensor of
    `dtype` (fp32 by default, or bf16) or into `out`."""
    device = packed._device
    if stream is not None:
        return _o._on_stream(stream, device, lambda: unpack8(packed, dtype, out=out),
                             (packed.data, out))
    if device != _current_device():
        with torch.cuda.device(device):
            return unpack8(packed, dtype, out=out)
    rows, cols = packed._rows, packed._cols
    if out is None:
        out = _empty((rows, cols), dtype=dtype or torch.float32, device=packed._place)
    elif tuple(out.shape) != (rows, cols) or (dtype is not None and out.dtype != dtype):
        raise ValueError("out must match the packed matrix")
    _, _, ld, code = _o._matrix(out, "out")
    _o._same_device(device, out)
    _b._check(_unpack8(rows, cols, packed._data.data_ptr(), out.data_ptr(), ld, code,
                       _current_stream(device)))
    return out


def matmul8(x, packed: Packed8, *, out=None, out_dtype=None, stream=None):
    """x W^T for an 8-bit W and many rows x (cam_matmul8), which are brought into
    the 8-bit form for it: x is [cols] or [tokens, cols]; the result is [rows] or
    [tokens, rows] in x's dtype (or `out_dtype`, or into `out`). There is no
    gradient, and an x that requires one is refused while gradients are
    recorded."""
    if x.requires_grad:
        _no_gradient("matmul8", "detach it", x)
    if out is None and out_dtype is None and stream is None and x.is_cuda:
        # the common call, with every check of the general one below
        code, shape, device = _CODES.get(x.dtype), x.shape, packed._device
        if code is not None and len(shape) == 2 and x.get_device() == device == _current_device():
            tokens, cols = shape
            ld, step = x.stride()
            if cols == packed._cols and step == 1 and ld >= cols:
                rows, place = packed._rows, packed._place
                size = _workspace((tokens, rows, cols), _L.cam_matmul8_workspace, tokens, rows, cols)
                y = _empty((tokens, rows), dtype=x.dtype, device=place)
                space = _empty(size, dtype=_BYTE, device=place)
                rc = _matmul8(tokens, rows, cols, x.data_ptr(), ld, code, packed._data.data_ptr(),
                              y.data_ptr(), rows, code, space.data_ptr(), size,
                              _current_stream(device))
                if rc:
                    _b._check(rc)
                return y
    if x.dim() == 1:
        if out is not None:
            matmul8(x.unsqueeze(0), packed, out=out.unsqueeze(0) if out.dim() == 1 else out,
                    out_dtype=out_dtype, stream=stream)
            return out
        return matmul8(x.unsqueeze(0), packed, out_dtype=out_dtype, stream=stream)[0]
    tokens, cols, ld, code = _o._matrix(x, "x")
    if cols != packed._cols:
        raise ValueError(f"x has {cols} columns, the matrix {packed._cols}")
    device = x.get_device()
    if device != packed._device:
        raise ValueError("tensors must live on one CUDA device")
    if stream is not None:
        return _o._on_stream(stream, device,
                             lambda: matmul8(x, packed, out=out, out_dtype=out_dtype),
                             (x, packed.data, out))
    if device != _current_device():
        with torch.cuda.device(device):
            return matmul8(x, packed, out=out, out_dtype=out_dtype)
    rows = packed._rows
    y = out
    if y is None:
        y = _empty((tokens, rows), dtype=out_dtype or x.dtype, device=x.device)
    elif tuple(y.shape) != (tokens, rows) or (out_dtype is not None and y.dtype != out_dtype):
        raise ValueError("out must match x and the matrix")
    _, _, ld_y, code_y = _o._matrix(y, "out")
    _o._same_device(device, y)
    size = _workspace((tokens, rows, cols), _L.cam_matmul8_workspace, tokens, rows, cols)
    space = _empty(size, dtype=torch.uint8, device=x.device)
    _b._check(_matmul8(tokens, rows, cols, x.data_ptr(), ld, code, packed._data.data_ptr(),
                       y.data_ptr(), ld_y, code_y, space.data_ptr(), size,
                       _current_stream(device)))
    return y


def _head_inputs(hidden, head, tokens):
    """(rows, vocab, width, row strides, dtype code, device) of a head's call."""
    rows, width, ld_x, code = _o._matrix(hidden, "hidden")
    vocab, width_w, ld_w, code_w = _o._matrix(head, "head")
    if width != width_w:
        raise ValueError(f"hidden has {width} columns, the head {width_w}")
    if code != code_w:
        raise ValueError("hidden and head must have one dtype")
    device = hidden.get_device()
    _o._same_device(device, head, tokens)
    if tokens is not None:
        _o._check_tokens(tokens, rows)
    return rows, vocab, width, ld_x, ld_w, code, device


def head_logprobs(hidden, head, tokens=None, *, stream=None) -> _o.TokenLogprobs:
    """token_logprobs of the logits hidden head^T, which are not stored
    (cam_head_logprobs): hidden is [rows, width], head [vocab, width], of one
    dtype; tokens is int64 [rows], a negative id is no token. No alternatives
    (`top`) are looked for. There is no gradient: inputs that require one are
    refused while gradients are recorded (probe.differentiable_head_logprobs)."""
    rows, vocab, width, ld_x, ld_w, code, device = _head_inputs(hidden, head, tokens)
    if hidden.requires_grad or head.requires_grad:
        _no_gradient("head_logprobs", "take probe.differentiable_head_logprobs", hidden, head)
    if stream is not None:
        return _o._on_stream(stream, device, lambda: head_logprobs(hidden, head, tokens),
                             (hidden, head, tokens), lambda r: (r._stats,))
    if device != _current_device():
        with torch.cuda.device(device):
            return head_logprobs(hidden, head, tokens)
    x, w, place = hidden.data_ptr(), head.data_ptr(), hidden.device
    stats = _empty((4, rows), dtype=_FLOAT, device=place)  # logp, entropy, lse, lse_lo
    at = stats.data_ptr()
    size = _workspace((rows, vocab, width, x % 16, ld_x, w % 16, ld_w, code),
                      _L.cam_head_logprobs_workspace, rows, vocab, width, x, ld_x, w, ld_w, code)
    space = _empty(size, dtype=_BYTE, device=place)
    at_token = None if tokens is None else tokens.data_ptr()
    rc = _head(rows, vocab, width, x, ld_x, w, ld_w, code, at_token,
               None if at_token is None else at, at + 4 * rows, at + 8 * rows, at + 12 * rows,
               space.data_ptr(), size, _current_stream(device))
    if rc:
        _b._check(rc)
    return _o.TokenLogprobs(stats, tokens is not None, None, None)


def head_logprobs_backward(hidden, head, tokens, lse, entropy, grad_logp=None, grad_entropy=None, *,
                           lse_lo=None, need_hidden=True, need_head=True, stream=None):
    """The gradients of head_logprobs' logp and entropy with respect to hidden
    and head (cam_head_logprobs_backward), in their dtype, as new tensors
    (grad_hidden, grad_head); None for one that is not needed. lse, entropy and
    lse_lo (optional) are as head_logprobs returned them; either gradient may be
    None, not both."""
    rows, vocab, width, ld_x, ld_w, code, device = _head_inputs(hidden, head, tokens)
    if not need_hidden and not need_head:
        return None, None
    if stream is not None:
        return _o._on_stream(
            stream, device,
            lambda: head_logprobs_backward(hidden, head, tokens, lse, entropy, grad_logp,
                                           grad_entropy, lse_lo=lse_lo, need_hidden=need_hidden,
                                           need_head=need_head),
            (hidden, head, tokens, lse, lse_lo, entropy, grad_logp, grad_entropy), lambda r: r)
    if device != _current_device():
        with torch.cuda.device(device):
            return head_logprobs_backward(hidden, head, tokens, lse, entropy, grad_logp,
                                          grad_entropy, lse_lo=lse_lo, need_hidden=need_hidden,
                                          need_head=need_head)
    shape = (rows,)
    at_lse, at_lo = _o._row_value(lse, shape, device), _o._row_value(lse_lo, shape, device)
    at_entropy = _o._row_value(entropy, shape, device)
    at_g, at_h = _o._row_value(grad_logp, shape, device), _o._row_value(grad_entropy, shape, device)
    grad_hidden = grad_head = at_hidden = at_head = None
    place = hidden.device
    if need_hidden:
        grad_hidden = _empty((rows, width), dtype=hidden.dtype, device=place)
        at_hidden = grad_hidden.data_ptr()
    if need_head:
        grad_head = _empty((vocab, width), dtype=head.dtype, device=place)
        at_head = grad_head.data_ptr()
    w = head.data_ptr()
    size = _workspace((rows, vocab, width, w % 16, ld_w, code, device),
                      _L.cam_head_logprobs_backward_workspace, rows, vocab, width, w, ld_w, code)
    space = _empty(size, dtype=_BYTE, device=place)
    rc = _head_backward(rows, vocab, width, hidden.data_ptr(), ld_x, w, ld_w, code,
                        None if tokens is None else tokens.data_ptr(), at_lse, at_lo, at_entropy,
                        at_g, at_h, at_hidden, width, at_head, width, space.data_ptr(), size,
                        _current_stream(device))
    if rc:
        _b._check(rc)
    return grad_hidden, grad_head


def operators_status() -> int:
    """The status word of this module's tensor-core kernels on the current device
    (cam_operators_status): 0 unless one has given up waiting. Waits for all work."""
    out = ctypes.c_int32()
    _b._check(_L.cam_operators_status(ctypes.byref(out)))
    return out.value
