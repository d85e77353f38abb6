"""The operators beside the merge, for torch users: a merged global published
in 4 bits (``pack4``, ``unpack4``), its products with a few tokens
(``gemv4``), and what a model says of given tokens (``token_logprobs``) with
its gradient (``token_logprobs_backward``). All of them run in libcam's CUDA
kernels (declarations in include/cam.h); there is no fallback. They are also
reached as ``binding.pack4`` and so on.

Inputs are CUDA tensors, fp32 or bf16, 2-D with contiguous rows (any row
stride). Work is queued on the current stream, or on ``stream``; tensors used
there are then recorded on it. Results are the same bits from call to call.

These calls are short (a decoding step makes many of them), so the code below
asks torch for as little as it can.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as _b

LOGPROBS_MAX_TOP = _b.LOGPROBS_MAX_TOP
_CODES = {torch.float32: _b.F32, torch.bfloat16: _b.BF16}
_empty, _FLOAT, _INT64 = torch.empty, torch.float32, torch.int64
_L = _b.lib()


def _initialised_device() -> int:
    return torch.cuda.current_device()


# (current_device() but for its check that CUDA is initialised, which it is wherever a
# CUDA tensor exists)
_current_device = getattr(torch._C, "_cuda_getDevice", _initialised_device)


def _raw_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# (torch keeps the handle of the current stream without an object for it, which takes a
# twentieth of the time)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


_gemv4, _logprobs, _logprobs_backward = \
    _L.cam_gemv4, _L.cam_token_logprobs, _L.cam_token_logprobs_backward
_pack4, _unpack4 = _L.cam_pack4, _L.cam_unpack4


def _failed(rc: int):
    _b._check(rc)


def _refuse(t, what: str):
    """Raises what is wrong with a matrix argument."""
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{what} must be a 2-D CUDA tensor")
    if t.dtype not in _CODES:
        raise ValueError(f"{what} must be fp32 or bf16, not {t.dtype}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{what} must have contiguous rows")
    raise ValueError(f"{what} must not have overlapping rows")


def _matrix(t, what: str):
    """(rows, cols, elements between row starts, dtype code) of a matrix argument."""
    code, shape = _CODES.get(t.dtype), t.shape
    if code is None or len(shape) != 2 or not t.is_cuda:
        _refuse(t, what)
    rows, cols = shape
    ld, step = t.stride()
    if step != 1 and cols > 1:
        _refuse(t, what)
    if ld < cols:
        if rows > 1:
            _refuse(t, what)
        ld = cols  # (a single row's stride is never used)
    return rows, cols, ld, code


def _same_device(device: int, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError("tensors must live on one CUDA device")


def _on_stream(stream, device: int, call, args, results=lambda result: (result,)):
    """What `call` returns, called with `stream` as the current stream: a block of the
    caller's stream may still be in use by work queued there, which `stream` does not wait
    for, so results are allocated under the stream that writes them. `args` are recorded
    on `stream`, the tensors of `results(call's result)` that are not among them on the
    caller's stream, where they are used and let go of."""
    if stream.device.index != device:
        raise ValueError("stream must be one of the tensors' device")
    args = [t for t in args if t is not None]
    caller = torch.cuda.current_stream(device)
    recorded = not _b._capturing(stream)
    if recorded:
        _b._record_streams(args, stream, int(stream.cuda_stream))
    with torch.cuda.stream(stream):
        result = call()
    if recorded and caller.cuda_stream != stream.cuda_stream:
        _b._record_streams([t for t in results(result)
                            if t is not None and not any(t is u for u in args)],
                           caller, int(caller.cuda_stream))
    return result


def pack4_bytes(rows: int, cols: int, group: int = 64) -> int:
    """The bytes of a rows x cols matrix in the 4-bit form (cam_pack4_bytes)."""
    out = ctypes.c_int64()
    _b._check(_L.cam_pack4_bytes(rows, cols, group, ctypes.byref(out)))
    return out.value


class Packed4:
    """A matrix in the 4-bit form (include/cam.h): ``data`` is its bytes (uint8,
    1-D, on the GPU), which may be saved and made a Packed4 of again, as may the
    Packed4 itself. The fields are read-only: the calls read as many bytes as
    they say."""

    __slots__ = ("_data", "_rows", "_cols", "_group", "_device", "_place")

    def __init__(self, data, rows: int, cols: int, group: int):
        if not data.is_cuda or data.dtype != torch.uint8 or not data.is_contiguous() \
                or data.data_ptr() % 16:
            raise ValueError("data must be a contiguous 16-byte aligned uint8 CUDA tensor")
        if data.numel() != pack4_bytes(rows, cols, group):
            raise ValueError(f"data must hold {pack4_bytes(rows, cols, group)} bytes")
        self._set(data, rows, cols, group, data.get_device())

    def _set(self, data, rows, cols, group, device):
        self._data, self._rows, self._cols, self._group = data, rows, cols, group
        self._device, self._place = device, data.device
        return self

    data = property(lambda self: self._data)
    rows = property(lambda self: self._rows)
    cols = property(lambda self: self._cols)
    group = property(lambda self: self._group)
    shape = property(lambda self: (self._rows, self._cols))

    def __reduce__(self):  # (copies and saved files: of the bytes they come with)
        return Packed4, (self._data, self._rows, self._cols, self._group)


def pack4(weight, group: int = 64, *, stream=None) -> Packed4:
    """The 4-bit form of a matrix (cam_pack4): a merged global's weight as it is
    published. `group` columns (32, 64 or 128) share a scale."""
    rows, cols, ld, code = _matrix(weight, "weight")
    device = weight.get_device()
    if stream is not None:
        return _on_stream(stream, device, lambda: pack4(weight, group), (weight,),
                          lambda packed: (packed.data,))
    if device != _current_device():
        with torch.cuda.device(device):
            return pack4(weight, group)
    if group in (32, 64, 128):
        size = -(-rows // 16) * -(-cols // 128) * (1024 + 4096 // group)  # (cam_pack4_bytes)
    else:
        size = pack4_bytes(rows, cols, group)  # (refuses it)
    data = _empty(size, dtype=torch.uint8, device=weight.device)
    rc = _pack4(rows, cols, weight.data_ptr(), ld, code, group, data.data_ptr(),
                _current_stream(device))
    if rc:
        _failed(rc)
    return Packed4.__new__(Packed4)._set(data, rows, cols, group, device)


def unpack4(packed: Packed4, dtype=None, *, out=None, stream=None):
    """The values a 4-bit matrix stands for (cam_unpack4), as a new tensor of
    `dtype` (fp32 by default, or bf16) or into `out`."""
    device = packed._device
    if stream is not None:
        return _on_stream(stream, device, lambda: unpack4(packed, dtype, out=out),
                          (packed.data, out))
    if device != _current_device():
        with torch.cuda.device(device):
            return unpack4(packed, dtype, out=out)
    rows, cols = packed._rows, packed._cols
    if out is None:
        out = _empty((rows, cols), dtype=dtype or torch.float32, device=packed._place)
        ld, code = cols, _CODES.get(out.dtype)
        if code is None:
            _refuse(out, "values")
    else:
        if tuple(out.shape) != (rows, cols) or (dtype is not None and out.dtype != dtype):
            raise ValueError("out must match the packed matrix")
        _, _, ld, code = _matrix(out, "out")
        _same_device(device, out)
    rc = _unpack4(rows, cols, packed._data.data_ptr(), packed._group, out.data_ptr(), ld, code,
                  _current_stream(device))
    if rc:
        _failed(rc)
    return out


def gemv4(x, packed: Packed4, *, out=None, out_dtype=None, stream=None):
    """x W^T for a 4-bit W and a few rows x (cam_gemv4): x is [cols] or
    [tokens, cols]; the result is [rows] or [tokens, rows] in x's dtype (or
    `out_dtype`, or into `out`). For serving: there is no gradient, and an x that
    requires one is refused while gradients are recorded."""
    if x.requires_grad and torch.is_grad_enabled():
        raise ValueError("gemv4 has no gradient, and x requires one: detach it, or call under "
                         "torch.no_grad()")
    if out is None and out_dtype is None and stream is None:
        # the call of a decoding step, with every check of the general one below
        code, shape, device = _CODES.get(x.dtype), x.shape, packed._device
        if code is not None and len(shape) == 2 and x.get_device() == device == _current_device():
            tokens, cols = shape
            ld, step = x.stride()
            if cols == packed._cols and step == 1 and ld >= cols:
                rows = packed._rows
                y = _empty((tokens, rows), dtype=x.dtype, device=packed._place)
                rc = _gemv4(tokens, rows, cols, x.data_ptr(), ld, code, packed._data.data_ptr(),
                            packed._group, y.data_ptr(), rows, code, _current_stream(device))
                if rc:
                    _failed(rc)
                return y
    if x.dim() == 1:
        if out is not None:
            gemv4(x.unsqueeze(0), packed, out=out.unsqueeze(0) if out.dim() == 1 else out,
                  out_dtype=out_dtype, stream=stream)
            return out
        return gemv4(x.unsqueeze(0), packed, out_dtype=out_dtype, stream=stream)[0]
    tokens, cols, ld, code = _matrix(x, "x")
    if cols != packed._cols:
        raise ValueError(f"x has {cols} columns, the matrix {packed._cols}")
    device = x.get_device()
    if device != packed._device:
        raise ValueError("tensors must live on one CUDA device")
    if stream is not None:
        return _on_stream(stream, device,
                          lambda: gemv4(x, packed, out=out, out_dtype=out_dtype),
                          (x, packed.data, out))
    if device != _current_device():
        with torch.cuda.device(device):
            return gemv4(x, packed, out=out, out_dtype=out_dtype)
    rows = packed._rows
    if out is None:
        y = _empty((tokens, rows), dtype=out_dtype or x.dtype, device=x.device)
        code_y = code if out_dtype is None else _CODES.get(out_dtype)
        if code_y is None:
            _refuse(y, "out")
        ld_y = rows
    else:
        y = out
        if tuple(y.shape) != (tokens, rows) or (out_dtype is not None and y.dtype != out_dtype):
            raise ValueError("out must match x and the matrix")
        _, _, ld_y, code_y = _matrix(y, "out")
        _same_device(device, y)
    rc = _gemv4(tokens, rows, cols, x.data_ptr(), ld, code, packed._data.data_ptr(),
                packed._group, y.data_ptr(), ld_y, code_y, _current_stream(device))
    if rc:
        _failed(rc)
    return y


class TokenLogprobs:
    """What token_logprobs found, one entry per row of logits (fp32; ids int64):
    logp of the given tokens (None without tokens), entropy, lse, top_logp and
    top_ids ([rows, top], None for top = 0), and lse_lo, what rounding lse to
    fp32 left out (for the gradient). Unpacks in that order. The first three
    and the last are rows of one tensor, made when they are first asked for
    (an allocation for each takes twice the host time where they are not all read)."""

    __slots__ = ("_stats", "_rows", "top_logp", "top_ids")
    _fields = ("logp", "entropy", "lse", "top_logp", "top_ids", "lse_lo")

    def __init__(self, stats, with_tokens: bool, top_logp, top_ids):
        self._stats = stats
        self._rows = {} if with_tokens else {0: None}
        self.top_logp, self.top_ids = top_logp, top_ids

    def _row(self, i: int):
        rows = self._rows
        if i not in rows:
            rows[i] = self._stats[i]
        return rows[i]

    logp = property(lambda self: self._row(0))
    entropy = property(lambda self: self._row(1))
    lse = property(lambda self: self._row(2))
    lse_lo = property(lambda self: self._row(3))

    def __iter__(self):
        return iter([getattr(self, name) for name in self._fields])

    def __repr__(self):
        return "TokenLogprobs(" + ", ".join(f"{n}={getattr(self, n)!r}" for n in self._fields) + ")"


def _check_tokens(tokens, rows: int):
    if tokens.dtype != _INT64 or tokens.shape != (rows,) or not tokens.is_contiguous():
        raise ValueError("tokens must be a contiguous int64 tensor with one id per row")


def token_logprobs(logits, tokens=None, *, top: int = 0, stream=None) -> TokenLogprobs:
    """Log probabilities of given tokens, with the entropy and the `top` most
    likely alternatives of each row (cam_token_logprobs). logits is [rows,
    vocab]; tokens is int64 [rows], a negative id is no token."""
    rows, vocab, ld, code = _matrix(logits, "logits")
    device = logits.get_device()
    if tokens is not None:
        _check_tokens(tokens, rows)
        _same_device(device, tokens)
    if not 0 <= top <= LOGPROBS_MAX_TOP:
        raise ValueError(f"top must be in [0, {LOGPROBS_MAX_TOP}]")
    if stream is not None:
        return _on_stream(stream, device, lambda: token_logprobs(logits, tokens, top=top),
                          (logits, tokens), lambda r: (r._stats, r.top_logp, r.top_ids))
    if device != _current_device():
        with torch.cuda.device(device):
            return token_logprobs(logits, tokens, top=top)
    place = logits.device
    stats = _empty((4, rows), dtype=_FLOAT, device=place)  # logp, entropy, lse, lse_lo
    at = stats.data_ptr()
    top_logp = top_ids = at_token = at_top = at_ids = None
    if tokens is not None:
        at_token = tokens.data_ptr()
    if top:
        top_logp = _empty((rows, top), dtype=_FLOAT, device=place)
        top_ids = _empty((rows, top), dtype=_INT64, device=place)
        at_top, at_ids = top_logp.data_ptr(), top_ids.data_ptr()
    rc = _logprobs(rows, vocab, logits.data_ptr(), ld, code, at_token, top,
                   None if at_token is None else at, at + 4 * rows, at + 8 * rows, at + 12 * rows,
                   at_top, at_ids, _current_stream(device))
    if rc:
        _failed(rc)
    return TokenLogprobs(stats, tokens is not None, top_logp, top_ids)


def _row_value(t, shape, device: int):
    """The pointer of an fp32 array with one entry per row (None stays None)."""
    if t is None:
        return None
    if t.dtype is not _FLOAT or t.shape != shape or not t.is_contiguous():
        raise ValueError("lse, entropy and the gradients must be contiguous fp32, one per row")
    if t.get_device() != device:
        raise ValueError("tensors must live on one CUDA device")
    return t.data_ptr()


def token_logprobs_backward(logits, tokens, lse, entropy, grad_logp=None, grad_entropy=None, *,
                            lse_lo=None, out=None, stream=None):
    """The gradient of token_logprobs' logp and entropy with respect to the
    logits (cam_token_logprobs_backward), in the logits' dtype: a new tensor or
    into `out`, which may be `logits` itself. lse, entropy and lse_lo (optional)
    are as token_logprobs returned them; either gradient may be None, not both."""
    rows, vocab, ld, code = _matrix(logits, "logits")
    device = logits.get_device()
    if stream is not None:
        return _on_stream(
            stream, device,
            lambda: token_logprobs_backward(logits, tokens, lse, entropy, grad_logp, grad_entropy,
                                            lse_lo=lse_lo, out=out),
            (logits, tokens, lse, lse_lo, entropy, grad_logp, grad_entropy, out))
    if device != _current_device():
        with torch.cuda.device(device):
            return token_logprobs_backward(logits, tokens, lse, entropy, grad_logp, grad_entropy,
                                           lse_lo=lse_lo, out=out)
    at_token = None
    if tokens is not None:
        _check_tokens(tokens, rows)
        _same_device(device, tokens)
        at_token = tokens.data_ptr()
    shape = (rows,)
    at_lse, at_lo = _row_value(lse, shape, device), _row_value(lse_lo, shape, device)
    at_entropy = _row_value(entropy, shape, device)
    at_g, at_h = _row_value(grad_logp, shape, device), _row_value(grad_entropy, shape, device)
    if out is None:
        out = _empty((rows, vocab), dtype=logits.dtype, device=logits.device)
        ld_out = vocab
    else:
        if out.shape != logits.shape or out.dtype != logits.dtype:
            raise ValueError("out must match logits")
        ld_out = _matrix(out, "out")[2]
        _same_device(device, out)
    rc = _logprobs_backward(rows, vocab, logits.data_ptr(), ld, code, at_token, at_lse, at_lo,
                            at_entropy, at_g, at_h, out.data_ptr(), ld_out,
                            _current_stream(device))
    if rc:
        _failed(rc)
    return out
