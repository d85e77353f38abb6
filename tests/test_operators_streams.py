"""A `stream` given to the calls beside the merge: their results come from that
stream's memory. A block of the caller's stream may still be in use by work
queued there, which the given stream does not wait for. On the host by the
stream that the allocator is asked with, on the GPU by the stream that the
result's memory belongs to."""
import contextlib

import pytest
import torch

from checkpoint_averaging_gb300 import binding as B
from checkpoint_averaging_gb300 import build as cam_build


@pytest.fixture(scope="module", autouse=True)
def built():
    cam_build.build()


class Stream:
    def __init__(self, handle):
        self.cuda_stream, self.device = handle, torch.device("cuda", 0)


class Tensor:
    """What the calls ask of a CUDA tensor; `recorded`: the streams it was recorded on."""
    is_cuda, device, requires_grad = True, torch.device("cuda", 0), False

    def __init__(self, shape, dtype=torch.float32, home=None):
        self.shape = torch.Size(shape if isinstance(shape, tuple) else (shape,))
        self.dtype, self.home, self.recorded = dtype, home, []

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def get_device(self):
        return 0

    def data_ptr(self):
        return 0x100000

    def is_contiguous(self):
        return True

    def record_stream(self, stream):
        self.recorded.append(stream.cuda_stream)

    def __getitem__(self, i):
        return Tensor(tuple(self.shape[1:]), self.dtype)


CALLER, GIVEN = Stream(0x11), Stream(0x22)


@pytest.fixture
def fakes(monkeypatch):
    """operators with a fake allocator and library; what they were asked for."""
    from checkpoint_averaging_gb300 import operators as O

    current, made, launched = [CALLER], [], []

    @contextlib.contextmanager
    def under(stream):
        current.append(stream)
        yield
        current.pop()

    def empty(shape, dtype, device):
        made.append(Tensor(shape, dtype, current[-1].cuda_stream))
        return made[-1]

    def launch(*args):
        launched.append(args[-1])
        return 0

    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(O, "_current_stream", lambda device: current[-1].cuda_stream)
    monkeypatch.setattr(O, "_current_device", lambda: 0)
    monkeypatch.setattr(O, "_empty", empty)
    monkeypatch.setattr(B, "_capturing", lambda stream: False)
    for name in ("_pack4", "_unpack4", "_gemv4", "_logprobs", "_logprobs_backward"):
        monkeypatch.setattr(O, name, launch)
    return O, made, launched


def packed_of(O):
    size = O.pack4_bytes(20, 130, 64)
    return O.Packed4(Tensor(size, torch.uint8), 20, 130, 64)


def calls(O, empty, stream):
    """[(call, its arguments' tensors)] with results of their own."""
    x, logits = empty(3, 130), empty(4, 50)
    w4 = packed_of(O) if isinstance(x, Tensor) else O.pack4(empty(20, 130), 64)
    rows = [empty(4) for _ in range(3)]
    return [(lambda: O.pack4(x, 64, stream=stream), (x,)),
            (lambda: O.unpack4(w4, stream=stream), (w4.data,)),
            (lambda: O.gemv4(x, w4, stream=stream), (x, w4.data)),
            (lambda: O.token_logprobs(logits, top=3, stream=stream), (logits,)),
            (lambda: O.token_logprobs_backward(logits, None, rows[0], rows[1], None, rows[2],
                                               stream=stream), (logits, *rows))]


def tensors_of(O, result):
    if isinstance(result, O.Packed4):
        return [result.data]
    if isinstance(result, O.TokenLogprobs):
        return [result._stats, result.top_logp, result.top_ids]
    return [result]


@pytest.mark.parametrize("which", range(5))
def test_results_are_allocated_under_the_given_stream(fakes, which):
    O, made, launched = fakes
    call, args = calls(O, lambda *shape: Tensor(shape), GIVEN)[which]
    result = call()
    assert launched == [GIVEN.cuda_stream]
    found = tensors_of(O, result)
    assert len(made) == len(found) and all(a is b for a, b in zip(made, found))
    for t in found:
        assert t.home == GIVEN.cuda_stream
        assert CALLER.cuda_stream in t.recorded  # where it is used and let go of
    for t in args:
        assert t.recorded == [GIVEN.cuda_stream]


@pytest.mark.parametrize("which", range(5))
def test_without_a_stream_nothing_is_recorded(fakes, which):
    O, made, launched = fakes
    call, args = calls(O, lambda *shape: Tensor(shape), None)[which]
    call()
    assert launched == [CALLER.cuda_stream]
    assert all(t.home == CALLER.cuda_stream for t in made)
    assert not any(t.recorded for t in (*made, *args))


def test_a_stream_of_another_device_is_refused(fakes):
    O, made, launched = fakes
    other = Stream(0x33)
    other.device = torch.device("cuda", 1)
    for call, _ in calls(O, lambda *shape: Tensor(shape), other):
        with pytest.raises(ValueError, match="stream"):
            call()
    assert not launched


def test_out_is_written_where_it_is(fakes):
    O, made, launched = fakes
    x, logits, rows = Tensor((3, 130)), Tensor((4, 50)), Tensor((4,))
    y, values = Tensor((3, 20)), Tensor((20, 130))
    w4 = packed_of(O)
    assert O.gemv4(x, w4, out=y, stream=GIVEN) is y
    assert O.unpack4(w4, out=values, stream=GIVEN) is values
    assert O.token_logprobs_backward(logits, None, rows, rows, None, rows, out=logits,
                                     stream=GIVEN) is logits
    assert launched == [GIVEN.cuda_stream] * 3 and not made
    for t in (x, y, values, logits, rows):
        assert t.recorded == [GIVEN.cuda_stream]


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
@pytest.mark.parametrize("which", range(5))
def test_results_belong_to_the_given_stream(which):
    from checkpoint_averaging_gb300 import operators as O

    s = torch.cuda.Stream()
    call, _ = calls(O, lambda *shape: torch.ones(shape, device="cuda"), s)[which]
    torch.cuda.synchronize()
    result = call()
    s.synchronize()
    home = {}
    for segment in torch.cuda.memory_snapshot():
        home[segment["address"]] = (segment["total_size"], segment["stream"])
    for t in tensors_of(O, result):
        stream = [st for at, (size, st) in home.items() if at <= t.data_ptr() < at + size]
        assert stream == [s.cuda_stream]
