"""A `stream` given to the calls for whole contexts: results and workspaces come from
that stream's memory, inputs are recorded on it (test_operators_streams.py has the
stand-ins and the calls for few tokens)."""
import contextlib

import pytest
import torch
from test_operators_streams import CALLER, GIVEN, Stream, Tensor

from checkpoint_averaging_gb300 import binding as B
from checkpoint_averaging_gb300 import build as cam_build


@pytest.fixture(scope="module", autouse=True)
def built():
    cam_build.build()


@pytest.fixture
def fakes(monkeypatch):
    """contexts with a fake allocator and library; what they were asked for."""
    from checkpoint_averaging_gb300 import contexts as C
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
    for module in (C, O):
        monkeypatch.setattr(module, "_current_stream", lambda device: current[-1].cuda_stream)
        monkeypatch.setattr(module, "_current_device", lambda: 0)
        monkeypatch.setattr(module, "_empty", empty)
    monkeypatch.setattr(C, "_workspace", lambda key, query, *args: 4096)
    monkeypatch.setattr(B, "_capturing", lambda stream: False)
    for name in ("_pack8", "_unpack8", "_matmul8", "_head", "_head_backward"):
        monkeypatch.setattr(C, name, launch)
    return C, made, launched


def calls(C, empty, stream):
    """[(call, its arguments' tensors)] with results of their own."""
    x, head = empty(3, 130), empty(50, 130)
    if isinstance(x, Tensor):
        w8 = C.Packed8(Tensor(C.pack8_bytes(20, 130), torch.uint8), 20, 130)
    else:
        w8 = C.pack8(empty(20, 130))
    rows = [empty(3) for _ in range(3)]
    return [(lambda: C.pack8(x, stream=stream), (x,)),
            (lambda: C.unpack8(w8, stream=stream), (w8.data,)),
            (lambda: C.matmul8(x, w8, stream=stream), (x, w8.data)),
            (lambda: C.head_logprobs(x, head, stream=stream), (x, head)),
            (lambda: C.head_logprobs_backward(x, head, None, rows[0], rows[1], None, rows[2],
                                              stream=stream), (x, head, *rows))]


def tensors_of(C, result):
    if isinstance(result, C.Packed8):
        return [result.data]
    if hasattr(result, "_stats"):
        return [result._stats]
    return list(result) if isinstance(result, tuple) else [result]


@pytest.mark.parametrize("which", range(5))
def test_results_are_allocated_under_the_given_stream(fakes, which):
    C, made, launched = fakes
    call, args = calls(C, lambda *shape: Tensor(shape), GIVEN)[which]
    result = call()
    assert launched == [GIVEN.cuda_stream]
    assert all(t.home == GIVEN.cuda_stream for t in made)  # workspaces among them
    for t in tensors_of(C, result):
        assert any(t is u for u in made)
        assert CALLER.cuda_stream in t.recorded  # where it is used and let go of
    for t in args:
        assert t.recorded == [GIVEN.cuda_stream]


@pytest.mark.parametrize("which", range(5))
def test_without_a_stream_nothing_is_recorded(fakes, which):
    C, made, launched = fakes
    call, args = calls(C, lambda *shape: Tensor(shape), None)[which]
    call()
    assert launched == [CALLER.cuda_stream]
    assert all(t.home == CALLER.cuda_stream for t in made)
    assert not any(t.recorded for t in (*made, *args))


def test_a_stream_of_another_device_is_refused(fakes):
    C, made, launched = fakes
    other = Stream(0x33)
    other.device = torch.device("cuda", 1)
    for call, _ in calls(C, lambda *shape: Tensor(shape), other):
        with pytest.raises(ValueError, match="stream"):
            call()
    assert not launched


def test_out_is_written_where_it_is(fakes):
    C, made, launched = fakes
    x, y, values = Tensor((3, 130)), Tensor((3, 20)), Tensor((20, 130))
    w8 = C.Packed8(Tensor(C.pack8_bytes(20, 130), torch.uint8), 20, 130)
    assert C.matmul8(x, w8, out=y, stream=GIVEN) is y
    assert C.unpack8(w8, out=values, stream=GIVEN) is values
    assert launched == [GIVEN.cuda_stream] * 2
    assert [t.dtype for t in made] == [torch.uint8]  # the product's workspace
    for t in (x, y, values):
        assert t.recorded == [GIVEN.cuda_stream]


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
@pytest.mark.parametrize("which", range(5))
def test_results_belong_to_the_given_stream(which):
    from checkpoint_averaging_gb300 import contexts as C

    s = torch.cuda.Stream()
    call, _ = calls(C, lambda *shape: torch.ones(shape, device="cuda"), s)[which]
    torch.cuda.synchronize()
    result = call()
    s.synchronize()
    home = {g["address"]: (g["total_size"], g["stream"]) for g in torch.cuda.memory_snapshot()}
    for t in tensors_of(C, result):
        assert [st for at, (size, st) in home.items() if at <= t.data_ptr() < at + size] == [s.cuda_stream]
