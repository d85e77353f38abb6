"""The holder of a 4-bit matrix: its fields belong together, and the calls read
its bytes where they are at the time of the call. On the host with a stand-in
for the bytes and for the library, on the GPU with copies and saved files."""
import copy
import io
import pickle

import pytest
import torch

from checkpoint_averaging_gb300 import binding as B
from checkpoint_averaging_gb300 import build as cam_build


@pytest.fixture(scope="module", autouse=True)
def built():
    cam_build.build()


class Bytes:
    """Stands for a uint8 CUDA tensor; each has an address of its own."""
    is_cuda, dtype, device = True, torch.uint8, torch.device("cuda", 0)
    next_at = 0x100000

    def __init__(self, n):
        self.n = n
        self.move()

    def move(self):
        self.at, Bytes.next_at = Bytes.next_at, Bytes.next_at + 0x10000

    def numel(self):
        return self.n

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at

    def get_device(self):
        return 0

    def __reduce__(self):  # (a copy lies elsewhere)
        return Bytes, (self.n,)


def packed():
    return B.Packed4(Bytes(B.pack4_bytes(20, 130, 64)), 20, 130, 64)


@pytest.fixture
def read_from(monkeypatch):
    """The address that the library is given when a matrix is unpacked."""
    from checkpoint_averaging_gb300 import operators as O

    monkeypatch.setattr(O, "_current_stream", lambda device: 0)
    monkeypatch.setattr(O, "_current_device", lambda: 0)
    monkeypatch.setattr(O, "_empty", lambda shape, dtype, device: torch.empty(1))

    def address(w4):
        found = []
        monkeypatch.setattr(O, "_unpack4", lambda rows, cols, at, *rest: found.append(at) or 0)
        B.unpack4(w4)
        return found[0]

    return address


@pytest.mark.parametrize("field,value", [("data", None), ("rows", 21), ("cols", 131), ("group", 32),
                                         ("shape", (1, 1))])
def test_fields_are_read_only(field, value):
    w4 = packed()
    with pytest.raises(AttributeError):
        setattr(w4, field, value)
    assert (w4.rows, w4.cols, w4.group, w4.shape) == (20, 130, 64, (20, 130))


@pytest.mark.parametrize("how", [copy.deepcopy, lambda w4: pickle.loads(pickle.dumps(w4))])
def test_a_copy_reads_its_own_bytes(read_from, how):
    w4 = packed()
    other = how(w4)
    assert other.data is not w4.data and other.data.data_ptr() != w4.data.data_ptr()
    assert read_from(other) == other.data.data_ptr()
    assert read_from(w4) == w4.data.data_ptr()
    assert (other.rows, other.cols, other.group) == (20, 130, 64)


def test_bytes_that_moved_are_read_where_they_are(read_from):
    w4 = packed()
    w4.data.move()
    assert read_from(w4) == w4.data.data_ptr()


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
def test_copies_and_saved_matrices_stand_for_the_same_values():
    w = torch.randn(40, 300, generator=torch.Generator().manual_seed(8)).cuda()
    x = torch.randn(2, 300, generator=torch.Generator().manual_seed(9)).cuda()
    w4 = B.pack4(w, 64)
    values, y = B.unpack4(w4), B.gemv4(x, w4)
    file = io.BytesIO()
    torch.save(w4, file)
    file.seek(0)
    for other in (copy.copy(w4), copy.deepcopy(w4), torch.load(file, weights_only=False)):
        assert torch.equal(B.unpack4(other), values)
        if other.data is not w4.data:
            other.data.zero_()
            assert not torch.equal(B.gemv4(x, other), y)
            assert torch.equal(B.gemv4(x, w4), y)
