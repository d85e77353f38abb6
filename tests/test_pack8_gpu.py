"""The 8-bit form and its products on the GPU, against the definitions in 64 bits
(include/cam.h). The form is exact: scales are powers of two and e4m3 rounds once.
A product's terms are exact; its sum runs over cols / 32 tensor-core steps, each of
which keeps 24 bits of the sum so far and of its own 32 terms (two roundings of at
most 2^-23 of sum |x w| a step), and a result in bf16 rounds by 2^-8 of itself:
tolerance (2 ceil(cols / 32) + 16) 2^-23 sum |x w| (+ 2^-8 |y|)."""
import copy
import io
import math

import pytest
import torch

from checkpoint_averaging_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    yield
    torch.cuda.synchronize()
    assert B.operators_status() == 0


def values(w):
    """What a matrix stands for in the 8-bit form, in 64 bits on the CPU."""
    w = w.detach().double().cpu()
    rows, cols = w.shape
    n = -(-cols // 128)
    full = torch.zeros(rows, n * 128, dtype=torch.float64)
    full[:, :cols] = w
    full = full.view(rows, n, 128)
    big = full.abs().amax(2, keepdim=True)
    fine = torch.isfinite(big)
    size = big.where(fine, torch.ones_like(big))
    part, power = torch.frexp(size)  # size = part 2^power, 1/2 <= part < 1
    e = (power - 9 + (part > 0.875)).clamp(min=-126).double()
    q = full.where(fine, torch.zeros_like(full)) * torch.exp2(-e)
    _, power = torch.frexp(q)
    step = torch.exp2((power - 1).clamp(min=-6).double() - 3)
    q = torch.round(q / step) * step  # (torch.round: ties to even)
    q = torch.where(e == 120, q.clamp(-240, 240), q)
    out = (q * torch.exp2(e)).masked_fill(~fine, math.nan)
    return out.view(rows, n * 128)[:, :cols]


def same(got, want):
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))


def rand(rows, cols, seed, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, cols, generator=g) * scale).to(dtype).to(DEV)


SHAPES = [(1, 1), (1, 128), (3, 127), (5, 129), (31, 16), (32, 17), (33, 300), (127, 64), (128, 128),
          (129, 257), (257, 1000), (512, 512), (1000, 1413), (4, 16384)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_the_form(rows, cols, dtype):
    w = rand(rows, cols, rows + cols, dtype, 0.02)
    packed = B.pack8(w)
    assert packed.shape == (rows, cols) and packed.data.numel() == B.pack8_bytes(rows, cols)
    want = values(w)
    same(B.unpack8(packed), want)
    same(B.unpack8(packed, BF16), want)  # four significant bits: exact
    assert torch.equal(packed.data[:rows * -(-cols // 16) * 16], B.pack8(w).data[:rows * -(-cols // 16) * 16])
    same(B.unpack8(B.pack8(B.unpack8(packed))), want)  # what is in the form stays


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 2), (4, 0), (8, 4)])
def test_strides_and_alignment(pad, offset, dtype):
    rows, cols = 67, 203
    base = rand(rows, cols + pad + offset, 5, dtype)
    w = base[:, offset:offset + cols]
    want = values(w)
    same(B.unpack8(B.pack8(w)), want)
    room = torch.full((rows, cols + pad + offset), 7.0, dtype=dtype, device=DEV)
    B.unpack8(B.pack8(w), out=room[:, offset:offset + cols])
    same(room[:, offset:offset + cols], want.to(dtype).double())
    assert (room[:, :offset] == 7).all() and (room[:, offset + cols:] == 7).all()


def test_values_of_every_kind():
    w = torch.zeros(12, 300)
    w[1, 5] = math.nan
    w[2, 130] = math.inf
    w[3, 299] = -math.inf
    w[4] = 448.0 * 2.0 ** torch.arange(300).remainder(3)       # at the border of a scale
    w[5, :128] = torch.tensor(448.0 * 2.0 ** -3).nextafter(torch.tensor(1e9))
    w[6] = 3.4028234e38                                        # the largest
    w[7] = 1e-45                                               # the smallest
    w[8] = 2.0 ** -126 * 448
    w[9] = torch.linspace(-1, 1, 300)
    w[10, ::7] = 1e-30                                         # lost beside 1
    w[10, 0] = 1.0
    w[11] = -0.0
    w = w.to(DEV)
    same(B.unpack8(B.pack8(w)), values(w))
    # every e4m3 number, and the middles between neighbours
    q = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    both = torch.cat([q, (q[1:] + q[:-1]) / 2, torch.full((1,), 448.0, dtype=torch.float64)])
    table = torch.zeros(2, 256)
    table[0, :len(both) // 2 + 1] = both[:len(both) // 2 + 1].float()
    table[1, :len(both) - len(both) // 2] = both[len(both) // 2:].float()
    table[:, 127] = table[:, 255] = 448.0
    table = table.to(DEV)
    same(B.unpack8(B.pack8(table)), values(table))
    same(B.unpack8(B.pack8(-table)), values(-table))


def check(x, w, dtype=None, y=None):
    packed = B.pack8(w)
    if y is None:
        y = B.matmul8(x, packed, out_dtype=dtype)
    else:
        assert B.matmul8(x, packed, out=y) is y
    a, b = values(x), values(w)
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    tol = (2 * -(-x.shape[1] // 32) + 16) * 2.0 ** -23 * size
    if y.dtype == BF16:
        tol += 2.0 ** -8 * want.abs()
    got = y.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    off = ((got - want).abs() - tol).nan_to_num(0.0)
    assert not off.numel() or off.max() <= 0, off.max()
    return y


PRODUCTS = [(1, 1, 1), (1, 500, 128), (2, 192, 64), (16, 512, 1408), (127, 193, 257), (128, 384, 130),
            (129, 192, 128), (130, 191, 127), (256, 576, 300), (257, 385, 1000), (500, 1001, 513),
            (3, 20000, 70), (1000, 100, 16384)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,rows,cols", PRODUCTS)
def test_products(tokens, rows, cols, dtype):
    x, w = rand(tokens, cols, 1, dtype), rand(rows, cols, 2, dtype, 0.02)
    # rows of very different sizes: each block has its own scale
    x *= torch.exp2(torch.arange(tokens, device=DEV).remainder(40) - 20)[:, None].to(dtype)
    w *= torch.exp2(torch.arange(rows, device=DEV).remainder(50) - 25)[:, None].to(dtype)
    y = check(x, w)
    assert y.dtype == dtype
    assert torch.equal(y, B.matmul8(x, B.pack8(w)))  # the same bits again


def test_blocks_of_very_different_sizes():
    x, w = rand(200, 640, 3), rand(300, 640, 4)
    scale = torch.exp2(torch.arange(5, device=DEV) * 9.0 - 18).repeat_interleave(128)
    check(x * scale, w)
    check(x * scale, w / scale)


@pytest.mark.parametrize("tokens", [5, 200])
@pytest.mark.parametrize("out", [F32, BF16])
def test_strides_of_products(tokens, out):
    x = rand(tokens, 333, 6)[:, 3:303]
    w = rand(210, 300, 7)
    for pad, offset in ((0, 0), (1, 0), (16, 16), (5, 3)):
        room = torch.full((tokens, 210 + pad + offset), 9.0, dtype=out, device=DEV)
        check(x, w, y=room[:, offset:offset + 210])
        assert (room[:, :offset] == 9).all() and (room[:, offset + 210:] == 9).all()
    check(x, w, BF16 if out is F32 else F32)
    y = torch.full((tokens + 2, 210), 9.0, dtype=out, device=DEV)  # rows behind stay
    check(x, w, y=y[:tokens])
    assert (y[tokens:] == 9).all()


@pytest.mark.parametrize("tokens", [5, 200])
@pytest.mark.parametrize("rows", [193, 222, 223, 224])
@pytest.mark.parametrize("pad, offset", [(0, 0), (0, 1), (1, 0), (1, 1), (2, 2)])
def test_results_that_start_between_words(tokens, rows, pad, offset):
    # bf16 rows on even and odd elements, whose last part has 1, 30, 31 or 32 columns
    x, w = rand(tokens, 300, 6), rand(rows, 300, 7)
    ld = rows + pad + (rows & 1) + offset
    room = torch.full((tokens + 1, ld), 9.0, dtype=BF16, device=DEV)
    check(x, w, y=room[:tokens, offset:offset + rows])
    assert (room[:tokens, :offset] == 9).all() and (room[:tokens, offset + rows:] == 9).all()
    assert (room[tokens] == 9).all()


@pytest.mark.parametrize("tokens", [5, 200])
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("rows", range(217, 225))
def test_columns_beside_a_result_stay(tokens, out, rows):
    # rows that start on 16 bytes and end anywhere
    x, w = rand(tokens, 300, 6), rand(rows, 300, 7)
    room = torch.full((tokens + 1, 240), 9.0, dtype=out, device=DEV)
    check(x, w, y=room[:tokens, :rows])
    assert (room[:tokens, rows:] == 9).all() and (room[tokens] == 9).all()


def test_broken_blocks_stay_visible():
    x, w = rand(200, 300, 8), rand(400, 300, 9)
    x[7, 290], x[150, 0] = math.nan, math.inf
    w[33, 140], w[399, 299] = -math.inf, math.nan
    y = check(x, w)
    assert torch.isnan(y[7]).all() and torch.isnan(y[:, 33]).all()
    assert int(torch.isnan(y).sum()) == 2 * 400 + 2 * 198


def test_empty_and_vectors():
    w = B.pack8(rand(50, 60, 1))
    assert B.matmul8(torch.empty(0, 60, device=DEV), w).shape == (0, 50)
    x = rand(1, 60, 2)
    assert torch.equal(B.matmul8(x[0], w), B.matmul8(x, w)[0])
    room = torch.empty(50, device=DEV)
    assert B.matmul8(x[0], w, out=room) is room and torch.equal(room, B.matmul8(x, w)[0])
    none = B.pack8(torch.empty(50, 0, device=DEV))
    assert torch.equal(B.matmul8(torch.empty(3, 0, device=DEV), none), torch.zeros(3, 50, device=DEV))
    assert B.matmul8(x, B.pack8(torch.empty(0, 60, device=DEV))).shape == (1, 0)


def test_refusals():
    w = B.pack8(rand(50, 60, 1))
    x = rand(4, 60, 2)
    with pytest.raises(ValueError, match="columns"):
        B.matmul8(rand(4, 61, 2), w)
    with pytest.raises(ValueError, match="fp32 or bf16"):
        B.matmul8(x.half(), w)
    with pytest.raises(ValueError, match="contiguous rows"):
        B.matmul8(rand(60, 4, 2).t(), w)
    with pytest.raises(ValueError, match="match"):
        B.matmul8(x, w, out=torch.empty(4, 51, device=DEV))
    with pytest.raises(ValueError, match="match"):
        B.unpack8(w, out=torch.empty(4, 51, device=DEV))
    with pytest.raises(ValueError, match="gradient"):
        B.matmul8(x.clone().requires_grad_(True), w)
    with torch.no_grad():
        B.matmul8(x.clone().requires_grad_(True), w)
    with pytest.raises(ValueError, match="bytes"):
        B.Packed8(w.data[:-512], 50, 60)
    with pytest.raises(ValueError, match="uint8"):
        B.Packed8(w.data.float(), 50, 60)
    with pytest.raises(AttributeError):
        w.rows = 3


def test_copies_and_saved_matrices():
    w = B.pack8(rand(50, 300, 1))
    x = rand(200, 300, 2)
    want = B.matmul8(x, w)
    file = io.BytesIO()
    torch.save(w, file)
    file.seek(0)
    for other in (copy.copy(w), copy.deepcopy(w), torch.load(file, weights_only=False),
                  B.Packed8(w.data.clone(), 50, 300)):
        assert other.shape == (50, 300) and torch.equal(B.matmul8(x, other), want)


def test_other_streams_and_graphs():
    x, w = rand(300, 520, 1, BF16), rand(700, 520, 2, BF16)
    want = B.matmul8(x, B.pack8(w))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    packed = B.pack8(w, stream=s)
    y = B.matmul8(x, packed, stream=s)
    v = B.unpack8(packed, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want) and torch.equal(v, B.unpack8(B.pack8(w)))
    # two graphs, replayed on two streams at once, each with a workspace of its own
    packed = B.pack8(w)
    graphs, outs, ins = [], [], [x.clone(), (x * 2).clone()]
    for a in ins:
        B.matmul8(a, packed)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(B.matmul8(a, packed))
        graphs.append(g)
    ins[0].copy_(x * 4)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want * 4) and torch.equal(outs[1], want * 2)
