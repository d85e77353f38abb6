"""The 4-bit form and its products on the GPU, against the definition in
include/cam.h in numpy: the bytes and values exactly, the products against
64 bits.

Tolerance of a product. Its products are exact; what rounds is binary32 sums
of n = cols / 32 + 96 terms at most in a row (steps of a group's sum, groups,
and the sums of warps, blocks and x's terms), each by 2^-22 of the terms'
magnitudes at most (a tensor-core step truncates): n 2^-22 sum |s q x|. A bf16
result adds 2^-8 of itself.
"""
import numpy as np
import pytest
import torch

from checkpoint_averaging_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    yield
    torch.cuda.synchronize()


def form(w, group):
    """(q int, s fp32) of the definition, [rows, groups, group] and [rows, groups]."""
    w = np.asarray(w, np.float32)
    n = -(-w.shape[1] // group)
    full = np.zeros((w.shape[0], n * group), np.float32)
    full[:, :w.shape[1]] = w
    full = full.reshape(w.shape[0], n, group)
    with np.errstate(all="ignore"):
        big = np.abs(full).max(-1)
        s = ((big / np.float32(7)).astype(np.float32).view(np.uint32) & 0xFFFF0000).view(np.float32)
        s = np.where(s >= np.float32(2.0 ** -126), s, np.float32(0))
        inv = np.where(s > 0, np.float32(1) / s, np.float32(0)).astype(np.float32)
        q = np.clip(np.rint(full * inv[..., None]), -7, 7)
    fine = np.isfinite(big)
    q = np.where(fine[..., None], q, 0).astype(np.int64)
    return q, np.where(fine, s, np.float32(np.nan)).astype(np.float32)


def values(q, s, cols):
    return (q.astype(np.float32) * s[..., None]).reshape(q.shape[0], -1)[:, :cols]


def decode(data, rows, cols, group):
    """(q, s) from the documented bytes, element by element of a tile."""
    tr, tc = -(-rows // 16), -(-cols // 128)
    per = 128 // group
    tiles = data.reshape(tr, tc, 1024 + 32 * per)
    words = np.ascontiguousarray(tiles[..., :1024]).view("<u4").reshape(tr, tc, 2, 32, 4)
    scale = np.ascontiguousarray(tiles[..., 1024:]).view("<u2").reshape(tr, tc, 8, 2, per)
    q = np.zeros((tr * 16, tc * 128), np.int64)
    s = np.zeros((tr * 16, tc * per), np.uint32)
    place = [0, 4, 1, 5, 2, 6, 3, 7]  # the nibble of each of eight columns
    for h in range(2):
        for lane in range(32):
            for i in range(4):
                for c in range(8):
                    nib = (words[:, :, h, lane, i] >> np.uint32(4 * place[c])) & np.uint32(15)
                    q[8 * h + lane // 4::16, 32 * i + 8 * (lane % 4) + c::128] = nib.astype(np.int64) - 8
        for r in range(8):
            for j in range(per):
                s[8 * h + r::16, j::per] = scale[:, :, r, h, j]
    return q, (s << 16).view(np.float32)


def matrix(rows, cols, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, cols, generator=g) * 0.02).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (16, 128), (17, 129), (5, 1000), (64, 512), (33, 77)])
def test_form_and_values_are_the_definition(rows, cols, group, dtype):
    w = matrix(rows, cols, rows + cols, dtype)
    q, s = form(w.float().numpy(), group)
    pk = B.pack4(w.to(DEV), group)
    assert pk.shape == (rows, cols) and pk.data.numel() == B.pack4_bytes(rows, cols, group)
    dq, ds = decode(pk.data.cpu().numpy(), rows, cols, group)
    n = q.shape[1]
    np.testing.assert_array_equal(dq[:rows, :n * group].reshape(q.shape), q)
    np.testing.assert_array_equal(ds[:rows, :n], s)
    assert not dq[rows:].any() and not dq[:, cols:].any()  # past the end: q = 0
    v = values(q, s, cols)
    np.testing.assert_array_equal(B.unpack4(pk).cpu().numpy(), v)
    np.testing.assert_array_equal(B.unpack4(pk, torch.bfloat16).cpu().float().numpy(),
                                  torch.from_numpy(v).to(torch.bfloat16).float().numpy())
    # half a step of the group, and the rounding of w * (1 / s)
    step = np.repeat(s, group, 1)[:, :cols]
    assert (np.abs(v - w.float().numpy()) <= step * 0.5001).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_and_unaligned_matrices(dtype):
    rows, cols = 19, 200
    flat = matrix(1, rows * 333 + 7, 5, dtype).to(DEV)[0]
    for at, ld in ((0, 333), (1, 204), (4, 200), (3, 333)):
        w = flat[at:at + rows * ld].as_strided((rows, cols), (ld, 1))
        q, s = form(w.float().cpu().numpy(), 64)
        pk = B.pack4(w, 64)
        out = torch.full((rows * ld + at,), 9.0, dtype=dtype, device=DEV)
        view = out[at:].as_strided((rows, cols), (ld, 1))
        assert B.unpack4(pk, out=view) is view
        want = torch.from_numpy(values(q, s, cols)).to(dtype)
        assert torch.equal(view.cpu(), want)
        assert int((out == 9.0).sum()) == out.numel() - rows * cols  # nothing else written


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("cols,ld", [(519, 519), (520, 523), (392, 400), (647, 649)])
def test_every_alignment_of_a_row(cols, ld, group, dtype):
    rows = 37
    flat = matrix(1, rows * ld + 9, cols, dtype).to(DEV)[0]
    for at in range(9):
        w = flat[at:at + rows * ld].as_strided((rows, cols), (ld, 1))
        q, s = form(w.float().cpu().numpy(), group)
        pk = B.pack4(w, group)
        assert torch.equal(pk.data, B.pack4(w.float(), group).data)
        out = torch.full((rows * ld + at,), 9.0, dtype=dtype, device=DEV)
        view = out[at:].as_strided((rows, cols), (ld, 1))
        B.unpack4(pk, out=view)
        assert torch.equal(view.cpu(), torch.from_numpy(values(q, s, cols)).to(dtype))
        assert int((out == 9.0).sum()) == out.numel() - rows * cols  # nothing else written


def test_zero_tiny_huge_and_broken_groups():
    w = torch.zeros(8, 128)
    w[1, 5] = 1e-45          # the scale underflows: the group stands for 0
    w[2, :32] = 3.4028234e38
    w[3, 40] = float("nan")
    w[4, 70] = float("inf")
    w[5, 100] = -float("inf")
    w[6] = -0.0
    w[7, :3] = torch.tensor([7.0, 0.5, 1.5])  # s = 1: ties to even
    q, s = form(w.numpy(), 32)
    pk = B.pack4(w.to(DEV), 32)
    v = B.unpack4(pk).cpu().numpy()
    np.testing.assert_array_equal(v, values(q, s, 128))
    assert (v[:2] == 0).all() and np.isfinite(v[2]).all() and v[7, 1] == 0 and v[7, 2] == 2
    for r, j in ((3, 1), (4, 2), (5, 3)):
        assert np.isnan(v[r, 32 * j:32 * j + 32]).all()
        assert (np.delete(v[r], np.s_[32 * j:32 * j + 32]) == 0).all()


@pytest.mark.parametrize("exponent", [-126, -120, -60, 0, 60, 121])
def test_every_scale_is_divided_by_exactly(exponent):
    # one group for each of the 128 significands a scale can have, at its smallest and its
    # largest |w|, the other weights anywhere below
    m = np.arange(128)
    s = ((1 + m / 128) * 2.0 ** exponent).astype(np.float32)
    g = np.random.default_rng(1)
    w = (g.uniform(-7, 7, (256, 64)) * np.concatenate([s, s])[:, None]).astype(np.float32)
    w[:128, 0] = s * np.float32(7)
    w[128:, 0] = -(s.astype(np.float64) * 7 * (1 + 1 / 128 / (1 + m / 128) - 1e-6)).astype(np.float32)
    w[:, 1] = np.float32(0.5) * np.concatenate([s, s])  # ties, and next to them
    w[:, 2] = np.float32(-2.5) * np.concatenate([s, s])
    w[:, 3] = np.nextafter(np.float32(1.5) * np.concatenate([s, s]), np.float32(0))
    q, want = form(w, 64)
    pk = B.pack4(torch.from_numpy(w).to(DEV), 64)
    dq, ds = decode(pk.data.cpu().numpy(), 256, 64, 64)
    np.testing.assert_array_equal(ds[:256, :1], want)
    np.testing.assert_array_equal(dq[:256, :64], q[:, 0])
    assert len(np.unique(want)) >= 128


def check_product(x, pk, w, group, y):
    q, s = form(w, group)
    v = values(q, s, w.shape[1]).astype(np.float64)
    xs = x.float().cpu().numpy().astype(np.float64).reshape(-1, w.shape[1])
    want = xs @ v.T
    mag = np.abs(xs) @ np.abs(v).T
    got = y.float().cpu().numpy().astype(np.float64).reshape(want.shape)
    tol = (w.shape[1] / 32 + 96) * 2.0 ** -22 * mag
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    assert (np.abs(got - want) <= tol).all(), np.abs(got - want).max()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("tokens,rows,cols", [
    (1, 1, 1), (1, 16, 128), (2, 17, 129), (3, 40, 1000), (1, 512, 1408), (5, 33, 31),
    (8, 100, 640), (9, 200, 384), (17, 48, 513), (32, 70, 300), (33, 64, 256), (70, 31, 130),
    (1, 64, 16384), (11, 24, 9000), (32, 20, 16384), (3, 10000, 96), (6, 11000, 260)])
def test_products(tokens, rows, cols, group, dtype):
    w = matrix(rows, cols, rows * 7 + cols)
    x = torch.randn(tokens, cols, generator=torch.Generator().manual_seed(tokens)).to(dtype).to(DEV)
    pk = B.pack4(w.to(DEV), group)
    y = B.gemv4(x, pk)
    assert y.shape == (tokens, rows) and y.dtype == dtype
    check_product(x, pk, w.numpy(), group, y)
    other = torch.float32 if dtype == torch.bfloat16 else torch.bfloat16
    check_product(x, pk, w.numpy(), group, B.gemv4(x, pk, out_dtype=other))
    assert torch.equal(B.gemv4(x, pk), y)  # the same bits again


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("tokens,rows,cols", [
    (1, 14700, 64), (1, 19400, 256), (2, 19456, 1), (5, 19456, 513), (6, 40000, 129),
    (11, 18999, 130), (16, 19000, 1024), (17, 38000, 640), (32, 19333, 384), (40, 19456, 128)])
def test_products_of_many_rows(tokens, rows, cols, group, dtype):
    # rows enough to fill the GPU with units of 128 of them
    test_products(tokens, rows, cols, group, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,rows,cols", [
    (3, 5000, 9001), (8, 2433, 16000), (12, 2600, 9000), (17, 4000, 3700), (32, 2500, 5000),
    (40, 1300, 8200)])
def test_products_of_long_rows_that_are_many(tokens, rows, cols, dtype):
    # x in slabs, taken by one block or by two side by side
    test_products(tokens, rows, cols, 64, dtype)


@pytest.mark.parametrize("tokens,cols", [(1, 131072), (2, 131072), (32, 131072)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_longest_rows(tokens, cols, dtype):
    w = matrix(18, cols, 3)
    x = torch.randn(tokens, cols, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    pk = B.pack4(w.to(DEV), 64)
    check_product(x, pk, w.numpy(), 64, B.gemv4(x, pk))


def test_product_shapes_strides_and_empty_sizes():
    w = matrix(50, 200, 1)
    pk = B.pack4(w.to(DEV), 32)
    big = torch.randn(4, 333, generator=torch.Generator().manual_seed(2)).to(DEV)
    for at in (0, 1, 3):
        x = big[:, at:at + 200]
        check_product(x, pk, w.numpy(), 32, B.gemv4(x, pk))
    y = B.gemv4(big[0, :200], pk)
    assert y.shape == (50,)
    check_product(big[0, :200], pk, w.numpy(), 32, y)
    out = torch.full((4, 64), 5.0, device=DEV, dtype=torch.bfloat16)
    B.gemv4(big[:, :200], pk, out=out[:, 7:57])
    check_product(big[:, :200], pk, w.numpy(), 32, out[:, 7:57])
    assert (out[:, :7] == 5).all() and (out[:, 57:] == 5).all()
    assert B.gemv4(big[:0, :200], pk).shape == (0, 50)
    none = B.pack4(torch.empty(0, 200, device=DEV), 32)
    assert B.gemv4(big[:, :200], none).shape == (4, 0)
    flat = B.pack4(torch.empty(9, 0, device=DEV), 32)
    assert (B.gemv4(torch.empty(3, 0, device=DEV), flat) == 0).all()


def test_products_with_infinities_nan_and_wide_x():
    w = matrix(20, 128, 4)
    w[3, 7] = float("nan")
    pk = B.pack4(w.to(DEV), 32)
    x = torch.randn(6, 128, generator=torch.Generator().manual_seed(3))
    x[1, 5] = float("inf")
    x[2, 9] = float("nan")
    x[3] *= 1e30
    x[4] *= 1e-30
    y = B.gemv4(x.to(DEV), pk).cpu()
    v = B.unpack4(pk).cpu().double()
    want = x.double() @ v.T
    mag = x.double().abs() @ v.abs().T
    fine = torch.isfinite(want)
    assert torch.isnan(y[:, 3]).all() and torch.isnan(y[2]).all()
    assert torch.equal(torch.isfinite(y), fine)
    assert ((y.double() - want).abs()[fine] <= (100 * 2.0 ** -22 * mag)[fine]).all()


def test_published_bytes_make_the_same_matrix():
    w = matrix(40, 300, 8)
    pk = B.pack4(w.to(DEV), 64)
    again = B.Packed4(pk.data.cpu().to(DEV), 40, 300, 64)
    assert torch.equal(B.unpack4(again), B.unpack4(pk))
    with pytest.raises(ValueError, match="bytes"):
        B.Packed4(pk.data[:-16].clone(), 40, 300, 64)
    with pytest.raises(ValueError):
        B.Packed4(pk.data.cpu(), 40, 300, 64)


def test_binding_refusals():
    w = matrix(8, 64, 1).to(DEV)
    pk = B.pack4(w, 32)
    with pytest.raises(ValueError, match="fp32 or bf16"):
        B.pack4(w.half(), 32)
    with pytest.raises(B.ArgError, match="group"):
        B.pack4(w, 100)
    with pytest.raises(ValueError, match="contiguous rows"):
        B.pack4(w.t(), 32)
    with pytest.raises(ValueError, match="columns"):
        B.gemv4(torch.zeros(1, 63, device=DEV), pk)
    with pytest.raises(ValueError, match="overlapping"):
        B.gemv4(torch.zeros(64, device=DEV).expand(3, 64), pk)
    with pytest.raises(ValueError, match="out"):
        B.gemv4(torch.zeros(1, 64, device=DEV), pk, out=torch.zeros(1, 9, device=DEV))


def test_another_stream_and_graph_capture():
    w = matrix(300, 256, 2).to(DEV)
    x = torch.randn(2, 256, generator=torch.Generator().manual_seed(9)).to(DEV)
    want_pk = B.pack4(w, 64)
    want = B.gemv4(x, want_pk)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = B.gemv4(x, B.pack4(w, 64, stream=s), stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.gemv4(x, want_pk, out=out)
    for _ in range(2):
        x.mul_(0.5)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, B.gemv4(x, want_pk))


def test_offsets_past_32_bits():
    rows, ld = 9, 300_000_000
    flat = torch.empty(rows * ld, dtype=torch.bfloat16, device=DEV)  # 5.4 GB, sparsely used
    w = flat.as_strided((rows, 100), (ld, 1))
    w.copy_(matrix(rows, 100, 6))
    pk = B.pack4(w, 32)
    q, s = form(w.float().cpu().numpy(), 32)
    np.testing.assert_array_equal(B.unpack4(pk).cpu().numpy(), values(q, s, 100))
    B.unpack4(pk, out=w)
    np.testing.assert_array_equal(w.float().cpu().numpy(),
                                  torch.from_numpy(values(q, s, 100)).bfloat16().float().numpy())
