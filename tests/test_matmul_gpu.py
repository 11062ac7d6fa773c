"""Block-scaled product, two-direction quantize and the serving linear layer on the GPU, against 64-bit products of
the values that the codes and scales stand for.

Tolerance of one output: the products of two elements are exact in fp32 (4- and 8-bit significands of at most 8
bits together) and so are the power-of-two scales; each of the k additions loses at most one unit in the last place
of 24 bits of the running sum, itself at most S = sum |a b|, so |error| <= k 2^-23 S, plus half a step of the
output's type (bf16 2^-8, fp32 2^-24 relative)."""
import pytest
import torch

from block_scaled_microscaling_b200 import mxq, ops

pytestmark = pytest.mark.gpu

FMTS = ["mxfp4", "mxfp8"]
# one token to several tiles; odd sizes; k of one block, of parts of a stage and of an MMA, of several stages; few
# tiles (k shared by a cluster), more tiles than SMs (a CTA walks several)
SHAPES = [(1, 32, 32), (1, 128, 64), (1, 4096, 4096), (3, 130, 96), (16, 257, 160), (17, 64, 224), (33, 100, 288), (64, 129, 512),
          (65, 640, 1056), (77, 1000, 2560), (128, 300, 512), (129, 31, 544), (200, 520, 1056), (257, 385, 96),
          (300, 1000, 2048), (1000, 2300, 320), (2100, 2600, 288), (130, 1, 32), (4700, 2400, 352),
          (5000, 4000, 2080), (4700, 2401, 352), (2300, 2552, 96), (2305, 2499, 64), (140, 77, 64), (200, 134, 96), (150, 6, 64)]


def values(seed, rows, cols, dtype=torch.bfloat16):
    """N(0, 1) blocks, each times 2^e with e uniform in -6 .. 6: a misplaced scale changes a result by a power of two."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    e = torch.randint(-6, 7, (rows, cols // 32), generator=g, device="cuda").repeat_interleave(32, 1)
    return torch.ldexp(x, e).to(dtype)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def close(got, want, total, k):
    assert got.shape == want.shape
    err = (got.double() - want).abs()
    bad = err > half_step(got.dtype) * want.abs() + k * 2.0 ** -23 * total
    assert not bad.any(), (int(bad.sum()), torch.nonzero(bad)[:4].tolist(), float((err / (want.abs() + 1e-30)).max()))


def decoded(x, fmt):
    return mxq.fake_quantize(x.contiguous(), fmt).double()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(m, n, k, fmt, dtype):
    a, b = values(m + k, m, k), values(n + 7 * k, n, k)
    ac, as_ = mxq.quantize_mma(a, fmt)
    bc, bs = mxq.quantize_mma(b, fmt)
    got = ops.matmul(ac, as_, bc, bs, fmt, dtype=dtype, check=True)
    assert got.dtype == dtype
    x, y = decoded(a, fmt), decoded(b, fmt)
    close(got, x @ y.T, x.abs() @ y.abs().T, k)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,n,k", [(5, 200, 416), (150, 300, 416), (2100, 2600, 256), (4700, 2400, 416)])
def test_product_of_small_integers_is_exact(m, n, k, fmt):
    """Codes of 0, 1, 2, 3, 4 and scales 1: every sum is an integer below 2^24, whatever the order."""
    g = torch.Generator(device="cuda").manual_seed(k)
    a = torch.randint(-4, 5, (m, k), generator=g, device="cuda").bfloat16()
    b = torch.randint(-4, 5, (n, k), generator=g, device="cuda").bfloat16()
    a[:, ::32], b[:, ::32] = 4, -4
    got = ops.matmul(*mxq.quantize_mma(a, fmt), *mxq.quantize_mma(b, fmt), fmt, dtype=torch.float32, check=True)
    assert torch.equal(got.double(), a.double() @ b.double().T)


@pytest.mark.parametrize("fmt", FMTS)
def test_product_extreme_scales_and_zero_blocks(fmt):
    a, b = values(1, 40, 256), values(2, 300, 256)
    a[3] = 0
    a[4] *= 2.0 ** 60
    b[7] *= 2.0 ** 50
    b[8] *= 2.0 ** -90
    a[5, 32:64] = 0
    x, y = decoded(a, fmt), decoded(b, fmt)
    got = ops.matmul(*mxq.quantize_mma(a, fmt), *mxq.quantize_mma(b, fmt), fmt, dtype=torch.float32, check=True)
    close(got, x @ y.T, x.abs() @ y.abs().T, 256)
    assert (got[3] == 0).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m", [3, 200, 10000])
def test_product_nan_blocks_stay_in_their_rows(m, fmt):
    a, b = values(1, m, 512), values(2, 300, 512)
    a[1, 100] = float("nan")
    b[130, 511] = float("inf")
    got = ops.matmul(*mxq.quantize_mma(a, fmt), *mxq.quantize_mma(b, fmt), fmt, check=True)
    nan = torch.zeros_like(got, dtype=torch.bool)
    nan[1], nan[:, 130] = True, True
    assert torch.equal(torch.isnan(got), nan)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (77, 300, 2560), (200, 300, 2048), (4700, 2400, 352)])
def test_product_repeats_bit_for_bit(m, n, k, fmt):
    a, b = mxq.quantize_mma(values(1, m, k), fmt), mxq.quantize_mma(values(2, n, k), fmt)
    first = ops.matmul(*a, *b, fmt)
    for _ in range(5):
        assert torch.equal(ops.matmul(*a, *b, fmt), first)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", [(150, 75, 96), (3, 75, 96), (130, 201, 2048), (4401, 2303, 64), (4401, 2304, 64), (4401, 2312, 64)])
def test_product_writes_only_its_output(m, n, k, dtype):
    a, b = mxq.quantize_mma(values(1, m, k), "mxfp8"), mxq.quantize_mma(values(2, n, k), "mxfp8")
    buf = torch.full((m * n + 64,), 7.0, dtype=dtype, device="cuda")
    out = buf[32:32 + m * n].view(m, n)
    ops.matmul(*a, *b, "mxfp8", out=out, check=True)
    assert (buf[:32] == 7).all() and (buf[-32:] == 7).all()
    assert torch.equal(out, ops.matmul(*a, *b, "mxfp8", dtype=dtype))


def test_product_empty_and_errors():
    a, s = torch.empty((0, 64), dtype=torch.uint8, device="cuda"), torch.empty(0, dtype=torch.uint8, device="cuda")
    b = mxq.quantize_mma(values(2, 40, 64), "mxfp8")
    assert ops.matmul(a, s, *b, "mxfp8").shape == (0, 40)
    assert ops.matmul(*b, a, s, "mxfp8").shape == (40, 0)
    buf = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    p, st = buf.data_ptr(), torch.cuda.current_stream().cuda_stream
    mm = ops.mxq_matmul
    assert mm(3, p, p + 4096, p + 8192, p + 12288, 4, 4, 32, p + 16384, 1, st) == 0
    assert mm(3, p + 8, p + 4096, p + 8192, p + 12288, 4, 4, 32, p + 16384, 1, st) == 3
    assert mm(3, p, p + 4097, p + 8192, p + 12288, 4, 4, 32, p + 16384, 1, st) == 3
    assert mm(3, p, p + 4096, p + 8192, p + 12288, 4, 4, 32, p + 16, 1, st) == 1           # out over an operand
    assert mm(3, p, p + 4096, p + 8192, p + 12288, 4, 4, 32, p + 12288 + 496, 1, st) == 1  # over the scales' padding
    host = torch.zeros(64, dtype=torch.uint8).data_ptr()
    assert mm(3, host, p + 4096, p + 8192, p + 12288, 4, 4, 32, p + 16384, 1, st) == 1
    torch.cuda.synchronize()


# ---- quantize_both --------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("row_fmt,col_fmt", [("mxfp4", "mxfp8"), ("mxfp8", "mxfp4"), ("mxfp8", None), (None, "mxfp8"), ("mxfp4", "mxfp4")])
@pytest.mark.parametrize("rows,cols", [(1, 32), (5, 64), (32, 96), (33, 160), (127, 128), (128, 256), (129, 416), (300, 4128)])
def test_quantize_both(rows, cols, row_fmt, col_fmt, dtype):
    x = values(rows + cols, rows, cols, dtype)
    x[rows // 2, 3] = float("nan")
    x[0, cols - 1] = float("-inf")
    rc, rs, cc, cs = ops.quantize_both(x, row_fmt, col_fmt)
    if row_fmt:
        want = mxq.quantize_mma(x, row_fmt)
        assert torch.equal(rc, want[0]) and torch.equal(rs, want[1])
    else:
        assert rc is None and rs is None
    if col_fmt:
        xt = torch.nn.functional.pad(x, (0, 0, 0, -rows % 32)).T.contiguous()
        want = mxq.quantize_mma(xt, col_fmt)
        assert cc.shape == want[0].shape and torch.equal(cc, want[0]) and torch.equal(cs, want[1])
    else:
        assert cc is None and cs is None


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_both_of_rows_alone_at_size(fmt, dtype):
    x = values(5, 1152, 1024, dtype)   # whole scale tiles, over a million values: another kernel
    x[700, 3] = float("nan")
    rc, rs, _, _ = ops.quantize_both(x, fmt)
    want = mxq.quantize_mma(x, fmt)
    assert torch.equal(rc, want[0]) and torch.equal(rs, want[1])


def test_quantize_both_errors():
    buf = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    p, st = buf.data_ptr(), torch.cuda.current_stream().cuda_stream
    qb = ops.mxq_quantize_both
    assert qb(3, 3, p, 1, 4, 32, p + 4096, p + 8192, p + 12288, p + 20480, st) == 0
    assert qb(3, 3, p, 1, 4, 32, p + 4096, p + 8192, p + 12288, p + 12288 + 512, st) == 1  # outputs overlap
    assert qb(3, 3, p, 1, 4, 32, p + 128, p + 8192, None, None, st) == 1                  # over src
    assert qb(3, 3, p, 1, 4, 32, p + 4096, None, None, None, st) == 1                     # half a direction
    assert qb(3, 3, p + 2, 1, 4, 32, p + 4096, p + 8192, None, None, st) == 3
    torch.cuda.synchronize()


# ---- linear (serving) -------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("shape,n", [((64,), 40), ((1, 1, 96), 33), ((3, 5, 256), 128), ((140, 320), 70)])
def test_linear(shape, n, fmt, dtype):
    k = shape[-1]
    x = values(sum(shape), max(1, torch.Size(shape[:-1]).numel()), k, dtype).view(shape)
    w = values(n, n, k)
    y = ops.linear(x, *mxq.quantize_mma(w, fmt), fmt, check=True)
    assert torch.equal(ops.linear(x, *mxq.quantize_mma(w, fmt), fmt), y)  # the plain call's way
    assert y.shape == (*shape[:-1], n) and y.dtype == dtype
    a, b = decoded(x.view(-1, k), fmt), decoded(w, fmt)
    close(y.view(-1, n), a @ b.T, a.abs() @ b.abs().T, k)


def test_linear_captured_and_on_another_stream():
    x, w = values(1, 20, 512), mxq.quantize_mma(values(2, 300, 512), "mxfp4")
    want = ops.linear(x, *w, "mxfp4")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.linear(x, *w, "mxfp4", stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ops.linear(x, *w, "mxfp4")
    x.copy_(values(9, 20, 512))
    graph.replay()
    assert torch.equal(out, ops.linear(x, *w, "mxfp4"))
    assert not torch.equal(out, want)
    mxq.check_device()
