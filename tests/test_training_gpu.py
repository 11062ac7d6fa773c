"""linear_ste and swiglu on the GPU: outputs and gradients against 64-bit formulas on the rounded operands and
against differences.

Tolerances: products as in test_matmul_gpu.py. swiglu computes in fp32 with an exponential and a division of at most
two units in the last place (2^-22 each); a dozen such steps stay below 2^-18 relative for bf16 and, the steps other
than these rounding by 2^-24, below 2^-20 for fp32. The factor 1 + g (1 - s) is a sum of terms of up to 1 + |g|, so its error counts against
that sum of magnitudes. Outputs then round by half a step of their type."""
import pytest
import torch

from block_scaled_microscaling_b200 import mxq, ops

from test_matmul_gpu import close, decoded, half_step, values

pytestmark = pytest.mark.gpu


def columns(x, fmt="mxfp8"):
    """x rounded with blocks of 32 rows, in 64 bits."""
    rows = x.shape[0]
    xt = torch.nn.functional.pad(x, (0, 0, 0, -rows % 32)).T.contiguous()
    return mxq.fake_quantize(xt, fmt).double().T[:rows]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("m,n,k", [(1, 32, 32), (31, 64, 96), (32, 160, 64), (77, 96, 544), (333, 1024, 288), (260, 32, 1024)])
def test_linear_ste(m, n, k, fmt, dtype):
    x, w, g = values(m, m, k, dtype), values(n, n, k, dtype), values(k, m, n, dtype)
    x.requires_grad_(), w.requires_grad_()
    y = ops.linear_ste(x, w, fmt)
    dx, dw = torch.autograd.grad(y, (x, w), g)
    mxq.check_device()
    assert (y.dtype, dx.dtype, dw.dtype) == (dtype,) * 3
    x, w = x.detach(), w.detach()
    a, b = decoded(x, fmt), decoded(w, fmt)
    close(y.detach(), a @ b.T, a.abs() @ b.abs().T, k)
    a, b = decoded(g, "mxfp8"), columns(w)
    close(dx, a @ b, a.abs() @ b.abs(), n)
    a, b = columns(g), columns(x)
    close(dw, a.T @ b, a.abs().T @ b.abs(), m)


def test_linear_ste_against_differences():
    """Operands on the formats' grid under every scale that can arise: the layer is then linear and differences of
    sum(y * g) over steps that stay on the grid are its gradient exactly."""
    rng = torch.Generator(device="cuda").manual_seed(0)
    pick = lambda *s: (torch.randint(1, 4, s, generator=rng, device="cuda") * (2 * torch.randint(0, 2, s, generator=rng, device="cuda") - 1)).float()  # noqa: E731
    x, w, g = pick(40, 64), pick(32, 64), pick(40, 32)
    x.requires_grad_(), w.requires_grad_()
    loss = lambda a, b: (ops.linear_ste(a, b, "mxfp8").double() * g).sum()  # noqa: E731
    dx, dw = torch.autograd.grad((ops.linear_ste(x, w) * g).sum(), (x, w))
    for t, d, f in ((x, dx, lambda a: loss(a, w)), (w, dw, lambda b: loss(x, b))):
        for i, j in ((0, 0), (7, 33), (31, 63)):
            up, down = t.detach().clone(), t.detach().clone()
            up[i, j] += 0.5
            down[i, j] -= 0.5
            assert float((f(up) - f(down)).detach()) == float(d[i, j])


def test_linear_ste_leading_dimensions_strides_and_partial_gradients():
    x, w = values(1, 6 * 128, 64).view(6, 128, 64).transpose(0, 1), values(2, 32, 64)
    x.requires_grad_()
    y = ops.linear_ste(x, w)
    assert y.shape == (128, 6, 32)
    g = values(3, 1, 32).view(1, 1, 32).expand(128, 6, 32)  # a broadcast gradient
    dx, = torch.autograd.grad(y, x, g)
    assert dx.shape == x.shape
    a, b = decoded(g.reshape(-1, 32), "mxfp8"), columns(w)
    close(dx.reshape(-1, 64), a @ b, a.abs() @ b.abs(), 32)
    x = x.detach()
    w.requires_grad_()
    dw, = torch.autograd.grad(ops.linear_ste(x, w), w, g)
    a, b = columns(g.reshape(-1, 32)), columns(x.reshape(-1, 64))
    close(dw, a.T @ b, a.abs().T @ b.abs(), 768)
    with torch.no_grad():
        assert not ops.linear_ste(x, w).requires_grad


def test_linear_ste_without_tokens():
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    w = values(2, 32, 64).requires_grad_()
    y = ops.linear_ste(x, w)
    assert y.shape == (0, 32)
    dx, dw = torch.autograd.grad(y, (x, w), torch.zeros_like(y))
    assert dx.shape == (0, 64) and (dw == 0).all() and dw.shape == w.shape


def test_a_second_derivative_is_refused():
    x, w = values(1, 4, 64).requires_grad_(), values(2, 32, 64).requires_grad_()
    for y in (ops.linear_ste(x, w), ops.swiglu(x)):
        d, = torch.autograd.grad(y.sum(), x, create_graph=True)
        with pytest.raises(RuntimeError):
            d.sum().backward()


def test_linear_ste_keeps_33_64ths_of_the_input():
    x, w = values(1, 4096, 2560).requires_grad_(), values(2, 32, 2560).requires_grad_()
    kept = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: kept.append(t) or t, lambda t: t):
        ops.linear_ste(x, w)
    size = sum(t.numel() * t.element_size() for t in kept if t.data_ptr() != w.data_ptr())
    assert size == x.numel() * 33 // 32


def swiglu64(gate, up):
    return gate / (1 + torch.exp(-gate)) * up


def swiglu_grads64(gate, up, dy):
    s = 1 / (1 + torch.exp(-gate))
    return dy * up * s * (1 + gate * (1 - s)), dy * gate * s, (dy * up * s).abs() * (1 + gate.abs())


def near(got, want, size):
    rel = 2.0 ** -18 if got.dtype == torch.bfloat16 else 2.0 ** -20
    err = (got.double() - want).abs()
    tiny = torch.finfo(got.dtype).tiny  # results below the normal range may flush
    bad = err > half_step(got.dtype) * want.abs() + rel * size + tiny
    assert not bad.any(), (int(bad.sum()), float(err[bad].max()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (5, 2560), (129, 96), (1000, 9728)])
def test_swiglu(rows, cols, packed, dtype):
    both = values(rows, rows, 2 * cols, dtype)
    dy = values(cols, rows, cols, dtype)
    gate, up = both[:, :cols], both[:, cols:]
    if packed:
        both.requires_grad_()
        y = ops.swiglu(both)
        d, = torch.autograd.grad(y, both, dy)
        assert d.shape == both.shape
        dgate, dup = d[:, :cols], d[:, cols:]
    else:
        a, b = gate.clone().requires_grad_(), up.clone().requires_grad_()
        y = ops.swiglu(a, b)
        dgate, dup = torch.autograd.grad(y, (a, b), dy)
    assert y.shape == dy.shape and y.dtype == dtype
    gate, up, dy = gate.detach(), up.detach(), dy.double()
    want = swiglu64(gate.double(), up.double())
    near(y.detach(), want, want.abs())
    g8, u8 = decoded(gate, "mxfp8"), decoded(up, "mxfp8")
    wg, wu, size = swiglu_grads64(g8, u8, dy)
    near(dgate, wg, size)
    near(dup, wu, wu.abs())


def test_swiglu_gradients_against_differences():
    """Central differences (step 2^-13) of the 64-bit function at the rounded point: error below step^2 times the
    third derivative (under 1) times the other factors, plus the tolerance above."""
    both = torch.randn((4, 64), generator=torch.Generator(device="cuda").manual_seed(0), device="cuda").requires_grad_()
    dy = torch.randn((4, 32), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    d, = torch.autograd.grad(ops.swiglu(both), both, dy)
    g, u = decoded(both.detach()[:, :32], "mxfp8"), decoded(both.detach()[:, 32:], "mxfp8")
    h = 2.0 ** -13
    dg = (swiglu64(g + h, u) - swiglu64(g - h, u)) / (2 * h) * dy
    du = (swiglu64(g, u + h) - swiglu64(g, u - h)) / (2 * h) * dy
    bound = lambda f: (h * h + 2.0 ** -20 * (1 + g.abs())) * (dy.abs() * f)  # noqa: E731
    assert ((d[:, :32].double() - dg).abs() <= bound(u.abs())).all()
    assert ((d[:, 32:].double() - du).abs() <= bound(g.abs())).all()


def test_swiglu_strided_halves_extremes_and_no_grad():
    both = values(1, 6 * 10, 128).view(6, 10, 128)
    gate, up = both[..., :64], both[..., 64:]
    want = ops.swiglu(gate.contiguous(), up.contiguous())
    assert torch.equal(ops.swiglu(gate, up), want)            # one stride for both
    assert torch.equal(ops.swiglu(gate, up.contiguous()), want)
    assert torch.equal(ops.swiglu(both), want)
    odd = torch.zeros((60, 65), dtype=torch.bfloat16, device="cuda")  # a stride that is not 16-byte aligned
    odd[:, :64] = gate.reshape(60, 64)
    assert torch.equal(ops.swiglu(odd[:, :64], up.reshape(60, 64)), want.view(60, 64))
    x = torch.tensor([0.0, -0.0, 200.0, -200.0, 1e38, -1e38, 90.0, -90.0] * 8, device="cuda")[None]
    y = ops.swiglu(x.clone().requires_grad_())
    assert torch.isfinite(y[0, 2:4]).all() and (y[0, 3] == 0) and torch.isfinite(y[0, 5])
    bad = values(2, 3, 128).requires_grad_()
    with torch.no_grad():
        bad[1, 5] = float("nan")       # gate's first block of row 1
    d, = torch.autograd.grad(ops.swiglu(bad), bad, torch.ones((3, 64), dtype=bad.dtype, device="cuda"))
    nan = torch.zeros_like(d, dtype=torch.bool)
    nan[1, :32], nan[1, 64:96] = True, True
    assert torch.equal(torch.isnan(d), nan)
    assert ops.swiglu(torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")).shape == (0, 32)


def test_swiglu_entry_point_strides_and_overlaps():
    buf = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    p, st = buf.data_ptr(), torch.cuda.current_stream().cuda_stream
    f, b = ops.mxq_swiglu_forward, ops.mxq_swiglu_backward
    ck = (p + 8192, p + 9216, p + 10240, p + 11264)
    assert f(p, p + 64, 1, 4, 32, 64, p + 4096, *ck, st) == 0          # halves of one matrix
    assert f(p, p + 64, 1, 4, 32, 64, p + 4096, None, None, None, None, st) == 0
    assert f(p, p + 64, 1, 4, 32, 64, p + 4096, p + 8192, None, None, None, st) == 1
    assert f(p, p + 64, 1, 4, 32, 64, p + 256, *ck, st) == 1           # out over gate
    assert f(p, p + 64, 1, 4, 32, 64, p + 8192, *ck, st) == 1          # out over a checkpoint
    assert f(p + 2, p + 64, 1, 4, 32, 64, p + 4096, *ck, st) == 3
    assert b(p + 4096, 1, *ck, 4, 32, p, p + 64, 64, st) == 0          # interleaved halves
    assert b(p + 4096, 1, *ck, 4, 32, p, p + 32, 64, st) == 1          # rows overlap
    assert b(p + 4096, 1, *ck, 4, 32, p, p, 64, st) == 1
    assert b(p + 4096, 1, *ck, 4, 32, p + 4096, p + 64, 64, st) == 1   # over grad
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_mlp_step_as_it_is_used(fmt):
    """down(swiglu(up(x))) with its gradients, twice, and captured into a graph: the same bits every time."""
    x, w1, w2 = values(1, 150, 256), values(2, 2 * 320, 256), values(3, 256, 320)
    leaves = [t.requires_grad_() for t in (x, w1, w2)]
    g = values(4, 150, 256)

    def step():
        y = ops.linear_ste(ops.swiglu(ops.linear_ste(x, w1, fmt)), w2, fmt)
        return [y.detach(), *torch.autograd.grad(y, leaves, g)]

    first, again = step(), step()
    mxq.check_device()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    assert all(torch.isfinite(t).all() for t in first)
    # forward against the definition
    a, b = decoded(x.detach(), fmt), decoded(w1.detach(), fmt)
    h = ops.linear_ste(x.detach(), w1.detach(), fmt)
    close(h, a @ b.T, a.abs() @ b.abs().T, 256)
    s = ops.swiglu(h)
    a, b = decoded(s, fmt), decoded(w2.detach(), fmt)
    close(first[0], a @ b.T, a.abs() @ b.abs().T, 320)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for t in out:
        t.zero_()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, out))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("which", ["gate", "up", "both"])
@pytest.mark.parametrize("base", [(1, 64), (1, 1, 64), (4, 1, 64), (1, 8, 64)])
def test_swiglu_of_broadcast_inputs(base, which, dtype):
    """Rows that share memory (strides of 0 in the last row dimension, in an outer one and in both): what a copy gives, with
    its gradients, which sum over the broadcast rows."""
    shape = (8, 64) if len(base) == 2 else (4, 8, 64)
    rows = torch.Size(shape[:-1]).numel()
    small = lambda seed: values(seed, torch.Size(base[:-1]).numel(), 64, dtype).view(base)  # noqa: E731
    gate = small(1) if which != "up" else values(1, rows, 64, dtype).view(shape)
    up = small(2) if which != "gate" else values(2, rows, 64, dtype).view(shape)
    dy = values(3, rows, 64, dtype).view(shape)
    views = [t.expand(shape).requires_grad_() for t in (gate, up)]
    copies = [t.detach().contiguous().requires_grad_() for t in views]
    y, want = ops.swiglu(*views), ops.swiglu(*copies)
    assert torch.equal(y, want)
    for got, exp in zip(torch.autograd.grad(y, views, dy), torch.autograd.grad(want, copies, dy)):
        assert torch.equal(got, exp)
    leaves = [gate.detach().requires_grad_(), up.detach().requires_grad_()]
    sums = torch.autograd.grad(ops.swiglu(*(t.expand(shape) for t in leaves)), leaves, dy)
    for got, leaf, per_row in zip(sums, leaves, torch.autograd.grad(ops.swiglu(*copies), copies, dy)):
        assert torch.equal(got, per_row.sum_to_size(leaf.shape))


def test_swiglu_of_a_broadcast_packed_input():
    both = values(5, 4, 128).view(4, 1, 128)
    assert torch.equal(ops.swiglu(both.expand(4, 8, 128)), ops.swiglu(both.expand(4, 8, 128).contiguous()))


@pytest.mark.parametrize("layer", ["linear_ste", "swiglu"])
def test_a_refusal_in_the_backward_pass_is_an_exception(layer):
    """A checkpoint that comes back in host memory is refused by the C entry point."""
    x, w = values(1, 40, 64).requires_grad_(), values(2, 96, 64)
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, lambda t: t.cpu()):
        y = ops.linear_ste(x, w) if layer == "linear_ste" else ops.swiglu(x)
    with pytest.raises(RuntimeError, match="mxq_.*status 1"):
        torch.autograd.grad(y, x, torch.ones_like(y))
    torch.cuda.synchronize()
    y = ops.swiglu(x)                          # and the next call works
    assert torch.autograd.grad(y, x, torch.ones_like(y))[0].shape == x.shape


def off(t, by=1):
    """t's values, `by` values behind a 16-byte boundary, contiguous."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device="cuda")
    buf[by:] = t.reshape(-1)
    return buf[by:].view(t.shape)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("by", [1, 2, 3])
def test_tensors_that_begin_off_a_16_byte_boundary(by, dtype):
    x, w, both = values(1, 40, 64, dtype), values(2, 96, 64, dtype), values(3, 40, 128, dtype)
    gy, gs = values(4, 40, 96, dtype), values(5, 40, 64, dtype)

    def grads(f, ins, dy):
        ins = [t.detach().requires_grad_() for t in ins]
        y = f(*ins)
        return [y.detach(), *torch.autograd.grad(y, ins, dy)]

    for f, ins, dy in ((ops.linear_ste, (x, w), gy), (ops.swiglu, (both,), gs), (ops.swiglu, (x, gs), gy[:, :64].contiguous())):
        want = grads(f, ins, dy)
        for moved in ([off(t, by) for t in ins], [off(ins[0], by), *ins[1:]], [*ins[:-1], off(ins[-1], by)]):
            assert moved[0].is_contiguous()
            for g in (dy, off(dy, by)):
                assert all(torch.equal(a, b) for a, b in zip(grads(f, moved, g), want))


@pytest.mark.parametrize("odd", [1, 5])
def test_gradients_that_are_slices(odd):
    """The gradient that cat() hands back begins behind the values in front of the output."""
    x, w = values(1, 40, 64).requires_grad_(), values(2, 128, 64).requires_grad_()
    aux, dy = torch.zeros(odd, dtype=torch.bfloat16, device="cuda").requires_grad_(), values(3, 1, 64 * 40 + 32)[0]
    y = ops.swiglu(ops.linear_ste(x, w))
    n = y.numel()
    got = torch.autograd.grad(torch.cat([aux, y.flatten()]), (x, w), torch.cat([dy[:odd], dy[:n]]))
    want = torch.autograd.grad(ops.swiglu(ops.linear_ste(x, w)), (x, w), dy[:n].view(y.shape))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    z = ops.linear_ste(x, w)
    dz = values(4, 40, 128)
    got = torch.autograd.grad(torch.cat([aux, z.flatten()]), (x, w), torch.cat([aux.detach(), dz.flatten()]))
    want = torch.autograd.grad(ops.linear_ste(x, w), (x, w), dz)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("low", [-3.3e38, -1e30, -200.0, -100.0])
def test_swiglu_gradients_of_gates_far_below_zero(low, dtype):
    """silu and its derivative vanish there, however large the other factors are. In fp32 s = e^-|g| / (1 + e^-|g|) lies below
    the normal range: its exponential is off by at most two steps of 2^-149, its product and the factor 1 + g (1 - s) by half a
    step each, together below (1 + |g|) 2^-147 before dy and u are multiplied in."""
    gate = torch.full((3, 64), low, device="cuda", dtype=dtype)
    up = torch.tensor([1.0, -3e38, 1e20, 0.0], device="cuda", dtype=dtype).repeat(3, 16)
    dy = torch.tensor([4.0, -3e38, 1e20, 1e-3], device="cuda", dtype=dtype).repeat_interleave(48).view(3, 64)
    gate.requires_grad_(), up.requires_grad_()
    y = ops.swiglu(gate, up)
    dgate, dup = torch.autograd.grad(y, (gate, up), dy)
    for t in (y, dgate, dup):
        assert torch.isfinite(t).all()
    g8, u8 = decoded(gate.detach(), "mxfp8"), decoded(up.detach(), "mxfp8")
    s, dy = 1 / (1 + torch.exp(-g8)), dy.double()
    below = (1 + g8.abs()) * 2.0 ** -147
    for got, want, by in ((dgate, dy * (s * (1 + g8 * (1 - s))) * u8, dy * u8), (dup, dy * (g8 * s), dy)):
        room = by.abs() * below + half_step(dtype) * want.abs() + 2.0 ** -18 * want.abs() + torch.finfo(dtype).tiny
        assert ((got.double() - want).abs() <= room).all()
    if low < -200:
        assert (dgate == 0).all() and (dup == 0).all()
