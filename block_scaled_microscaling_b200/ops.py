"""Operators of language models on the microscaled formats (include/mxq_ops.h).

    from block_scaled_microscaling_b200 import quantize_mma, linear, linear_ste, swiglu
    w_codes, w_scales = quantize_mma(w, "mxfp4")             # once
    y = linear(x, w_codes, w_scales, "mxfp4")                 # x rounded to MXFP4, block-scaled product

    y = swiglu(linear_ste(x, w1))                             # training: 8-bit checkpoints, STE gradients

    cache = KVCache.empty(pages, kv_heads, page_size, head_dim)
    kv_append(k, v, cache, slots)                             # MXFP4, paged
    out = kv_attention(q, cache, block_table, seq_lens)

As in mxq.py, the mxq_* functions take raw integers and return the status; the helpers allocate outputs with
torch, refuse tensors that the C calls could not read or write safely, launch on the current stream (or `stream`)
and raise MXQError on a non-zero status. linear_ste and swiglu with their gradients, and plain calls of the others, go
through the C++ module _ops (csrc/ops_torch.cpp), which does the same in a few microseconds and leaves every other case
and the errors to the code here. Of these functions linear_ste and swiglu alone are differentiable: the results of the
others carry no gradient, also where an input requires one. The kernels of the product and of attention for many queries bound their waits:
check=True (of matmul and linear) synchronizes and raises if one ran out; else call check_device() before trusting
the outputs.
"""
import ctypes
import math
import os
import re

from . import mxq
from .mxq import MXQError, _as2d, _check, _dt, _finish, _fits, _fmt, _on_gpu, _torch

OPS_EXPORTS = ["mxq_matmul", "mxq_quantize_both", "mxq_linear_workspace_bytes", "mxq_linear", "mxq_swiglu_forward", "mxq_swiglu_backward", "mxq_kv_append",
               "mxq_kv_read", "mxq_kv_attention_workspace_bytes", "mxq_kv_attention"]
PRODUCT_FORMATS = ("mxfp4", "mxfp8")


class _Cache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("pages", ctypes.c_int64), ("kv_heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


_ready = None


def lib():
    """The loaded libmxq.so with the operators' signatures set."""
    global _ready
    if _ready is None:
        L = mxq.lib()
        i32, i64, vp, sz, f32 = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
        cache = ctypes.POINTER(_Cache)
        for name, args, res in [
            ("mxq_matmul", [i32, vp, vp, vp, vp, i64, i64, i64, vp, i32, vp], i32),
            ("mxq_quantize_both", [i32, i32, vp, i32, i64, i64, vp, vp, vp, vp, vp], i32),
            ("mxq_linear_workspace_bytes", [i32, i64, i64], sz),
            ("mxq_linear", [i32, vp, i32, i64, i64, vp, vp, i64, vp, vp, sz, vp], i32),
            ("mxq_swiglu_forward", [vp, vp, i32, i64, i64, i64, vp, vp, vp, vp, vp, vp], i32),
            ("mxq_swiglu_backward", [vp, i32, vp, vp, vp, vp, i64, i64, vp, vp, i64, vp], i32),
            ("mxq_kv_append", [cache, vp, i64, vp, i64, i32, i64, vp, vp], i32),
            ("mxq_kv_read", [cache, vp, i64, vp, vp, i32, vp], i32),
            ("mxq_kv_attention_workspace_bytes", [cache, i64, i64, i32, i32, i64], sz),
            ("mxq_kv_attention", [cache, vp, i64, i64, i64, i32, i64, vp, i32, vp, i64, vp, i64, f32, i32, i32, vp, vp, vp, sz,
                                  vp], i32),
        ]:
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _ready = L
    return _ready


_native_module = None


def _native():
    """The C++ module for plain calls."""
    global _native_module
    if _native_module is None:
        if not os.path.exists(os.path.join(mxq.HERE, "_ops.so")):
            raise RuntimeError("_ops.so is missing: build it with `python -m block_scaled_microscaling_b200.build`")
        _torch()
        from . import _ops
        _native_module = _ops
    return _native_module


def _plain(call, *args):
    """What the C++ module makes of a call: None where the case is not a plain one (other types among them), so that the
    code here says why. A refusal of a C entry point is raised with its status."""
    try:
        return call(*args)
    except TypeError:
        return None
    except RuntimeError as e:
        refused = re.match(r"(mxq_\w+): status (\d+)", str(e))
        if not refused:
            raise
        raise MXQError(int(refused[2]), refused[1]) from None


# ---- the C entry points, same names and arguments --------------------------------

def mxq_matmul(fmt, a_codes, a_scales, b_codes, b_scales, m, n, k, out, dtype, stream):
    return lib().mxq_matmul(fmt, a_codes, a_scales, b_codes, b_scales, m, n, k, out, dtype, stream)


def mxq_quantize_both(row_fmt, col_fmt, src, dtype, rows, cols, row_codes, row_scales, col_codes, col_scales, stream):
    return lib().mxq_quantize_both(row_fmt, col_fmt, src, dtype, rows, cols, row_codes, row_scales, col_codes, col_scales,
                                   stream)


def mxq_linear_workspace_bytes(fmt, m, k):
    return lib().mxq_linear_workspace_bytes(fmt, m, k)


def mxq_linear(fmt, x, dtype, m, k, b_codes, b_scales, n, out, workspace, workspace_bytes, stream):
    return lib().mxq_linear(fmt, x, dtype, m, k, b_codes, b_scales, n, out, workspace, workspace_bytes, stream)


def mxq_swiglu_forward(gate, up, dtype, rows, cols, ld, out, gate_codes, gate_scales, up_codes, up_scales, stream):
    return lib().mxq_swiglu_forward(gate, up, dtype, rows, cols, ld, out, gate_codes, gate_scales, up_codes, up_scales,
                                    stream)


def mxq_swiglu_backward(grad, dtype, gate_codes, gate_scales, up_codes, up_scales, rows, cols, dgate, dup, ld, stream):
    return lib().mxq_swiglu_backward(grad, dtype, gate_codes, gate_scales, up_codes, up_scales, rows, cols, dgate, dup, ld,
                                     stream)


def mxq_kv_append(cache, k, k_stride, v, v_stride, dtype, tokens, slots, stream):
    """cache: a (k_codes, k_scales, v_codes, v_scales, pages, kv_heads, page_size, head_dim) tuple of integers."""
    return lib().mxq_kv_append(ctypes.byref(_Cache(*cache)), k, k_stride, v, v_stride, dtype, tokens, slots, stream)


def mxq_kv_read(cache, slots, tokens, k, v, dtype, stream):
    return lib().mxq_kv_read(ctypes.byref(_Cache(*cache)), slots, tokens, k, v, dtype, stream)


def mxq_kv_attention_workspace_bytes(cache, batch, q_rows, max_q, q_heads, max_keys):
    return lib().mxq_kv_attention_workspace_bytes(ctypes.byref(_Cache(*cache)), batch, q_rows, max_q, q_heads, max_keys)


def mxq_kv_attention(cache, q, q_rows, q_row_stride, q_head_stride, q_heads, batch, q_starts, max_q, seq_lens, max_keys,
                     block_table, table_stride, scale, window, fill, out, lse, workspace, workspace_bytes, stream):
    return lib().mxq_kv_attention(ctypes.byref(_Cache(*cache)), q, q_rows, q_row_stride, q_head_stride, q_heads, batch,
                                  q_starts, max_q, seq_lens, max_keys, block_table, table_stride, scale, window, fill, out, lse,
                                  workspace, workspace_bytes, stream)


# ---- the product -------------------------------------------------------------------

def _product_fmt(fmt):
    f = _fmt(fmt)
    if fmt not in PRODUCT_FORMATS:
        raise MXQError(4, f"format {fmt!r}")
    return f


def _u8(t, what):
    if t.dtype != _torch().uint8:
        raise TypeError(f"{what} must be uint8, got {t.dtype}")


def _on(stream, call):
    """call() with `stream` current, so that what it allocates belongs to the stream that uses it."""
    if stream is None:
        return call()
    with _torch().cuda.stream(stream):
        return call()


def _raw_stream(t):
    """Handle of the stream current on t's device (torch.cuda.current_stream() takes as long as a launch)."""
    return _torch()._C._cuda_getCurrentRawStream(t.device.index)


def _bytes(n, like):
    torch = _torch()
    return torch.empty(n, dtype=torch.uint8, device=like.device)


def matmul(a_codes, a_scales, b_codes, b_scales, fmt, out=None, dtype=None, stream=None, check=False):
    """out[m, n] = a b^T of the microscaled operands a [m, k], b [n, k]: codes [rows, k/32*P] and scales in the tile
    layout, as quantize_mma or quantize_both return them; `dtype` bf16 (default) or fp32."""
    torch = _torch()
    f = _product_fmt(fmt)
    for t, what in ((a_codes, "a_codes"), (b_codes, "b_codes")):
        _on_gpu(t, what)
        _u8(t, what)
        if t.dim() != 2 or t.shape[1] % (4 * mxq.ELEM_BITS[fmt]):
            raise ValueError(f"{what} must be [rows, k/32 * {4 * mxq.ELEM_BITS[fmt]}], got {tuple(t.shape)}")
    (m, pa), (n, pb) = a_codes.shape, b_codes.shape
    if pa != pb:
        raise ValueError(f"operands differ in k: {pa} and {pb} bytes a row")
    k = pa // (4 * mxq.ELEM_BITS[fmt]) * 32
    if k == 0:
        raise MXQError(2, "k == 0")
    for t, rows, what in ((a_scales, m, "a_scales"), (b_scales, n, "b_scales")):
        _on_gpu(t, what)
        _u8(t, what)
        _fits(t, mxq.mxq_mma_scales_bytes(rows, k), what)
    _fits(a_codes, 0, "a_codes")
    _fits(b_codes, 0, "b_codes")

    def call():
        o = out
        if o is None:
            o = torch.empty((m, n), dtype=dtype or torch.bfloat16, device=a_codes.device)
        elif dtype is not None and o.dtype != dtype:
            raise TypeError(f"out is {o.dtype}, dtype {dtype}")
        _on_gpu(o, "out")
        if o.numel() != m * n:
            raise ValueError(f"out must hold {m} x {n} values")
        _fits(o, 0, "out")
        _check(mxq_matmul(f, a_codes.data_ptr(), a_scales.data_ptr(), b_codes.data_ptr(), b_scales.data_ptr(), m, n, k,
                          o.data_ptr(), _dt(o), _raw_stream(o)), "mxq_matmul")
        return o

    o = _on(stream, call)
    _finish(check)
    return o


def quantize_both(x, row_fmt=None, col_fmt=None, stream=None):
    """x [rows, cols] as an operand along its rows and / or its columns, read once:
    (row_codes [rows, cols/32*P], row_scales, col_codes [cols, rows32/32*P], col_scales), scales in the tile layout,
    the columns filled up with zeros to rows32 = the next multiple of 32 rows. A format of None leaves that direction
    out (None, None)."""
    torch = _torch()
    if row_fmt is None and col_fmt is None:
        raise ValueError("row_fmt or col_fmt is needed")
    fr = 0 if row_fmt is None else _product_fmt(row_fmt)
    fc = 0 if col_fmt is None else _product_fmt(col_fmt)
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D tensor")
    _on_gpu(x, "x")
    dt = _dt(x)
    rows, cols = x.shape
    rows32 = (rows + 31) // 32 * 32
    if cols == 0 or cols % 32:
        raise MXQError(2, f"cols={cols}")

    def call():
        e = lambda *s: torch.empty(s, dtype=torch.uint8, device=x.device)  # noqa: E731
        rc = rs = cc = cs = None
        if row_fmt is not None:
            rc, rs = mxq.empty_codes(row_fmt, rows, cols, x.device), e(mxq.mxq_mma_scales_bytes(rows, cols))
        if col_fmt is not None:
            cc, cs = mxq.empty_codes(col_fmt, cols, rows32, x.device), e(mxq.mxq_mma_scales_bytes(cols, rows32) if rows else 0)
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        _check(mxq_quantize_both(fr, fc, x.data_ptr(), dt, rows, cols, p(rc), p(rs), p(cc), p(cs),
                                 _raw_stream(x)), "mxq_quantize_both")
        return rc, rs, cc, cs

    return _on(stream, call)


def linear(x, w_codes, w_scales, fmt, out=None, stream=None, check=False):
    """x [..., k] (bf16/fp32, contiguous) rounded to `fmt`, times the weight w [n, k] held in `fmt` (codes
    [n, k/32*P] and tile-layout scales, as quantize_mma(w, fmt) returns them): [..., n] of x's dtype. For serving: the
    result carries no gradient (linear_ste is the layer to train)."""
    if out is None and stream is None and not check:
        y = _plain(_native().linear, x, w_codes, w_scales, mxq.FORMATS.get(fmt, -1))
        if y is not None:
            return y
    if not x.is_contiguous() or x.dim() == 0:
        raise ValueError("x must be contiguous, of at least one dimension")
    _on_gpu(x, "x")
    f = _product_fmt(fmt)
    rows, k = _as2d(x)
    if w_codes.dim() != 2 or w_codes.shape[1] * 32 != k * 4 * mxq.ELEM_BITS[fmt]:
        raise ValueError(f"w_codes {tuple(w_codes.shape)} do not belong to rows of {k} values in {fmt}")
    n = w_codes.shape[0]
    for t, need, what in ((w_codes, 0, "w_codes"), (w_scales, mxq.mxq_mma_scales_bytes(n, k), "w_scales")):
        _on_gpu(t, what)
        _u8(t, what)
        _fits(t, need, what)

    def call():
        o = out
        if o is None:
            o = _torch().empty((*x.shape[:-1], n), dtype=x.dtype, device=x.device)
        else:
            _on_gpu(o, "out")
            if o.dtype != x.dtype or o.numel() != rows * n:
                raise ValueError(f"out must hold {rows} x {n} values of {x.dtype}")
            _fits(o, 0, "out")
        need = mxq_linear_workspace_bytes(f, rows, k)
        ws = _bytes(need, x)
        _check(mxq_linear(f, x.data_ptr(), _dt(x), rows, k, w_codes.data_ptr(), w_scales.data_ptr(), n, o.data_ptr(),
                          ws.data_ptr(), need, _raw_stream(x)), "mxq_linear")
        return o

    o = _on(stream, call)
    _finish(check)
    return o


# ---- training: straight-through gradients from 8-bit checkpoints ----------------------

def linear_ste(x, weight, fmt="mxfp8"):
    """Differentiable linear layer in microscaled products: x [..., k], weight [n, k], k and n multiples of 32.
      forward   y = Q(x) Q(weight)^T, Q rounding to `fmt` along k
      backward  dx = Q8(dy) Q8(weight), blocks along n;  dweight = Q8(dy)^T Q8(x), blocks along the tokens
    with Q8 rounding to MXFP8 (gradients pass straight through the rounding of the operands). Of x only its MXFP8
    codes along the tokens are kept for the backward pass: the operand of the weight's gradient as it stands, 33/64 of
    x's bf16 bytes. Any number of tokens."""
    y = _plain(_native().linear_ste, x, weight, mxq.FORMATS.get(fmt, -1))
    if y is not None:
        return y
    _product_fmt(fmt)
    _on_gpu(x, "x")
    _on_gpu(weight, "weight")
    _dt(x), _dt(weight)
    if weight.dim() != 2 or x.dim() == 0 or x.shape[-1] != weight.shape[1]:
        raise ValueError(f"x {tuple(x.shape)} and weight {tuple(weight.shape)} do not fit")
    if weight.shape[1] == 0 or weight.shape[1] % 32 or weight.shape[0] == 0 or weight.shape[0] % 32:
        raise MXQError(2, f"weight {tuple(weight.shape)}: both sizes must be multiples of 32")
    raise MXQError(1, f"linear_ste of tensors on {x.device} and {weight.device}")


def swiglu(gate, up=None):
    """silu(gate) * up, differentiable; gate and up are kept for the backward pass as MXFP8 (33/64 of their bf16
    bytes) and the gradients are those of the rounded values. With up=None, `gate` is [..., 2 cols]: gate, then up
    (the output of one projection), and so is its gradient. cols % 32 == 0; bf16 or fp32."""
    y = _plain(_native().swiglu, gate, up)
    if y is not None:
        return y
    _on_gpu(gate, "gate")
    _dt(gate)
    if gate.dim() == 0:
        raise ValueError("need at least one dimension")
    cols = gate.shape[-1]
    if up is None:
        if cols % 2:
            raise MXQError(2, f"{cols} values a row are not gate and up")
        cols //= 2
    else:
        _on_gpu(up, "up")
        if up.shape != gate.shape or up.dtype != gate.dtype or up.device != gate.device:
            raise ValueError("gate and up must have one shape, dtype and device")
    if cols == 0 or cols % 32:
        raise MXQError(2, f"cols={cols}")
    raise MXQError(1, f"swiglu of tensors on {gate.device}")


# ---- the paged MXFP4 key/value cache ---------------------------------------------------

class KVCache:
    """Keys and values in MXFP4: codes uint8 [pages, kv_heads, page_size, head_dim/2], scales uint8 [pages, kv_heads,
    page_size, head_dim/32], both contiguous. Token slot s is row s % page_size of page s // page_size."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales):
        self._native = _plain(_native().cache, k_codes, k_scales, v_codes, v_scales)
        shape = k_codes.shape
        if self._native is not None:
            self.pages, self.kv_heads, self.page_size, half = shape
            self.head_dim = 2 * half
            self._tensors = (k_codes, k_scales, v_codes, v_scales)
            return
        if len(shape) != 4:
            raise ValueError("codes must be [pages, kv_heads, page_size, head_dim / 2]")
        if min(shape[1:3]) < 1 or shape[3] < 16:
            raise ValueError(f"a cache needs heads, rows in a page and blocks of 32 dimensions, got codes {tuple(shape)}")
        self.pages, self.kv_heads, self.page_size, self.head_dim = *shape[:3], shape[3] * 2
        want = {"codes": tuple(shape), "scales": (*shape[:3], shape[3] // 16)}
        for t, what in ((k_codes, "k_codes"), (k_scales, "k_scales"), (v_codes, "v_codes"), (v_scales, "v_scales")):
            _on_gpu(t, what)
            _u8(t, what)
            if tuple(t.shape) != want[what[2:]]:
                raise ValueError(f"{what} must be {want[what[2:]]}, got {tuple(t.shape)}")
            _fits(t, 0, what)
        self._tensors = (k_codes, k_scales, v_codes, v_scales)

    k_codes, k_scales, v_codes, v_scales = (property(lambda self, i=i: self._tensors[i]) for i in range(4))

    @classmethod
    def empty(cls, pages, kv_heads, page_size, head_dim, device="cuda"):
        """A cache of zeros."""
        torch = _torch()
        z = lambda n: torch.zeros((pages, kv_heads, page_size, n), dtype=torch.uint8, device=device)  # noqa: E731
        return cls(z(head_dim // 2), z(head_dim // 32), z(head_dim // 2), z(head_dim // 32))

    @property
    def device(self):
        return self.k_codes.device

    def _raw(self):
        return (self.k_codes.data_ptr(), self.k_scales.data_ptr(), self.v_codes.data_ptr(), self.v_scales.data_ptr(),
                self.pages, self.kv_heads, self.page_size, self.head_dim)


def _ints(t, dtype, what, numel=None):
    _on_gpu(t, what)
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    _fits(t, 0, what)
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{what} must hold {numel} values, got {t.numel()}")


def _tokens(t, cache, what):
    """Token stride of keys or values [tokens, kv_heads, head_dim] (heads of a token contiguous)."""
    _on_gpu(t, what)
    if t.dim() != 3 or tuple(t.shape[1:]) != (cache.kv_heads, cache.head_dim):
        raise ValueError(f"{what} must be [tokens, {cache.kv_heads}, {cache.head_dim}], got {tuple(t.shape)}")
    if t.stride(2) != 1 or (cache.kv_heads > 1 and t.stride(1) != cache.head_dim):
        raise ValueError(f"the heads of a token of {what} must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else cache.kv_heads * cache.head_dim


def kv_append(k, v, cache, slots, stream=None):
    """Round keys and values [tokens, kv_heads, head_dim] (bf16/fp32; the token stride is free) to MXFP4 and write
    token t to slot slots[t] (int64). Slots outside the cache are skipped; the others must differ."""
    if stream is None and cache._native is not None and _plain(_native().kv_append, cache._native, k, v, slots):
        return
    ks, vs = _tokens(k, cache, "k"), _tokens(v, cache, "v")
    if k.shape[0] != v.shape[0] or k.dtype != v.dtype:
        raise ValueError("k and v must have one shape and dtype")
    _ints(slots, _torch().int64, "slots", k.shape[0])
    _check(mxq_kv_append(cache._raw(), k.data_ptr(), ks, v.data_ptr(), vs, _dt(k), k.shape[0], slots.data_ptr(),
                         _raw_stream(k) if stream is None else stream.cuda_stream), "mxq_kv_append")


def kv_read(cache, slots, dtype=None, stream=None):
    """(k, v) [tokens, kv_heads, head_dim] held at slots (int64), exact in bf16 (default) or fp32; zeros for a slot
    outside the cache."""
    if dtype is None and stream is None and cache._native is not None:
        kv = _plain(_native().kv_read, cache._native, slots)
        if kv is not None:
            return kv
    torch = _torch()
    _ints(slots, torch.int64, "slots")

    def call():
        k, v = (torch.empty((slots.numel(), cache.kv_heads, cache.head_dim), dtype=dtype or torch.bfloat16,
                            device=cache.device) for _ in range(2))
        _check(mxq_kv_read(cache._raw(), slots.data_ptr(), slots.numel(), k.data_ptr(), v.data_ptr(), _dt(k),
                           _raw_stream(slots)), "mxq_kv_read")
        return k, v

    return _on(stream, call)


def kv_attention(q, cache, block_table, seq_lens, q_starts=None, max_q=None, scale=None, window=0, max_keys=None, out=None,
                 lse=False, stream=None):
    """Causal attention of bf16 queries over the cache.

    q            [rows, heads, head_dim] (row and head strides free, multiples of 8); heads a multiple of kv_heads
    block_table  int32 [batch, pages]: page of keys page_size * i .. of a sequence
    seq_lens     int32 [batch]: keys of each sequence, the new tokens' among them
    q_starts     int32 [batch + 1]: sequence b's queries are rows q_starts[b] .. q_starts[b + 1] (starts do not
                 decrease), at most max_q of them; None: rows / batch queries each
    max_q        with q_starts: the most queries of a sequence, which the host knows and the call cannot see. It chooses the
                 kernel and the grid, so give it: the default, rows, computes a ragged batch of single tokens with the
                 kernel for many queries (right, but slow)
    scale        of the scores (default head_dim ** -0.5); window: keys a query sees at most (0: all)
    max_keys     an upper bound of seq_lens, if known, for a better split of the work (longer sequences are cut)
    Keys that a query does not see do not enter it, whatever they hold; where a chunk has one that only some of its queries
    see and that is far larger than the others, its rows are computed one by one (right, but slow).
    Returns out [rows, heads, head_dim]; with lse=True (out, log-sum-exp fp32 [rows, heads]). A query that sees no key
    gives 0 (and -inf), and so do rows of no sequence and queries beyond max_q, which a given `out` keeps. For serving: the
    results carry no gradient."""
    if out is None and not lse and stream is None and cache._native is not None:
        o = _plain(_native().kv_attention, cache._native, q, block_table, seq_lens, q_starts, max_q, scale, window, max_keys)
        if o is not None:
            return o
    torch = _torch()
    _on_gpu(q, "q")
    if q.dim() != 3 or q.shape[2] != cache.head_dim or q.dtype != torch.bfloat16:
        raise ValueError(f"q must be bfloat16 [rows, heads, {cache.head_dim}], got {q.dtype} {tuple(q.shape)}")
    rows, heads, d = q.shape
    if q.stride(2) != 1:
        raise ValueError("the values of a head of q must be contiguous")
    if heads == 0 or heads % cache.kv_heads:
        raise ValueError(f"{heads} heads are no multiple of the cache's {cache.kv_heads}")
    batch = seq_lens.numel()
    _ints(seq_lens, torch.int32, "seq_lens")
    _ints(block_table, torch.int32, "block_table")
    if block_table.dim() != 2 or block_table.shape[0] != batch:
        raise ValueError(f"block_table must be [{batch}, pages], got {tuple(block_table.shape)}")
    if q_starts is None:
        per = rows // batch if batch else 0
        if per * batch != rows or (max_q is not None and max_q != per):
            raise ValueError(f"{rows} rows are not {batch} sequences of {'one length' if max_q is None else max_q}")
        max_q = per
    else:
        _ints(q_starts, torch.int32, "q_starts", batch + 1)
        max_q = rows if max_q is None else min(max_q, rows)
        if max_q < 0:
            raise ValueError("max_q < 0")
    if window < 0:
        raise ValueError("window < 0")
    window = min(window, 2 ** 31 - 1)  # a sequence has fewer keys: each query sees all of them
    most = block_table.shape[1] * cache.page_size
    max_keys = most if max_keys is None else min(max_keys, most)
    if max_keys < 0:
        raise ValueError("max_keys < 0")

    def call():
        o = out
        if o is None:
            o = torch.empty((rows, heads, d), dtype=q.dtype, device=q.device)
            if batch == 0 or max_q == 0:
                o.zero_()
        elif o.shape != q.shape or o.dtype != q.dtype:
            raise ValueError(f"out must be {q.dtype} {tuple(q.shape)}")
        _on_gpu(o, "out")
        _fits(o, 0, "out")
        s = None
        if lse and (out is not None or batch == 0 or max_q == 0):
            s = torch.full((rows, heads), -math.inf, dtype=torch.float32, device=q.device)
        elif lse:
            s = torch.empty((rows, heads), dtype=torch.float32, device=q.device)
        raw = cache._raw()
        need = mxq_kv_attention_workspace_bytes(raw, batch, rows, max_q, heads, max_keys)
        ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
        _check(mxq_kv_attention(raw, q.data_ptr(), rows, q.stride(0) if rows > 1 else 0, q.stride(1) if heads > 1 else 0,
                                heads, batch, None if q_starts is None else q_starts.data_ptr(), max_q,
                                seq_lens.data_ptr(), max_keys, block_table.data_ptr(), block_table.shape[1],
                                d ** -0.5 if scale is None else scale, window, out is None, o.data_ptr(),
                                None if s is None else s.data_ptr(), None if ws is None else ws.data_ptr(), need,
                                _raw_stream(q)), "mxq_kv_attention")
        return (o, s) if lse else o

    return _on(stream, call)
