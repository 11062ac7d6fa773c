"""include/mxq_ops.h: exported symbols, a C99 caller, statuses before any CUDA call, and the refusals of the
torch helpers, all on the CPU (no kernel runs)."""
import os
import re
import subprocess

import pytest
import torch

from block_scaled_microscaling_b200 import build as mxq_build
from block_scaled_microscaling_b200 import mxq, ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mxq_ops.h")
FP4, FP8 = mxq.FORMATS["mxfp4"], mxq.FORMATS["mxfp8"]
F32, BF16 = 0, 1


@pytest.fixture(scope="module", autouse=True)
def library():
    mxq_build.build()
    return ops.lib()


class FakeCuda:
    """A host tensor that reports is_cuda = True; everything else is the tensor's own."""
    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


def fake(*shape, dtype=torch.bfloat16):
    return FakeCuda(torch.zeros(shape, dtype=dtype))


def u8(*shape):
    return fake(*shape, dtype=torch.uint8)


def test_exports_every_declared_symbol(library):
    syms = re.findall(r"MXQ_API\s+[\w\s\*]+?\b(mxq_\w+)\s*\(", open(HEADER).read())
    assert sorted(syms) == sorted(ops.OPS_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", mxq.LIB_PATH], capture_output=True, text=True).stdout
    exported = set(re.findall(r"\bT\s+(mxq_\w+)", out))
    assert set(syms) <= exported


def test_c99_caller(tmp_path):
    src = tmp_path / "c.c"
    src.write_text('#include <stdio.h>\n#include "mxq_ops.h"\n'
                   "int main(void) { mxq_kv_cache c = {0, 0, 0, 0, 100, 8, 64, 128};\n"
                   "  if (mxq_kv_attention_workspace_bytes(&c, 0, 1, 1, 32, 100) != 0) return 1;\n"
                   "  return mxq_matmul(MXQ_MXFP4_E2M1, 0, 0, 0, 0, 1, 1, 33, 0, MXQ_BF16, 0) == MXQ_ERR_SHAPE ? 0 : 2; }\n")
    exe = tmp_path / "c"
    lib_dir = os.path.dirname(mxq.LIB_PATH)
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src),
                    "-o", str(exe), "-L", lib_dir, "-lmxq", f"-Wl,-rpath,{lib_dir}"], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_product_statuses_before_any_cuda_call():
    mm = ops.mxq_matmul
    assert mm(9, None, None, None, None, 1, 1, 32, None, BF16, None) == 1       # format
    assert mm(FP4, None, None, None, None, 1, 1, 32, None, 5, None) == 1        # dtype
    assert mm(1, None, None, None, None, 1, 1, 32, None, BF16, None) == 4       # MXFP6: not a product format
    assert mm(0, None, None, None, None, 1, 1, 32, None, BF16, None) == 4       # AXS-6
    assert mm(FP4, None, None, None, None, 1, 1, 33, None, BF16, None) == 2     # k % 32
    assert mm(FP4, None, None, None, None, 1, 1, 0, None, BF16, None) == 2
    assert mm(FP4, None, None, None, None, -1, 1, 32, None, BF16, None) == 2
    assert mm(FP8, None, None, None, None, 1, -1, 32, None, BF16, None) == 2
    assert mm(FP8, None, None, None, None, 1 << 31, 1, 32, None, BF16, None) == 2
    assert mm(FP8, None, None, None, None, 1, 1, 1 << 32, None, BF16, None) == 2
    assert mm(FP8, None, None, None, None, (1 << 31) - 400, (1 << 31) - 400, 32, None, BF16, None) == 2  # out too large
    assert mm(FP8, None, None, None, None, 0, 5, 32, None, BF16, None) == 0     # empty
    assert mm(FP8, None, None, None, None, 5, 0, 32, None, BF16, None) == 0
    assert mm(FP8, None, None, None, None, 5, 5, 32, None, BF16, None) == 1     # null
    li = lambda fmt=FP4, m=4, n=4, k=32, dt=BF16: ops.mxq_linear(fmt, None, dt, m, k, None, None, n, None, None, 0, None)  # noqa: E731
    assert [li(fmt=1), li(fmt=9), li(k=40), li(m=-1), li(dt=2), li(m=0), li(n=0), li()] == [4, 1, 2, 2, 1, 0, 0, 1]
    assert ops.mxq_linear_workspace_bytes(FP4, 5, 64) == 5 * 32 + mxq.mxq_mma_scales_bytes(5, 64)
    assert ops.mxq_linear_workspace_bytes(FP8, 130, 96) == 130 * 96 + mxq.mxq_mma_scales_bytes(130, 96)
    assert [ops.mxq_linear_workspace_bytes(f, 5, k) for f, k in ((1, 64), (9, 64), (FP4, 40))] == [0, 0, 0]
    qb = ops.mxq_quantize_both
    assert qb(FP4, FP8, None, BF16, 5, 48, None, None, None, None, None) == 2
    assert qb(FP4, FP8, None, BF16, 5, 64, None, None, None, None, None) == 1   # neither direction
    assert qb(1, FP8, None, BF16, 5, 64, 16, 16, None, None, None) == 4
    assert qb(1, FP8, None, BF16, 0, 64, None, None, 16, 16, None) == 0         # the unused format does not count
    assert qb(FP4, 2, None, BF16, 5, 64, None, None, 16, 16, None) == 4
    assert qb(FP4, 17, None, BF16, 5, 64, None, None, 16, 16, None) == 1
    assert qb(FP4, FP8, None, 3, 5, 64, 16, 16, 16, 16, None) == 1
    assert qb(FP4, FP8, None, BF16, -1, 64, 16, 16, 16, 16, None) == 2
    assert qb(FP4, FP8, None, BF16, 5, 64, 16, 16, 16, 16, None) == 1           # null source


def test_swiglu_statuses_before_any_cuda_call():
    f = lambda rows, cols, ld, dt=BF16: ops.mxq_swiglu_forward(None, None, dt, rows, cols, ld, None, None, None, None, None, None)  # noqa: E731
    b = lambda rows, cols, ld, dt=BF16: ops.mxq_swiglu_backward(None, dt, None, None, None, None, rows, cols, None, None, ld, None)  # noqa: E731
    for call in (f, b):
        assert call(4, 48, 48) == 2
        assert call(4, 64, 32) == 2            # ld < cols
        assert call(-1, 64, 64) == 2
        assert call(1 << 40, 64, 1 << 20) == 2  # size overflow
        assert call(4, 64, 68) == 3            # row stride not 16-byte aligned
        assert call(4, 64, 64, 7) == 1
        assert call(0, 64, 64) == 0
        assert call(4, 64, 64) == 1            # null


def cache(pages=4, heads=2, page=16, dim=64):
    return (None, None, None, None, pages, heads, page, dim)


def test_cache_statuses_before_any_cuda_call():
    ap = lambda c, tokens=1, ks=128, vs=128, dt=BF16: ops.mxq_kv_append(c, None, ks, None, vs, dt, tokens, None, None)  # noqa: E731
    rd = lambda c, tokens=1, dt=BF16: ops.mxq_kv_read(c, None, tokens, None, None, dt, None)  # noqa: E731
    for call in (ap, rd):
        assert call(cache(dim=96)) == 4
        assert call(cache(dim=0)) == 2
        assert call(cache(page=24)) == 2
        assert call(cache(page=0)) == 2
        assert call(cache(pages=-1)) == 2
        assert call(cache(pages=1 << 40)) == 2
        assert call(cache(heads=0)) == 2
        assert call(cache(), -1) == 2
        assert call(cache(), dt=4) == 1
        assert call(cache(), 0) == 0
        assert call(cache()) == 1
    assert ap(cache(), ks=120) == 2            # stride below a token
    assert ap(cache(), vs=132) == 3            # misaligned stride
    at = lambda c=cache(), rows=2, rs=512, hs=64, heads=4, batch=2, starts=None, mq=1, ts=4, win=0, keys=64: ops.mxq_kv_attention(  # noqa: E731
        c, None, rows, rs, hs, heads, batch, starts, mq, None, keys, None, ts, 1.0, win, 0, None, None, None, 0, None)
    assert at(cache(dim=32)) == 4
    assert at(heads=3) == 2
    assert at(heads=0) == 2
    assert at(batch=-1) == 2
    assert at(mq=2) == 2                       # 2 rows are not 2 sequences of 2 queries
    assert at(win=-1) == 2
    assert at(keys=-1) == 2
    assert at(rs=516) == 3
    assert at(hs=68) == 3
    assert at(rows=0, mq=0) == 0
    assert at(rows=0, batch=0) == 0
    assert at(starts=16, mq=0) == 0
    assert at() == 1
    ws = ops.mxq_kv_attention_workspace_bytes
    assert ws(cache(dim=96), 1, 1, 1, 2, 64) == 0
    assert ws(cache(), 1, 1, 1, 2, 64) == 0                       # few keys: one split
    assert ws(cache(pages=4096), 1, 1, 1, 2, 65536) > 0           # many: partial sums
    assert ws(cache(pages=4096), 1, 1, 128, 2, 65536) == ws(cache(pages=4096), 1, 1, 1, 2, 65536)  # one row is one query


def test_helpers_refuse_host_tensors():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    c, s = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    w = torch.zeros((64, 64), dtype=torch.bfloat16)
    for call in [lambda: ops.matmul(c, s, c, s, "mxfp4"), lambda: ops.quantize_both(x, "mxfp4"),
                 lambda: ops.linear(x, c, s, "mxfp4"), lambda: ops.linear_ste(x, w), lambda: ops.swiglu(x),
                 lambda: ops.KVCache(*(torch.zeros((1, 1, 16, n), dtype=torch.uint8) for n in (32, 2, 32, 2)))]:
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_matmul_helper_refusals():
    s = u8(512)
    for call in [lambda: ops.matmul(u8(4, 32), s, u8(4, 48), s, "mxfp4"),      # different k
                 lambda: ops.matmul(u8(4, 40), s, u8(4, 40), s, "mxfp4"),      # not whole blocks
                 lambda: ops.matmul(u8(128), s, u8(4, 32), s, "mxfp4"),
                 lambda: ops.matmul(u8(4, 32), u8(511), u8(4, 32), s, "mxfp4"),
                 lambda: ops.matmul(u8(200, 32), s, u8(4, 32), s, "mxfp4"),    # 200 rows take two tile rows
                 lambda: ops.matmul(FakeCuda(torch.zeros((32, 4), dtype=torch.uint8).t()), s, u8(4, 32), s, "mxfp4"),
                 lambda: ops.matmul(u8(4, 32), s, u8(4, 32), s, "mxfp4", out=fake(4, 3)),
                 lambda: ops.matmul(u8(4, 32), s, u8(4, 32), s, "mxfp4", out=FakeCuda(torch.zeros((4, 8), dtype=torch.bfloat16)[:, ::2])),
                 lambda: ops.matmul(u8(4, 32), s, u8(4, 32), s, "nvfp4")]:
        with pytest.raises(ValueError):
            call()
    for call in [lambda: ops.matmul(u8(4, 32), s, u8(4, 32), s, "mxfp4", out=fake(4, 4), dtype=torch.float32),
                 lambda: ops.matmul(fake(4, 32), s, u8(4, 32), s, "mxfp4")]:
        with pytest.raises(TypeError):
            call()
    for fmt in ("axs6", "mxfp6_e2m3", "mxfp6_e3m2"):
        with pytest.raises(mxq.MXQError) as e:
            ops.matmul(u8(4, 32), s, u8(4, 32), s, fmt)
        assert e.value.status == 4
    with pytest.raises(mxq.MXQError) as e:
        ops.matmul(u8(4, 0), s, u8(4, 0), s, "mxfp4")
    assert e.value.status == 2


def test_linear_helper_refusals():
    for call in [lambda: ops.quantize_both(fake(4, 64)), lambda: ops.quantize_both(fake(2, 4, 64), "mxfp4"),
                 lambda: ops.quantize_both(FakeCuda(torch.zeros((64, 32)).t()), "mxfp4"),
                 lambda: ops.linear(fake(4, 64), u8(8, 16), u8(512), "mxfp4"),
                 lambda: ops.linear(FakeCuda(torch.zeros((64, 4)).t()), u8(8, 32), u8(512), "mxfp4"),
                 lambda: ops.linear_ste(fake(4, 64), fake(32, 32)), lambda: ops.linear_ste(fake(4, 64), fake(32)),
                 lambda: ops.swiglu(fake(4, 64), fake(4, 32)),
                 lambda: ops.swiglu(fake(4, 64), fake(4, 64, dtype=torch.float32))]:
        with pytest.raises(ValueError):
            call()
    for call in [lambda: ops.linear_ste(fake(4, 64), fake(33, 64)), lambda: ops.linear_ste(fake(4, 48), fake(32, 48)),
                 lambda: ops.quantize_both(fake(4, 48), "mxfp8"), lambda: ops.swiglu(fake(4, 96)),
                 lambda: ops.swiglu(fake(4, 63)), lambda: ops.swiglu(fake(4, 0), fake(4, 0))]:
        with pytest.raises(mxq.MXQError) as e:
            call()
        assert e.value.status == 2
    with pytest.raises(mxq.MXQError) as e:
        ops.linear_ste(fake(4, 64), fake(32, 64), "mxfp6_e2m3")
    assert e.value.status == 4
    for call in [lambda: ops.linear_ste(fake(4, 64, dtype=torch.float16), fake(32, 64)),
                 lambda: ops.swiglu(fake(4, 64, dtype=torch.float16))]:
        with pytest.raises(TypeError):
            call()


def fake_cache(pages=4, heads=2, page=16, dim=64):
    return ops.KVCache(*(u8(pages, heads, page, n) for n in (dim // 2, dim // 32, dim // 2, dim // 32)))


def test_cache_helper_refusals():
    i64 = lambda n: fake(n, dtype=torch.int64)  # noqa: E731
    i32 = lambda *n: fake(*n, dtype=torch.int32)  # noqa: E731
    c = fake_cache()
    for call in [lambda: ops.KVCache(u8(4, 16, 32), u8(4, 16, 2), u8(4, 16, 32), u8(4, 16, 2)),
                 lambda: ops.KVCache(u8(4, 2, 16, 32), u8(4, 2, 16, 1), u8(4, 2, 16, 32), u8(4, 2, 16, 2)),
                 lambda: ops.KVCache(u8(4, 2, 16, 32), u8(4, 2, 16, 2), u8(4, 2, 32, 32), u8(4, 2, 16, 2)),
                 lambda: ops.kv_append(fake(3, 2, 32), fake(3, 2, 64), c, i64(3)),
                 lambda: ops.kv_append(fake(3, 2, 64), fake(4, 2, 64), c, i64(3)),
                 lambda: ops.kv_append(fake(3, 2, 64), fake(3, 2, 64, dtype=torch.float32), c, i64(3)),
                 lambda: ops.kv_append(fake(3, 2, 64), fake(3, 2, 64), c, i64(2)),
                 lambda: ops.kv_append(FakeCuda(torch.zeros((3, 64, 2)).mT), fake(3, 2, 64, dtype=torch.float32), c, i64(3)),
                 lambda: ops.kv_read(c, torch.zeros(3, dtype=torch.int64)),
                 lambda: ops.kv_attention(fake(2, 4, 32), c, i32(2, 4), i32(2)),
                 lambda: ops.kv_attention(fake(2, 4, 64, dtype=torch.float32), c, i32(2, 4), i32(2)),
                 lambda: ops.kv_attention(fake(2, 3, 64), c, i32(2, 4), i32(2)),
                 lambda: ops.kv_attention(fake(2, 4, 64), c, i32(3, 4), i32(2)),
                 lambda: ops.kv_attention(fake(3, 4, 64), c, i32(2, 4), i32(2)),
                 lambda: ops.kv_attention(fake(4, 4, 64), c, i32(2, 4), i32(2), max_q=1),
                 lambda: ops.kv_attention(fake(2, 4, 64), c, i32(2, 4), i32(2), q_starts=i32(2)),
                 lambda: ops.kv_attention(fake(2, 4, 64), c, i32(2, 4), i32(2), window=-1),
                 lambda: ops.kv_attention(fake(2, 4, 64), c, i32(2, 4), i32(2), max_keys=-1),
                 lambda: ops.kv_attention(fake(2, 4, 64), c, i32(2, 4), torch.zeros(2, dtype=torch.int32)),
                 lambda: ops.kv_attention(FakeCuda(torch.zeros((2, 4, 128), dtype=torch.bfloat16)[..., ::2]), c, i32(2, 4), i32(2))]:
        with pytest.raises(ValueError):
            call()
    for call in [lambda: ops.kv_append(fake(3, 2, 64), fake(3, 2, 64), c, i32(3)),
                 lambda: ops.kv_read(c, i32(3)),
                 lambda: ops.kv_attention(fake(2, 4, 64), c, i64(8), i32(2)),
                 lambda: ops.kv_attention(fake(2, 4, 64), c, i32(2, 4), i64(2))]:
        with pytest.raises(TypeError):
            call()


def test_roles_with_warp_collectives_share_the_verdict_of_a_wait():
    """A bounded wait may end differently for the lanes of a warp. In a role of the many-query attention kernel whose lanes
    meet in shuffles or warp barriers, a lane that leaves alone would hang the others: the verdict has to be the warp's."""
    src = open(os.path.join(ROOT, "block_scaled_microscaling_b200", "csrc", "mxq_attention_tc.cu")).read()
    body = src[src.index("void __launch_bounds__(kTcThreads"):src.index("template <int D> cudaError_t go(")]
    roles = re.split(r"(?=// ---- )", body)[1:]
    assert len(roles) == 5
    together = 0
    for role in roles:
        waits = len(re.findall(r"\bmbar_wait\(", role))
        assert waits > 0
        if re.search(r"__syncwarp|__shfl|__reduce|__any_sync", role):
            together += 1
            assert len(re.findall(r"__all_sync\(0xFFFFFFFFu, mbar_wait\(", role)) == waits, role.splitlines()[0]
    assert together >= 3


@pytest.mark.parametrize("dim", [64, 128])
def test_a_workspace_for_many_keys_is_enough_for_fewer(dim):
    """The size never falls as max_keys grows, whatever the form that the call takes, and has no end at 2^31."""
    ws = ops.mxq_kv_attention_workspace_bytes
    for heads in (1, 2, 8):
        c = cache(pages=1 << 20, heads=heads, dim=dim)
        for group, batch, queries in [(4, 1, 128), (4, 1, 64), (4, 3, 40), (8, 9, 16), (1, 1, 300), (4, 1, 1), (4, 2, 1), (4, 600, 1), (16, 1, 2), (1, 5, 7)]:
            sizes = [ws(c, batch, batch * queries, queries, heads * group, 16 * k)
                     for k in (*range(1, 600, 3), 1000, 5000, 40000, 1 << 20, 1 << 26, (1 << 27) - 1, 1 << 27, 1 << 28, 1 << 50)]
            assert sizes == sorted(sizes), (heads, group, batch, queries)
            assert sizes[-1] == sizes[-4]


@pytest.mark.parametrize("heads,page,dim", [(0, 16, 64), (2, 0, 64), (2, 16, 0), (2, 16, 16)])
def test_a_cache_without_heads_rows_or_dimensions_is_refused(heads, page, dim):
    with pytest.raises(ValueError, match="a cache needs"):
        fake_cache(heads=heads, page=page, dim=dim)
    assert fake_cache(pages=0).pages == 0


def test_the_torch_module_shares_the_cpp_library():
    """A second C++ library linked into the module (a compiler with the static one alone) ended the process at the first
    exception."""
    path = os.path.join(os.path.dirname(mxq.LIB_PATH), "_ops.so")
    needed = subprocess.run(["readelf", "-d", path], capture_output=True, text=True, check=True).stdout
    assert "[libstdc++.so.6]" in needed
    own = subprocess.run(["nm", "-D", "--defined-only", path], capture_output=True, text=True, check=True).stdout
    assert "_ZNSo" not in own and "St6locale" not in own      # streams, locales


@pytest.mark.parametrize("status", [1, 2, 3, 4, 5])
def test_the_status_of_a_refused_training_call_is_kept(status, monkeypatch):
    """The module reports the entry point and its status; the exception carries both, whatever the devices are."""
    def refuse(*args):
        raise RuntimeError(f"mxq_quantize_both: status {status} ({mxq.mxq_status_string(status)})")

    module = type("M", (), {"linear_ste": staticmethod(refuse), "swiglu": staticmethod(refuse)})
    monkeypatch.setattr(ops, "_native", lambda: module)
    for call in (lambda: ops.linear_ste(fake(4, 64), fake(32, 64)), lambda: ops.swiglu(fake(4, 64)), lambda: ops.swiglu(fake(4, 32), fake(4, 32))):
        with pytest.raises(mxq.MXQError, match="mxq_quantize_both") as e:
            call()
        assert e.value.status == status

    def other(*args):
        raise RuntimeError("CUDA out of memory")

    monkeypatch.setattr(module, "swiglu", staticmethod(other))
    with pytest.raises(RuntimeError, match="out of memory"):
        ops.swiglu(fake(4, 64))
