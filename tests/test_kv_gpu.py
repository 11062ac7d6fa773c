"""Paged MXFP4 cache on the GPU: append and read bit for bit, attention against a 64-bit implementation.

Tolerance of attention: with w the softmax weights, each score's error ds <= scale * (D + 4) 2^-23 sum |q k| (D
fp32 additions of exact products, four roundings) changes a weight by a factor of at most e^(2 ds); the weights round
to f16 (half a step, 2^-11, or 2^-25 of the largest near zero), the hardware's 2^x adds 2^-21, and the sums of n keys
in fp32 n 2^-23: |error| <= sum w |v| (2^-10 + 4 ds + n 2^-23) + n 2^-24 max |v|, plus half a step of bf16."""
import math

import pytest
import torch

from block_scaled_microscaling_b200 import mxq, ops

pytestmark = pytest.mark.gpu


def rand(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def junk_cache(seed, pages, kv, page, d):
    """A cache of arbitrary bytes: every code, every scale byte, NaN scales among them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return ops.KVCache(*(torch.randint(256, (pages, kv, page, n), generator=g, device="cuda", dtype=torch.uint8)
                         for n in (d // 2, d // 32, d // 2, d // 32)))


def state(c):
    return [t.clone() for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,kv,page,d", [(1, 1, 16, 64), (1, 8, 64, 128), (37, 2, 48, 128), (300, 3, 16, 64), (1000, 8, 128, 128)])
def test_append_and_read(tokens, kv, page, d, dtype):
    pages = tokens // page + 3
    c = junk_cache(1, pages, kv, page, d)
    before = state(c)
    k, v = (3 * rand(2, tokens, kv, d)).to(dtype), rand(3, tokens, kv, d).to(dtype)
    slots = torch.randperm(pages * page, device="cuda")[:tokens]
    ops.kv_append(k, v, c, slots)
    at, off = slots // page, slots % page
    for x, codes, scales, oc, os_ in ((k, c.k_codes, c.k_scales, *before[:2]), (v, c.v_codes, c.v_scales, *before[2:])):
        want = mxq.quantize(x.contiguous(), "mxfp4")
        assert torch.equal(codes[at, :, off].reshape(-1), want[0].view(-1))
        assert torch.equal(scales[at, :, off].reshape(-1), want[1].view(-1))
        oc[at, :, off], os_[at, :, off] = codes[at, :, off], scales[at, :, off]
        assert torch.equal(codes, oc) and torch.equal(scales, os_)  # nothing else changed
    for dt in (torch.bfloat16, torch.float32):
        gk, gv = ops.kv_read(c, slots, dtype=dt)
        assert gk.dtype == dt and gk.shape == k.shape
        assert torch.equal(gk.float(), mxq.fake_quantize(k.contiguous(), "mxfp4").float())
        assert torch.equal(gv.float(), mxq.fake_quantize(v.contiguous(), "mxfp4").float())


def test_append_strided_tokens_and_slots_outside():
    c = junk_cache(1, 4, 2, 16, 64)
    before = state(c)
    qkv = rand(5, 6, 8, 64).bfloat16()        # heads 4, 5 are keys, 6, 7 values of a fused projection
    k, v = qkv[:, 4:6], qkv[:, 6:8]
    slots = torch.tensor([5, -1, 63, 64, 1 << 40, 0], device="cuda")
    ops.kv_append(k, v, c, slots)
    gk, gv = ops.kv_read(c, slots)
    ok = torch.tensor([True, False, True, False, False, True], device="cuda")
    assert torch.equal(gk[ok], mxq.fake_quantize(k[ok].contiguous(), "mxfp4"))
    assert torch.equal(gv[ok], mxq.fake_quantize(v[ok].contiguous(), "mxfp4"))
    assert (gk[~ok] == 0).all() and (gv[~ok] == 0).all()
    keep = torch.ones((4, 16), dtype=torch.bool, device="cuda")
    for s in (5, 63, 0):
        keep[s // 16, s % 16] = False
    for now, old in zip(state(c), before):
        assert torch.equal(now.transpose(1, 2)[keep], old.transpose(1, 2)[keep])
    ops.kv_append(k[:0], v[:0], c, slots[:0])
    assert ops.kv_read(c, slots[:0])[0].shape == (0, 2, 64)


def test_nan_and_zero_rows_through_the_cache():
    c = ops.KVCache.empty(1, 1, 16, 64)
    k, v = rand(1, 2, 1, 64).bfloat16(), rand(2, 2, 1, 64).bfloat16()
    k[0, 0, 40], v[1] = float("nan"), 0
    ops.kv_append(k, v, c, torch.arange(2, device="cuda"))
    gk, gv = ops.kv_read(c, torch.arange(2, device="cuda"))
    assert torch.equal(torch.isnan(gk), torch.isnan(mxq.fake_quantize(k, "mxfp4"))) and torch.isnan(gk[0, 0, 32:]).all()
    assert (gv[1] == 0).all()


# ---- attention ------------------------------------------------------------------------------

def tables(lens, page, pages, width=None, seed=0):
    per = [-(-n // page) for n in lens]
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int()
    assert sum(per) <= pages
    t = torch.full((len(lens), width or max(1, max(per, default=1))), -7, dtype=torch.int32)
    at = 0
    for i, n in enumerate(per):
        t[i, :n] = order[at:at + n]
        at += n
    return t.cuda()


def reference(q, cache, table, lens, starts, window=0, scale=None):
    """(out, lse, tolerance of out, rows written) in 64 bits, one sequence at a time."""
    rows, heads, d = q.shape
    kv, page = cache.kv_heads, cache.page_size
    scale = d ** -0.5 if scale is None else scale
    out = torch.zeros((rows, heads, d), dtype=torch.float64, device="cuda")
    lse = torch.full((rows, heads), -math.inf, dtype=torch.float64, device="cuda")
    tol, mine = torch.zeros_like(out), torch.zeros(rows, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        r0, r1 = starts[b], starts[b + 1]
        mine[r0:r1] = True
        if n == 0 or r1 == r0:
            continue
        j = torch.arange(n, device="cuda")
        pg = table[b, j // page].long()
        there = (pg >= 0) & (pg < cache.pages)
        slots = torch.where(there, pg * page + j % page, -1)
        k, v = (t.double().repeat_interleave(heads // kv, 1) for t in ops.kv_read(cache, slots, dtype=torch.float32))  # [n, heads, d]
        x = q[r0:r1].double()
        pos = n - (r1 - r0) + torch.arange(r1 - r0, device="cuda")[:, None]
        seen = (j <= pos) & there
        if window:
            seen &= j > pos - window
        s = torch.einsum("ihd,jhd->hij", x, k) * scale
        s = s.masked_fill(~seen, -math.inf)
        top = s.amax(-1, keepdim=True)
        w = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
        w = torch.where(seen, w, 0.0)
        total = w.sum(-1, keepdim=True)
        lse[r0:r1] = (top + torch.log(total))[..., 0].T
        w = w / torch.where(total == 0, 1.0, total)
        v = v.transpose(0, 1)[:, None]                           # [heads, 1, n, d]
        use = seen[None, :, :, None]
        pv = torch.where(use, w[..., None] * v, 0.0)
        out[r0:r1] = pv.sum(2).transpose(0, 1)
        ds = (torch.einsum("ihd,jhd->hij", x.abs(), k.abs().nan_to_num()) * abs(scale)).masked_fill(~seen, 0).amax(-1) * (d + 4) * 2.0 ** -23
        most = torch.where(use, v.abs().nan_to_num(), 0.0).amax(2)
        tol[r0:r1] = (pv.abs().sum(2) * (2.0 ** -10 + 4 * ds[..., None] + n * 2.0 ** -23) + n * 2.0 ** -24 * most).transpose(0, 1)
    return out, lse, tol, mine


def filled(seed, pages, kv, page, d, k_scale=1.0, v_scale=1.0):
    c = junk_cache(seed, pages, kv, page, d)
    slots = torch.arange(pages * page, device="cuda")
    k = rand(seed + 1, pages * page, kv, d) * k_scale
    k[..., 3] *= 8
    ops.kv_append(k.bfloat16(), (rand(seed + 2, pages * page, kv, d) * v_scale).bfloat16(), c, slots)
    return c


def spoil_tails(c, table, lens):
    """Bytes behind each sequence's last key: every code and NaN scales."""
    for b, n in enumerate(lens):
        if n % c.page_size:
            pg = int(table[b, n // c.page_size])
            for t, x in ((c.k_codes, 0x77), (c.k_scales, 0xFF), (c.v_codes, 0x77), (c.v_scales, 0xFF)):
                t[pg, :, n % c.page_size:] = x


def check(q, c, table, lens, starts=None, window=0, scale=None, max_q=None, **kw):
    st = starts if starts is not None else [i * (q.shape[0] // len(lens)) for i in range(len(lens) + 1)]
    dev_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    dev_starts = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    if max_q is None and starts is not None:
        max_q = max([b - a for a, b in zip(st, st[1:])] + [0])
    got, lse = ops.kv_attention(q, c, table, dev_lens, q_starts=dev_starts, max_q=max_q, window=window, scale=scale, lse=True, **kw)
    plain = ops.kv_attention(q, c, table, dev_lens, q_starts=dev_starts, max_q=max_q, window=window, scale=scale, **kw)
    assert torch.equal(plain.nan_to_num(nan=7.5), got.nan_to_num(nan=7.5))  # the plain call's way
    out, want_lse, tol, mine = reference(q, c, table, lens, st, window, scale)
    nan = torch.isnan(out)
    assert torch.equal(torch.isnan(got), nan)
    err = (got.double() - out).abs()
    bad = (err > tol + out.abs() * 2.0 ** -8) & ~nan
    assert not bad.any(), (int(bad.sum()), torch.nonzero(bad)[:5].tolist(), float(err[bad].max()))
    assert torch.equal(lse == -math.inf, want_lse == -math.inf)
    fin = torch.isfinite(want_lse)
    # a log-sum-exp is off by the scores' errors and a few roundings of its own size
    ds = 2.0 ** -12
    assert ((lse.double() - want_lse).abs()[fin] <= ds * (1 + want_lse.abs()[fin])).all()
    assert (got[~mine] == 0).all()
    return got


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv,group", [(1, 1), (2, 4), (1, 8), (3, 3), (2, 12), (1, 32)])
@pytest.mark.parametrize("lens", [[1], [16], [333], [17, 0, 5], [130, 64, 1, 200], [0, 0], [0, 129, 0, 0, 140, 0]])
def test_single_tokens(lens, kv, group, d):
    page, pages = 16, 44
    c = filled(len(lens) + d, pages, kv, page, d)
    table = tables(lens, page, pages)
    spoil_tails(c, table, lens)
    check(rand(7, len(lens), kv * group, d).bfloat16(), c, table, lens)


@pytest.mark.parametrize("page", [16, 48, 128])
@pytest.mark.parametrize("d,kv,group", [(64, 2, 4), (128, 1, 8), (128, 2, 2)])
@pytest.mark.parametrize("lens,news", [([40], [40]), ([300, 20, 7], [33, 20, 1]), ([5, 64], [9, 64]), ([600], [130]), ([33, 0, 18], [2, 3, 0])])
def test_several_queries_causal(lens, news, d, kv, group, page):
    pages = sum(-(-n // page) for n in lens) + 2
    c = filled(d + page, pages, kv, page, d)
    table = tables(lens, page, pages)
    spoil_tails(c, table, lens)
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    check(rand(8, starts[-1] + 3, kv * group, d).bfloat16(), c, table, lens, starts)


@pytest.mark.parametrize("window", [1, 16, 37, 1000])
@pytest.mark.parametrize("news", [[1, 1], [40, 3]])
def test_window(window, news):
    lens, page = [310, 45], 32
    c = filled(3, 14, 2, page, 128)
    table = tables(lens, page, 14)
    spoil_tails(c, table, lens)
    check(rand(9, sum(news), 8, 128).bfloat16(), c, table, lens, [0, news[0], sum(news)], window=window)


@pytest.mark.parametrize("d,group", [(128, 4), (64, 16)])
@pytest.mark.parametrize("news", [1, 5])
def test_long_sequences_are_split_and_joined(news, d, group):
    lens, page = [9000, 3, 4100], 64
    pages = sum(-(-n // page) for n in lens) + 1
    c = filled(4, pages, 2, page, d)
    table = tables(lens, page, pages)
    spoil_tails(c, table, lens)
    q = rand(10, 3 * news, 2 * group, d).bfloat16()
    got = check(q, c, table, lens, [0, news, 2 * news, 3 * news])
    assert ops.mxq_kv_attention_workspace_bytes(c._raw(), 3, 3 * news, news, 2 * group, table.shape[1] * page) > 0
    for _ in range(3):  # the same bits every time
        assert torch.equal(got, check(q, c, table, lens, [0, news, 2 * news, 3 * news]))


@pytest.mark.parametrize("batch", [500, 512, 513, 700])
def test_many_sequences(batch):
    """Up to 512 sequences share the CTAs evenly, more are split one by one; some have no key, some one, some many."""
    page, width = 16, 12
    g = torch.Generator().manual_seed(batch)
    lens = torch.randint(0, 60, (batch,), generator=g)
    lens[::7], lens[5::50] = 0, page * width - 3
    pages = 900
    c = filled(3, pages, 2, page, 64)
    table = torch.randint(0, pages, (batch, width), generator=g).int().cuda()
    check(rand(4, batch, 4, 64).bfloat16(), c, table, lens.tolist())


@pytest.mark.parametrize("d,kv,group", [(128, 2, 4), (64, 1, 8), (128, 1, 1)])
@pytest.mark.parametrize("lens,news", [([5000, 900, 0, 130], [100, 37, 5, 70]), ([3333], [129]), ([128 * 9], [40])])
def test_many_queries_over_long_prefixes(lens, news, d, kv, group):
    page = 32
    pages = sum(-(-n // page) for n in lens) + 1
    c = filled(7, pages, kv, page, d)
    table = tables(lens, page, pages)
    spoil_tails(c, table, lens)
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    q = rand(5, starts[-1] + 2, kv * group, d).bfloat16()
    got = check(q, c, table, lens, starts)
    assert torch.equal(got, check(q, c, table, lens, starts))
    check(q, c, table, lens, starts, window=500)


@pytest.mark.parametrize("max_q,group", [(1, 1), (2, 4), (3, 4), (1, 16)])
def test_shares_end_anywhere(max_q, group):
    """Lengths around multiples of a share, with rows of no sequence on both sides."""
    page, lens = 16, [1300, 128, 0, 2049, 127, 16, 700]
    pages = sum(-(-n // page) for n in lens) + 1
    c = filled(6, pages, 2, page, 128)
    table = tables(lens, page, pages)
    spoil_tails(c, table, lens)
    starts = [2 + max_q * i for i in range(len(lens) + 1)]
    check(rand(5, starts[-1] + 3, 2 * group, 128).bfloat16(), c, table, lens, starts)
    check(rand(5, starts[-1] + 3, 2 * group, 128).bfloat16(), c, table, lens, starts, window=333)


@pytest.mark.parametrize("k_scale,v_scale", [(2.0 ** -40, 2.0 ** -60), (2.0 ** 10, 2.0 ** 70), (30.0, 1e-4)])
def test_block_scales_far_from_one(k_scale, v_scale):
    lens, page = [200, 70], 16
    c = filled(5, 20, 2, page, 128, k_scale, v_scale)
    check((rand(11, 2, 8, 128) / k_scale).bfloat16(), c, tables(lens, page, 20), lens)
    check((rand(11, 60, 8, 128) / k_scale).bfloat16(), c, tables(lens, page, 20), lens)


def test_block_scales_that_grow_and_shrink_along_a_sequence():
    page, n = 16, 256
    c = ops.KVCache.empty(16, 1, page, 64)
    size = torch.exp2(torch.tensor([-30.0, 0, 14, -9, 21, 22, 3, -20], device="cuda")).repeat_interleave(32)[:, None, None]
    ops.kv_append((rand(1, n, 1, 64) * size.clamp(max=8)).bfloat16(), (rand(2, n, 1, 64) * size).bfloat16(), c, torch.arange(n, device="cuda"))
    table = torch.arange(16, dtype=torch.int32, device="cuda")[None]
    for rows in (1, 8, 60):
        check(rand(12, rows, 4, 64).bfloat16(), c, table, [n], [0, rows])


def test_large_scores_and_a_given_scale():
    lens, page = [150], 16
    c = filled(6, 10, 1, page, 128, 20.0)
    check((rand(13, 1, 8, 128) * 20).bfloat16(), c, tables(lens, page, 10), lens)
    check(rand(13, 1, 8, 128).bfloat16(), c, tables(lens, page, 10), lens, scale=0.01)
    check(rand(13, 1, 8, 128).bfloat16(), c, tables(lens, page, 10), lens, scale=0.0)
    check((rand(13, 1, 8, 128) * 2.0 ** 100).bfloat16(), c, tables(lens, page, 10), lens, scale=2.0 ** -104)
    for scale in (None, 0.01, 0.0, -0.05):
        check((rand(13, 50, 8, 128) * 20).bfloat16(), c, tables(lens, page, 10), lens, scale=scale)


def test_nan_blocks_reach_only_the_queries_that_see_them():
    n, page = 64, 16
    c = filled(7, 4, 1, page, 128)
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    c.v_scales[2, 0, 5, 1] = 0xFF      # key 37, dimensions 32 .. 63
    got = check(rand(14, n, 4, 128).bfloat16(), c, table, [n], [0, n])
    nan = torch.isnan(got)
    assert nan[37:, :, 32:64].all() and not nan[:37].any() and not nan[:, :, :32].any() and not nan[:, :, 64:].any()
    got = check(rand(14, n, 4, 128).bfloat16(), c, table, [n], [0, n], window=8)
    assert torch.isnan(got[37:45, :, 32:64]).all() and not torch.isnan(got[45:]).any()
    c.v_scales[2, 0, 5, 1] = 127
    c.k_scales[3, 0, 2, 0] = 0xFF      # key 50: every later query's scores
    got = ops.kv_attention(rand(14, n, 4, 128).bfloat16(), c, table, torch.tensor([n], dtype=torch.int32, device="cuda"))
    assert torch.isnan(got[50:]).all() and not torch.isnan(got[:50]).any()


def spoil(c, table, b, keys, scale):
    """Every code of keys of sequence b, and their scales one byte (0xFE: 2^127; 0xFF: NaN)."""
    for j in keys:
        pg, off = int(table[b, j // c.page_size]), j % c.page_size
        for t, x in ((c.k_codes, 0x77), (c.k_scales, scale), (c.v_codes, 0x77), (c.v_scales, scale)):
            t[pg, :, off] = x


@pytest.mark.parametrize("scale", [0xFE, 0xFF])
@pytest.mark.parametrize("window", [1, 5, 37, 130, 300])
@pytest.mark.parametrize("news,group,d", [([1, 1], 4, 128), ([3, 2], 4, 64), ([8, 5], 4, 128), ([40, 3], 4, 128), ([100, 70], 2, 64)])
def test_bytes_in_front_of_the_window_do_not_count(news, group, d, window, scale):
    """Keys in front of every query's window hold the largest scales, or NaN: few queries, queries in shares, row tiles."""
    page = 32
    for lens in ([310, 145], [700, 333]):
        pages = sum(-(-n // page) for n in lens) + 1
        c = filled(3, pages, 2, page, d)
        table = tables(lens, page, pages)
        for b, (n, new) in enumerate(zip(lens, news)):
            spoil(c, table, b, range(max(0, n - new - window + 1)), scale)
        spoil_tails(c, table, lens)
        starts = [0, news[0], sum(news)]
        check(rand(9, sum(news), 2 * group, d).bfloat16(), c, table, lens, starts, window=window)
        one = [0, news[0]]                                      # a sequence alone
        check(rand(9, news[0], 2 * group, d).bfloat16(), c, table[:1], lens[:1], one, window=window)


@pytest.mark.parametrize("scale", [0xFE, 0xFF])
@pytest.mark.parametrize("d,group,news", [(128, 4, 200), (64, 8, 70), (64, 1, 600)])
def test_bytes_behind_the_keys_of_a_row_tile_do_not_count(d, group, news, scale):
    """The last key, which the last query alone sees, holds the largest scales: queries of other row tiles (256 rows each) keep
    their results."""
    lens, page = [news + 50], 16
    c = filled(3, -(-lens[0] // page), 2, page, d)
    table = tables(lens, page, c.pages)
    spoil(c, table, 0, [lens[0] - 1], scale)
    q = rand(9, news, 2 * group, d).bfloat16()
    got = ops.kv_attention(q, c, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    out, _, tol, _ = reference(q, c, table, lens, [0, news])
    others = (news * group - 1) // 256 * 256 // group           # queries that share no tile with the last
    assert others > 0
    assert ((got.double() - out).abs() <= tol + out.abs() * 2.0 ** -8)[:others].all()


@pytest.mark.parametrize("group", [4, 16])
def test_bytes_behind_the_queries_that_are_computed_do_not_count(group):
    """Queries beyond max_q are left out, and the keys that they alone see do not count."""
    lens, page, max_q = [90], 16, 3
    c = filled(3, 6, 2, page, 128)
    table = tables(lens, page, 6)
    spoil(c, table, 0, range(83, 90), 0xFE)                       # queries stand at 80 .. 89
    q = rand(9, 10, 2 * group, 128).bfloat16()
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    got = ops.kv_attention(q, c, table, dev(lens), q_starts=dev([0, 10]), max_q=max_q)
    out, _, tol, _ = reference(q, c, table, lens, [0, 10])
    assert ((got.double() - out).abs() <= tol + out.abs() * 2.0 ** -8)[:max_q].all()


@pytest.mark.parametrize("window", [1, 4, 17, 40])
@pytest.mark.parametrize("lens", [[3000, 700], [1500, 0, 2, 900], [400] * 70])
def test_batches_that_see_few_keys(lens, window):
    page, d = 16, 128
    pages = sum(-(-n // page) for n in lens) + 1
    c = filled(2, pages, 2, page, d)
    table = tables(lens, page, pages)
    spoil_tails(c, table, lens)
    check(rand(4, len(lens), 8, d).bfloat16(), c, table, lens, window=window)


@pytest.mark.parametrize("d", [64, 128])
def test_many_queries_of_empty_sequences_give_zeros(d):
    batch, news = 150, 40   # more CTAs than fit at a time; 160 rows each
    c = filled(1, 4, 2, 16, d)
    q = rand(2, batch * news, 8, d).bfloat16()
    for n in (0, -3):
        lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
        out, lse = ops.kv_attention(q, c, torch.zeros(batch, 2, dtype=torch.int32, device="cuda"), lens, lse=True)
        assert (out == 0).all() and (lse == -math.inf).all()
    # the queries before the first key see nothing
    lens = torch.full((batch,), 5, dtype=torch.int32, device="cuda")
    out = ops.kv_attention(q, c, torch.zeros(batch, 2, dtype=torch.int32, device="cuda"), lens).view(batch, news, 8, d)
    assert (out[:, :-5] == 0).all() and (out[:, -5:] != 0).any(-1).all()


def test_offsets_beyond_32_bits():
    """4.9 GB of codes each: pages at both ends of the cache."""
    pages, kv, page, d = 150_000, 8, 64, 128
    c = ops.KVCache.empty(pages, kv, page, d)
    assert c.k_codes.numel() > 1 << 32
    lens = [200, 70]
    table = torch.tensor([[pages - 1, 0, pages - 2, 131_073], [pages - 3, pages // 2, 0, 0]], dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):
        pos = torch.arange(n, device="cuda")
        slots = table[b, pos // page].long() * page + pos % page
        k, v = rand(b, n, kv, d).bfloat16(), rand(b + 5, n, kv, d).bfloat16()
        ops.kv_append(k, v, c, slots)
        assert torch.equal(ops.kv_read(c, slots)[1], mxq.fake_quantize(v, "mxfp4"))
    check(rand(9, 2, 32, d).bfloat16(), c, table, lens)
    check(rand(9, 60, 32, d).bfloat16(), c, table, lens, [0, 40, 60])


def test_pages_outside_the_cache_are_not_seen():
    lens, page = [100, 40], 16
    c = filled(8, 12, 2, page, 64)
    table = tables(lens, page, 12)
    table[0, 2], table[0, 6], table[1, 0] = -1, 12, 2 ** 31 - 1
    check(rand(15, 2, 4, 64).bfloat16(), c, table, lens)
    check(rand(15, 60, 4, 64).bfloat16(), c, table, lens)
    table[:] = -1
    got, lse = ops.kv_attention(rand(15, 2, 4, 64).bfloat16(), c, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), lse=True)
    assert (got == 0).all() and (lse == -math.inf).all()


def test_lengths_beyond_the_table_negative_ones_and_max_keys():
    page = 16
    c = filled(9, 8, 1, page, 64)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    q = rand(16, 2, 4, 64).bfloat16()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    want = ops.kv_attention(q, c, table, i32(64, 0))
    assert torch.equal(ops.kv_attention(q, c, table, i32(1000000, -5)), want)
    assert torch.equal(ops.kv_attention(q, c, table, i32(64, 64), max_keys=30), ops.kv_attention(q, c, table, i32(30, 30)))
    assert (ops.kv_attention(q, c, table[:, :0], i32(64, 64)) == 0).all()


def test_rows_of_no_sequence_stay_and_starts_are_clamped():
    lens, page = [50, 20], 16
    c = filled(10, 8, 1, page, 64)
    table = tables(lens, page, 8)
    q = rand(17, 9, 4, 64).bfloat16()
    out = torch.full_like(q, 5.0)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ops.kv_attention(q, c, table, dev(lens), q_starts=dev([1, 3, 5]), max_q=2, out=out)
    want, _, _, mine = reference(q, c, table, lens, [1, 3, 5])
    assert (out[~mine] == 5).all() and mine.sum() == 4
    assert torch.equal(out[1:5], ops.kv_attention(q[1:5], c, table, dev(lens)))
    wild = ops.kv_attention(q, c, table, dev(lens), q_starts=dev([-100, 4, 1 << 30]), max_q=9)
    assert torch.equal(wild, ops.kv_attention(q, c, table, dev(lens), q_starts=dev([0, 4, 9]), max_q=9))
    # before the first sequence and behind the last: zeros in a fresh output
    fresh, lse = ops.kv_attention(q, c, table, dev(lens), q_starts=dev([1, 3, 5]), max_q=2, lse=True)
    assert torch.equal(fresh[1:5], out[1:5]) and (fresh[~mine] == 0).all() and (lse[~mine] == -math.inf).all()
    # queries beyond max_q are left out; the others keep their positions
    part = ops.kv_attention(q, c, table, dev(lens), q_starts=dev([0, 4, 9]), max_q=3)
    full = ops.kv_attention(q, c, table, dev(lens), q_starts=dev([0, 4, 9]), max_q=5)
    assert torch.equal(part[:3], full[:3]) and torch.equal(part[4:7], full[4:7]) and (part[3] == 0).all() and (part[7:] == 0).all()


def test_strided_queries_streams_and_graphs():
    lens, page = [500, 90], 16
    c = filled(11, 40, 2, page, 128)
    table = tables(lens, page, 40)
    dev_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    qkv = rand(18, 2, 12, 128).bfloat16()
    q = qkv[:, :8]
    want = ops.kv_attention(q.contiguous(), c, table, dev_lens)
    assert torch.equal(ops.kv_attention(q, c, table, dev_lens), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.kv_attention(q, c, table, dev_lens, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graphs, outs = [], []
    for _ in range(2):  # two captured calls, each with its own workspace, replayed at once
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(ops.kv_attention(q, c, table, dev_lens))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    dev_lens.copy_(torch.tensor([333, 12]))
    want = ops.kv_attention(q, c, table, dev_lens)
    torch.cuda.synchronize()
    for _ in range(20):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_no_queries_and_errors():
    c = filled(12, 4, 2, 16, 64)
    table = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    lens = torch.tensor([5, 6], dtype=torch.int32, device="cuda")
    assert ops.kv_attention(torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda"), c, table, lens).shape == (0, 4, 64)
    q = rand(1, 2, 4, 64).bfloat16()
    assert ops.kv_attention(q[:0], c, table[:0], lens[:0]).shape == (0, 4, 64)
    raw, st = c._raw(), torch.cuda.current_stream().cuda_stream
    out = torch.empty_like(q)
    call = lambda o, ws=None, n=0, keys=32, t=table, qq=q: ops.mxq_kv_attention(  # noqa: E731
        raw, qq.data_ptr(), 2, 256, 64, 4, 2, None, 1, lens.data_ptr(), keys, t.data_ptr(), t.shape[1], 1.0, 0, 0, o, None, ws, n, st)
    assert call(out.data_ptr()) == 0
    assert call(q.data_ptr()) == 1                       # out over q
    assert call(c.v_codes.data_ptr()) == 1               # out over the cache
    assert call(out.data_ptr() + 2) == 3
    wide = torch.zeros((2, 4096), dtype=torch.int32, device="cuda")
    assert call(out.data_ptr(), keys=65536, t=wide) == 1  # a workspace is needed
    torch.cuda.synchronize()


def test_decoding_as_it_is_used():
    """A prompt appended in one call and attended to, then tokens one at a time: each equals attention over the whole."""
    kv, heads, d, page, n = 2, 8, 128, 16, 70
    k, v, q = rand(1, n, kv, d).bfloat16(), rand(2, n, kv, d).bfloat16(), rand(3, n, heads, d).bfloat16()
    table = torch.tensor([[3, 0, 5, 1, 2]], dtype=torch.int32, device="cuda")
    pos = torch.arange(n, device="cuda")
    slots = table[0, pos // page].long() * page + pos % page
    whole = ops.KVCache.empty(6, kv, page, d)
    ops.kv_append(k, v, whole, slots)
    want = check(q, whole, table, [n], [0, n])
    c = ops.KVCache.empty(6, kv, page, d)
    ops.kv_append(k[:50], v[:50], c, slots[:50])
    ln = torch.tensor([50], dtype=torch.int32, device="cuda")
    outs = [ops.kv_attention(q[:50], c, table, ln)]
    for i in range(50, n):
        ops.kv_append(k[i:i + 1], v[i:i + 1], c, slots[i:i + 1])
        ln += 1
        outs.append(ops.kv_attention(q[i:i + 1], c, table, ln))
    got = torch.cat(outs).double()
    out, _, tol, _ = reference(q, c, table, [n], [0, n])
    assert ((got - out).abs() <= tol + out.abs() * 2.0 ** -8).all()
    assert all(torch.equal(a, b) for a, b in zip(state(c), state(whole)))
    assert want.shape == q.shape


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 200, 2 ** 31, 2 ** 32 + 100])
@pytest.mark.parametrize("lens,news,group", [([5], [8], 4), ([40], [43], 4), ([256], [260], 4), ([40], [43], 1), ([40, 3], [43, 6], 1),
                                             ([20, 200], [23, 2], 1), ([3, 2], [6, 6], 2), ([3000, 0, 6], [5, 2, 9], 1)])
def test_a_window_beyond_every_key_is_none(lens, news, group, window):
    """More queries than keys: the first ones stand before the first key, by up to their number."""
    page = 16
    c = filled(3, 256, 2, page, 64)
    table = tables(lens, page, 256)
    starts = [sum(news[:i]) for i in range(len(news) + 1)]
    q = rand(9, sum(news), 2 * group, 64).bfloat16()
    got = check(q, c, table, lens, starts, window=window)
    assert torch.equal(got, check(q, c, table, lens, starts))


@pytest.mark.parametrize("kv,group,batch,queries", [(2, 4, 1, 64), (8, 4, 1, 64), (3, 4, 3, 80), (2, 4, 1, 1), (2, 4, 3, 2), (1, 16, 1, 2)])
def test_a_workspace_serves_fewer_keys_and_narrower_tables(kv, group, batch, queries):
    """Asked for 2432 and for 6000 keys, used with fewer, and with a table that holds fewer."""
    page, d, width = 16, 64, 375
    c = filled(3, 40, kv, page, d)
    table = torch.randint(0, 40, (batch, width), generator=torch.Generator().manual_seed(1)).int().cuda()
    rows, heads = batch * queries, kv * group
    q = rand(1, rows, heads, d).bfloat16()
    lens = torch.full((batch,), 1 << 20, dtype=torch.int32, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    for asked in (2432, 6000):
        n = ops.mxq_kv_attention_workspace_bytes(c._raw(), batch, rows, queries, heads, asked)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        for keys, w in [(asked, width), (asked, asked // page - 8), (asked - 128, width), (asked, 57), (1000, width), (300, width), (128, width), (7, width)]:
            t = table[:, :w].contiguous()
            out = torch.empty_like(q)
            assert ops.mxq_kv_attention(c._raw(), q.data_ptr(), rows, heads * d, d, heads, batch, None, queries, lens.data_ptr(), keys,
                                        t.data_ptr(), w, d ** -0.5, 0, 0, out.data_ptr(), None, ws.data_ptr() if n else None, n, st) == 0
            assert torch.equal(out, ops.kv_attention(q, c, t, lens, max_keys=keys))


@pytest.mark.parametrize("heads,page,dim", [(0, 16, 64), (2, 0, 64), (2, 16, 0)])
def test_a_cache_without_heads_rows_or_dimensions_is_refused(heads, page, dim):
    with pytest.raises(ValueError, match="a cache needs"):
        ops.KVCache.empty(4, heads, page, dim)
    c = ops.KVCache.empty(0, 2, 16, 64)      # no pages: nothing to see
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    assert (ops.kv_attention(rand(1, 3, 4, 64).bfloat16(), c, i32(3, 2), i32(3) + 5) == 0).all()


def test_serving_results_carry_no_gradient():
    c = filled(3, 4, 2, 16, 64)
    table, lens = torch.arange(4, dtype=torch.int32, device="cuda")[None], torch.tensor([50], dtype=torch.int32, device="cuda")
    q = rand(1, 3, 4, 64).bfloat16().requires_grad_()
    out, lse = ops.kv_attention(q, c, table, lens, lse=True)
    assert not out.requires_grad and not lse.requires_grad and not ops.kv_attention(q, c, table, lens).requires_grad
    x, w = rand(1, 3, 64).bfloat16().requires_grad_(), mxq.quantize_mma(rand(2, 32, 64).bfloat16(), "mxfp8")
    assert not ops.linear(x, *w, "mxfp8").requires_grad and not ops.linear(x, *w, "mxfp8", check=True).requires_grad
    k = rand(3, 1, 2, 64).bfloat16().requires_grad_()
    ops.kv_append(k, k, c, torch.zeros(1, dtype=torch.int64, device="cuda"))


def test_ragged_single_tokens_without_max_q():
    """max_q left out: the kernel for many queries, the same result within both errors."""
    page, lens = 16, [130, 0, 64, 1, 700]
    c = filled(5, 60, 2, page, 64)
    table = tables(lens, page, 60)
    spoil_tails(c, table, lens)
    check(rand(7, 5, 8, 64).bfloat16(), c, table, lens, list(range(6)), max_q=None)
    check(rand(7, 5, 8, 64).bfloat16(), c, table, lens, list(range(6)), max_q=5)
    check(rand(7, 40, 8, 64).bfloat16(), c, table, lens, [8, 9, 9, 10, 11, 12], max_q=40)


HIDDEN = [  # (keys of each sequence, queries, group, head_dim, window, key counted from the last, page)
    ([90], [3], 4, 128, 0, 0, 16), ([90], [8], 4, 64, 0, 3, 16), ([700, 300], [5, 2], 1, 64, 0, 0, 32), ([3000], [8], 4, 128, 0, 5, 64),
    ([3000, 2000], [4, 4], 4, 128, 0, 2, 64), ([16], [16], 2, 128, 0, 9, 16), ([70], [70], 4, 128, 0, 60, 16), ([70], [70], 1, 64, 0, 0, 16),
    ([500], [100], 4, 128, 0, 40, 16), ([5000], [64], 4, 128, 0, 1, 64), ([5000], [40], 8, 64, 0, 30, 64), ([2000], [300], 1, 128, 0, 290, 32),
    ([90], [4], 4, 128, 20, 22, 16), ([3000, 900], [8, 8], 4, 64, 500, 506, 32), ([3000], [6], 1, 128, 1000, 1003, 32), ([300], [60], 4, 128, 30, 80, 16),
    ([3000], [64], 4, 128, 1000, 1040, 64), ([2000], [200], 1, 64, 150, 333, 32), ([40], [43], 2, 64, 0, 0, 16), ([200], [60], 2, 128, 3, 59, 16)]


@pytest.mark.parametrize("k_byte,v_byte", [(127, 0xFC), (0xFC, 127), (0xFC, 0xFC), (147, 147), (127, 240), (0xFF, 0xFF)])
@pytest.mark.parametrize("case", range(len(HIDDEN)))
def test_keys_that_some_queries_do_not_see(case, k_byte, v_byte):
    """A key with huge blocks that only some queries of a tile see: later ones in a causal chunk, earlier ones where a window
    leaves it behind. The others' results are those without it."""
    lens, news, group, d, window, back, page = HIDDEN[case]
    c = filled(3, sum(-(-n // page) for n in lens) + 1, 2, page, d)
    table = tables(lens, page, c.pages)
    spoil_tails(c, table, lens)
    starts = [sum(news[:i]) for i in range(len(news) + 1)]
    q = rand(9, sum(news), 2 * group, d).bfloat16()
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    call = lambda: ops.kv_attention(q, c, table, dev(lens), q_starts=dev(starts), max_q=max(news), window=window, lse=True)  # noqa: E731
    out, want_lse, tol, _ = reference(q, c, table, lens, starts, window)
    clean = call()
    blind = torch.ones(sum(news), dtype=torch.bool, device="cuda")   # queries that see none of the huge keys
    for b, (n, new) in enumerate(zip(lens, news)):
        key = n - 1 - back
        pos = n - new + torch.arange(new, device="cuda")
        blind[starts[b]:starts[b + 1]] = (key > pos) | ((key <= pos - window) if window else False)
        for t, x in ((c.k_codes, 0x77), (c.v_codes, 0x77), (c.k_scales, k_byte), (c.v_scales, v_byte)):
            t[int(table[b, key // page]), :, key % page] = x
    assert blind.any() and not blind.all()
    got, lse = call()
    assert ((got.double() - out).abs() <= tol + out.abs() * 2.0 ** -8)[blind].all()
    fin = torch.isfinite(want_lse) & blind[:, None]
    assert torch.equal(lse == -math.inf, want_lse == -math.inf) or k_byte != 127
    assert ((lse.double() - want_lse).abs()[fin] <= 2.0 ** -12 * (1 + want_lse.abs()[fin])).all()
    assert torch.equal(got, call()[0]) or not torch.isfinite(got).all()
    if k_byte == 127:    # the others: that key with the rest
        check(q, c, table, lens, starts, window=window)
    if k_byte == 0xFF:
        assert torch.isnan(got[~blind]).all()
    assert torch.isfinite(clean[0]).all()


@pytest.mark.parametrize("news,group,d", [(5, 4, 128), (1, 4, 64), (60, 4, 128), (90, 1, 64)])
@pytest.mark.parametrize("prefix", [0, 16, 37, 300])
def test_prefixes_of_zeros(prefix, news, group, d):
    """Keys and values of zeros in front, and in the middle of the new ones: scale bytes of 0 next to ordinary ones."""
    page, n = 16, prefix + news
    c = ops.KVCache.empty(25, 2, page, d)
    table = tables([n], page, 25)
    pos = torch.arange(n, device="cuda")
    k, v = rand(1, n, 2, d).bfloat16(), rand(2, n, 2, d).bfloat16()
    k[:prefix], v[:prefix] = 0, 0
    k[prefix + news // 2], v[prefix + news // 2] = 0, 0
    ops.kv_append(k, v, c, table[0, pos // page].long() * page + pos % page)
    check(rand(3, news, 2 * group, d).bfloat16(), c, table, [n], [0, news])
    check(rand(3, news, 2 * group, d).bfloat16(), c, table, [n], [0, news], window=20)


def test_tokens_written_beside_huge_ones():
    """Through kv_append: the chunk's last token holds the largest values of bf16, the first ones small values; a later chunk
    whose window has left the token behind."""
    page, n, d = 16, 80, 128
    for news in (6, 40):
        c = ops.KVCache.empty(12, 2, page, d)
        table, pos = tables([n], page, 12, width=12), torch.arange(n, device="cuda")
        k, v = rand(1, n, 2, d).bfloat16(), (rand(2, n, 2, d) * 1e-3).bfloat16()
        want_k, want_v = k.clone(), v.clone()
        v[-1] = torch.finfo(torch.bfloat16).max
        slots = table[0, pos // page].long() * page + pos % page
        ops.kv_append(want_k, want_v, c, slots)
        q = rand(3, news, 8, d).bfloat16()
        clean = check(q, c, table, [n], [0, news])
        ops.kv_append(k, v, c, slots)
        got = check(q, c, table, [n], [0, news])
        assert ((got[:-1] - clean[:-1]).abs() <= 2 * 2.0 ** -8 * clean[:-1].abs() + 1e-6).all()


@pytest.mark.parametrize("rows", [1, 2, 8, 60])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("k_exp,v_exp", [(0, -118), (0, -122), (0, 108), (-112, 0), (-120, -120), (100, 0)])
def test_blocks_at_the_ends_of_the_range(k_exp, v_exp, d, rows):
    """Scale bytes next to 0 and 254, the queries so large or small that the scores are ordinary. Below bf16's normal range a
    step is 2^-133; fp32's subnormals, 2^-149 apart, are below that. At the upper end the sums are bounded by fp32: 150 keys, weights
    of up to 2^8, values of 6 x 2^(108 + 2) at most, stay below 2^128 (with 2^124 they would not)."""
    lens, page = [150], 16
    c = filled(5, 10, 2, page, d, 2.0 ** k_exp, 2.0 ** v_exp)
    table = tables(lens, page, 10)
    q = (rand(11, rows, 8, d) * 2.0 ** min(-k_exp, 118)).bfloat16()
    scale = 2.0 ** (max(0, -k_exp - 118) - 3)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    got, lse = ops.kv_attention(q, c, table, dev(lens), q_starts=dev([0, rows]), max_q=rows, scale=scale, lse=True)
    out, want, tol, _ = reference(q, c, table, lens, [0, rows], scale=scale)
    err = (got.double() - out).abs()
    assert (err <= tol + out.abs() * 2.0 ** -8 + 2.0 ** -134).all(), float((err / out.abs()).max())
    assert ((lse.double() - want).abs() <= 2.0 ** -12 * (1 + want.abs())).all()
    assert got.float().abs().max() > 2.0 ** (v_exp - 6)
