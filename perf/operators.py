"""Operators of language models on the library's microscaled formats: what is measured, each in a plain form of
elementary torch operations and as the library's own call.

- product: activations rounded to MXFP4 or MXFP8 and multiplied with a weight that is held in that format (serving).
- linear: a training step of a linear layer whose three products run in microscaled formats; the input is kept as an
  8-bit checkpoint for the weight's gradient.
- swiglu: silu(gate) * up and its gradients, with gate and up kept as 8-bit checkpoints in between.
- cache: keys and values appended to a paged MXFP4 cache and read back.
- attention: queries over that cache (paged, causal, grouped heads, optionally a sliding window).

Blocks of 32 values share the scale 2^(floor(log2 amax) - emax); values round to nearest, ties to even, saturating.
"""
import math

import torch

own = False

EMAX = {"mxfp4": 2, "mxfp8": 8}
PAYLOAD = {"mxfp4": 16, "mxfp8": 32}  # bytes of 32 codes
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases --------------------------------------------------------------------------------------

def listed():
    return [
        # one token through a square projection: a decoding step, where latency counts
        dict(name="product 1 token", op="product", m=1, n=4096, k=4096, fmt="mxfp4"),
        # an odd batch of decoding sequences through an MLP's first projection
        dict(name="product 77 tokens mxfp8", op="product", m=77, n=9728, k=2560, fmt="mxfp8"),
        # a long prefill through the same projection
        dict(name="product 16384 tokens", op="product", m=16384, n=9728, k=2560, fmt="mxfp4"),
        # a short training batch that is no multiple of the block length, through a key projection
        dict(name="linear 333 tokens", op="linear", m=333, n=1024, k=2560, fmt="mxfp8"),
        # a full training batch, the forward product in 4 bits
        dict(name="linear 8192 tokens mxfp4", op="linear", m=8192, n=9728, k=2560, fmt="mxfp4"),
        # a few tokens in 32 bits: launches count
        dict(name="swiglu 37 rows f32", op="swiglu", m=37, n=2560, dtype="f32", packed=False),
        # a training batch, gate and up as the halves of one projection
        dict(name="swiglu 16384 rows", op="swiglu", m=16384, n=9728, dtype="bf16", packed=True),
        # one decoding step of a batch: a token for each of 61 sequences
        dict(name="cache 61 tokens", op="cache", m=61, kv=8, d=128, page=16),
        # the prompt of a long request
        dict(name="cache 16384 tokens", op="cache", m=16384, kv=8, d=128, page=64),
        # one sequence, one new token: few rows, so the keys are split
        dict(name="attention 1 sequence", op="attention", b=1, q=1, keys=4000, heads=32, kv=8, d=128, page=16, window=0),
        # a batch of long sequences of ragged lengths, one new token each
        dict(name="attention 16 sequences", op="attention", b=16, q=1, keys=32768, heads=32, kv=8, d=128, page=64, window=0),
        # a chunk of 128 queries over a long prefix
        dict(name="attention 128 queries", op="attention", b=1, q=128, keys=32768, heads=32, kv=8, d=128, page=32, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "product", "linear", "swiglu", "cache", "attention", "attention"])
    if op in ("product", "linear"):
        most = max(c["m"] * c["n"] * c["k"] for c in listed() if c["op"] == op)
        n, k = 32 * _log(rng, 1, 304), 32 * _log(rng, 1, 304)
        if op == "product":
            n = max(1, n - rng.choice([0, 0, 1, 5, 8]))
        m = _log(rng, 1, max(1, min(16384, most // (n * k))))
        return dict(op=op, m=m, n=n, k=k, fmt=rng.choice(["mxfp4", "mxfp8"]))
    if op == "swiglu":
        n, dtype = 32 * _log(rng, 1, 304), rng.choice(["bf16", "f32"])
        return dict(op=op, m=_log(rng, 1, 16384 if dtype == "bf16" else 8192), n=n, dtype=dtype, packed=rng.random() < 0.5)
    d, page = rng.choice([64, 128]), rng.choice([16, 32, 48, 64, 128])
    if op == "cache":
        return dict(op=op, m=_log(rng, 1, 16384), kv=rng.choice([1, 2, 4, 8]), d=d, page=page)
    kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8, 16])
    if kv * group > 32:
        group = 32 // kv
    q, b = rng.choice([1, 1, 1, 2, 5, _log(rng, 1, 128)]), _log(rng, 1, 64)
    most = min(32768, 16 * 32768 // b, 128 * 32768 * 32 // (b * q * kv * group))
    keys = _log(rng, 1, max(1, most))
    return dict(op=op, b=b, q=q, keys=keys, heads=kv * group, kv=kv, d=d, page=page, window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]))


def _lengths(case):
    """Keys and queries of each sequence (ragged: three quarters to all of the longest)."""
    b, keys, q = case["b"], case["keys"], case["q"]
    lens = [max(1, keys - keys * (37 * i % 64) // 256) for i in range(b)]
    news = [max(1, q - q * (29 * i % 64) // 256) for i in range(b)]
    return lens, news


def work(case):
    op = case["op"]
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        wide = PAYLOAD[case["fmt"]] + 1
        return {"bytes": 2 * m * k + n * k // 32 * wide + 2 * m * n, "flops": 2 * m * n * k}
    if op == "linear":  # x, w and the output's gradient in; the output and two gradients out
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 2 * (2 * m * k + 2 * n * k + 2 * m * n), "flops": 6 * m * n * k}
    if op == "swiglu":  # forward: two in, one out, two checkpoints out; backward: one and the checkpoints in, two out
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": case["m"] * case["n"] * (6 * size + 2 * 2 * 33 / 32), "flops": 20 * case["m"] * case["n"]}
    if op == "cache":  # bf16 in and bf16 out; 17 bytes for 32 values written and read
        v = 2 * case["m"] * case["kv"] * case["d"]
        return {"bytes": v * (4 + 2 * 17 / 32) + 8 * case["m"], "flops": 4 * v}
    lens, news = _lengths(case)
    w = case["window"]
    seen = [sum(min(max(0, L - n + i + 1), w or L) for i in range(n)) for L, n in zip(lens, news)]
    used = [min(L, w + n - 1) if w else L for L, n in zip(lens, news)]
    rows = sum(news) * case["heads"] * case["d"]
    return {"bytes": sum(used) * case["kv"] * case["d"] * 2 * 17 / 32 + 4 * rows, "flops": 4 * sum(seen) * case["heads"] * case["d"]}


# ---- microscaled values in plain operations ------------------------------------------------------

def _scale_exponents(x, fmt):
    """floor(log2 amax) - emax of each block of 32 along the last dimension (fp32 in, int32 out)."""
    amax = x.abs().unflatten(-1, (-1, 32)).amax(-1)
    e = torch.frexp(amax).exponent - 1 - EMAX[fmt]
    return torch.where(amax == 0, torch.full_like(e, -127), e).clamp(-127, 127)


def _round(x, fmt):
    """(values of the element format, scale exponents) of x, fp32, blocks along the last dimension."""
    es = _scale_exponents(x, fmt)
    y = torch.ldexp(x.unflatten(-1, (-1, 32)), -es[..., None])
    mag = y.abs()
    if fmt == "mxfp4":
        step = 0.5 + 0.5 * (mag >= 2).float() + (mag >= 4).float()
        mag = (torch.round(mag / step) * step).clamp(max=6.0)
    else:
        e = (torch.frexp(mag).exponent - 1).clamp(min=-6) - 3
        mag = torch.ldexp(torch.round(torch.ldexp(mag, -e)), e).clamp(max=448.0)
    return torch.copysign(mag, y), es


def _rounded(x, fmt):
    """The values that x, rounded to the format, stands for."""
    v, es = _round(x.float(), fmt)
    return torch.ldexp(v, es[..., None]).flatten(-2)


def _codes(x, fmt):
    """(packed codes, scale bytes) of x: uint8 [..., cols / 32 * payload] and [..., cols / 32]."""
    v, es = _round(x.float(), fmt)
    if fmt == "mxfp8":
        codes = v.to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)
    else:
        grid = torch.tensor(E2M1, device=x.device)
        c = torch.searchsorted(grid, v.abs().contiguous()).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
        c = c.flatten(-2)
        codes = c[..., 0::2] | (c[..., 1::2] << 4)
    return codes.contiguous(), (es + 127).to(torch.uint8)


def _values(codes, scales, fmt):
    """What packed codes and scale bytes stand for, in fp32."""
    if fmt == "mxfp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        grid = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
        v = grid[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    s = torch.where(scales == 255, torch.full_like(scales, 0, dtype=torch.float32) / 0.0, torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.int() - 127))
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def _tiled(scales):
    """Scale bytes [rows, blocks] in 128 x 4 tiles: row r, column c of a tile at byte (r % 32) * 16 + (r / 32) * 4 + c."""
    rows, kb = scales.shape
    p = torch.nn.functional.pad(scales, (0, -kb % 4, 0, -rows % 128))
    return p.view(p.shape[0] // 128, 4, 32, p.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untiled(tiled, rows, kb):
    r128, kb4 = -(-rows // 128), -(-kb // 4)
    return tiled.view(r128, kb4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(r128 * 128, kb4 * 4)[:rows, :kb]


# ---- inputs -------------------------------------------------------------------------------------

def _activations(g, m, k, dtype=torch.bfloat16):
    """Heavy-tailed activations with a few outlier channels."""
    x = torch.randn((m, k), generator=g, device="cuda")
    x = x / (0.4 + torch.rand((m, 1), generator=g, device="cuda"))
    x[:, torch.randint(k, (max(1, k // 512),), generator=g, device="cuda")] *= 30
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if op == "product":
        x = _activations(g, case["m"], case["k"])
        codes, scales = _codes((0.02 * rand(case["n"], case["k"])).bfloat16(), case["fmt"])
        return dict(case=case, x=x, w_codes=codes, w_scales=_tiled(scales))
    if op == "linear":
        x, w = _activations(g, case["m"], case["k"]), (0.02 * rand(case["n"], case["k"])).bfloat16()
        return dict(case=case, x=x.requires_grad_(), w=w.requires_grad_(), grad=(1e-3 * rand(case["m"], case["n"])).bfloat16())
    if op == "swiglu":
        m, n, dt = case["m"], case["n"], DTYPES[case["dtype"]]
        both = _activations(g, m, 2 * n, dt)
        ins = [both] if case["packed"] else [both[:, :n].contiguous(), both[:, n:].contiguous()]
        return dict(case=case, ins=[t.requires_grad_() for t in ins], grad=(1e-2 * rand(m, n)).to(dt))
    kv, d, page = case["kv"], case["d"], case["page"]
    if op == "cache":
        m = case["m"]
        pages = -(-m // page) + 2
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:m]
        shape = (pages, kv, page)
        cache = [torch.zeros((*shape, w), dtype=torch.uint8, device="cuda") for w in (d // 2, d // 32, d // 2, d // 32)]
        k, v = _activations(g, m, kv * d).view(m, kv, d), rand(m, kv, d).bfloat16()
        return dict(case=case, k=k, v=v, cache=cache, slots=slots)
    lens, news = _lengths(case)
    per = [-(-n // page) for n in lens]
    pages = sum(per) + 3
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((case["b"], max(per)), -1, dtype=torch.int32, device="cuda")
    for i, n in enumerate(per):
        table[i, :n] = order[sum(per[:i]):sum(per[:i + 1])]
    k, v = rand(pages, kv, page, d), rand(pages, kv, page, d)
    k[..., torch.randint(d, (3,), generator=g, device="cuda")] *= 6
    cache = [*_codes(k.bfloat16(), "mxfp4"), *_codes(v.bfloat16(), "mxfp4")]
    del k, v
    # what lies behind a sequence's last key is left over from other requests: any bytes
    for i, n in enumerate(lens):
        if n % page:
            for t in cache:
                junk = torch.randint(256, (kv, page - n % page, t.shape[-1]), generator=g, device="cuda", dtype=torch.uint8)
                t[table[i, per[i] - 1].long(), :, n % page:] = junk
    starts = torch.tensor([0] + news, device="cuda").cumsum(0).int()
    q = rand(sum(news), case["heads"], d).bfloat16()
    return dict(case=case, q=q, cache=cache, table=table, lens=torch.tensor(lens, device="cuda").int(), starts=starts, most=max(news))


# ---- one pass -----------------------------------------------------------------------------------

def _library():
    import block_scaled_microscaling_b200 as mx
    return mx


def run(state):
    return {"product": _product, "linear": _linear, "swiglu": _swiglu, "cache": _cache, "attention": _attention}[state["case"]["op"]](state)


def _product(s):
    case, fmt = s["case"], s["case"]["fmt"]
    if own:
        return _library().linear(s["x"], s["w_codes"], s["w_scales"], fmt)
    w = _values(s["w_codes"], _untiled(s["w_scales"], case["n"], case["k"] // 32), fmt)
    return (_rounded(s["x"], fmt) @ w.T).bfloat16()


def _along_rows(x, fmt):
    """x rounded with blocks of 32 rows of a column (the last block filled up with zeros)."""
    m = x.shape[0]
    return _rounded(torch.nn.functional.pad(x.float(), (0, 0, 0, -m % 32)).T.contiguous(), fmt).T[:m]


def _linear(s):
    fmt = s["case"]["fmt"]
    if own:
        y = _library().linear_ste(s["x"], s["w"], fmt)
        return (y.detach(), *torch.autograd.grad(y, (s["x"], s["w"]), s["grad"]))
    x, w, grad = s["x"].detach(), s["w"].detach(), s["grad"]
    y = _rounded(x, fmt) @ _rounded(w, fmt).T
    dx = _rounded(grad, "mxfp8") @ _along_rows(w, "mxfp8")
    dw = _along_rows(grad, "mxfp8").T @ _along_rows(x, "mxfp8")
    return y.bfloat16(), dx.bfloat16(), dw.bfloat16()


def _swiglu(s):
    ins, grad = s["ins"], s["grad"]
    if own:
        y = _library().swiglu(*ins)
        return (y.detach(), *torch.autograd.grad(y, ins, grad))
    both = torch.cat([t.detach() for t in ins], -1)
    gate, up = both.float().chunk(2, -1)
    y = (gate * torch.sigmoid(gate) * up).to(both.dtype)
    gate, up, dy = _rounded(gate, "mxfp8"), _rounded(up, "mxfp8"), grad.float()
    sig = torch.sigmoid(gate)
    dgate, dup = dy * up * sig * (1 + gate * (1 - sig)), dy * gate * sig
    if s["case"]["packed"]:
        return y, torch.cat([dgate, dup], -1).to(both.dtype)
    return y, dgate.to(both.dtype), dup.to(both.dtype)


def _cache(s):
    cache, slots = s["cache"], s["slots"]
    if own:
        mx = _library()
        c = mx.KVCache(*cache)
        mx.kv_append(s["k"], s["v"], c, slots)
        return mx.kv_read(c, slots)
    page = s["case"]["page"]
    at, off = slots // page, slots % page
    out = []
    for x, codes, scales in ((s["k"], *cache[:2]), (s["v"], *cache[2:])):
        c, e = _codes(x, "mxfp4")
        codes[at, :, off], scales[at, :, off] = c, e
        out.append(_values(codes[at, :, off], scales[at, :, off], "mxfp4").bfloat16())
    return tuple(out)


def _attention(s):
    case = s["case"]
    if own:
        mx = _library()
        return mx.kv_attention(s["q"], mx.KVCache(*s["cache"]), s["table"], s["lens"], q_starts=s["starts"], max_q=s["most"], window=case["window"])
    b, kv, d, page, n = case["b"], case["kv"], case["d"], case["page"], s["most"]
    group, dev = case["heads"] // kv, s["q"].device
    j = torch.arange(s["table"].shape[1] * page, device=dev)
    at = s["table"][:, j // page].clamp(min=0).long()                      # [b, keys]
    key, off = j < s["lens"][:, None], j % page
    kc, ks, vc, vs = (t[at, :, off.expand_as(at)].transpose(1, 2) for t in s["cache"])   # [b, kv, keys, ..]
    k = _values(kc, ks, "mxfp4")
    v = torch.where(key[:, None, :, None], _values(vc, vs, "mxfp4"), torch.zeros((), device=dev))
    i = torch.arange(n, device=dev)
    new = (s["starts"][1:] - s["starts"][:-1])[:, None]
    row = (s["starts"][:-1, None] + i).clamp(max=s["q"].shape[0] - 1).long()
    q = s["q"][row].float().view(b, n, kv, group, d).permute(0, 2, 3, 1, 4).reshape(b, kv, group * n, d)
    scores = (q @ k.transpose(-1, -2) / math.sqrt(d)).view(b, kv, group, n, -1)
    pos = s["lens"][:, None] - new + i                                      # [b, n]
    seen = key[:, None, :] & (j <= pos[..., None])
    if case["window"]:
        seen &= j > pos[..., None] - case["window"]
    scores = torch.where(seen[:, None, None], scores, torch.full((), -math.inf, device=dev))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = (p.view(b, kv, group * n, -1) @ v).view(b, kv, group, n, d) / torch.where(total == 0, torch.ones_like(total), total)
    o = o.permute(0, 3, 1, 2, 4).reshape(b, n, case["heads"], d)
    out = torch.zeros_like(s["q"])
    out[row[i < new]] = o[i < new].bfloat16()
    return out


# ---- the definitions in 64 bits -------------------------------------------------------------------

def _grid64(fmt, device):
    """Magnitudes of the element format in the order of their codes, from the fields of each code."""
    ebits, mbits, bias, n = (2, 1, 1, 8) if fmt == "mxfp4" else (4, 3, 7, 127)
    out = []
    for c in range(n):
        e, f = c >> mbits, (c & ((1 << mbits) - 1)) / (1 << mbits)
        out.append(math.ldexp(f, 1 - bias) if e == 0 else math.ldexp(1 + f, e - bias))
    return torch.tensor(out, dtype=torch.float64, device=device)


def _near64(x, fmt, dim):
    """x in 64 bits, each block of 32 along `dim` replaced by the nearest values of the format under its scale."""
    x = x.detach().double().movedim(dim, -1)
    n = x.shape[-1]
    if n % 32:
        x = torch.cat([x, x.new_zeros((*x.shape[:-1], 32 - n % 32))], -1)
    blocks = x.reshape(*x.shape[:-1], -1, 32)
    top = blocks.abs().max(-1, keepdim=True).values
    scale = torch.exp2((torch.floor(torch.log2(top.clamp(min=2.0 ** -140))) - EMAX[fmt]).clamp(-127, 127))
    # log2 is rounded: near a power of two floor may be one off
    span = 2.0 ** EMAX[fmt]
    scale = torch.where(top / scale >= 2 * span, scale * 2, torch.where((top > 0) & (top / scale < span), (scale / 2).clamp(min=2.0 ** -127), scale))
    grid = _grid64(fmt, x.device)
    mag = (blocks / scale).abs()
    hi = torch.searchsorted(grid, mag.contiguous()).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    below, above = mag - grid[lo], grid[hi] - mag
    code = torch.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)
    near = torch.copysign(grid[code], blocks) * scale
    return near.flatten(-2)[..., :n].movedim(-1, dim)


def _decode64(codes, scales, fmt):
    grid = _grid64(fmt, codes.device)
    if fmt == "mxfp4":
        c = torch.stack((codes % 16, codes // 16), -1).reshape(*codes.shape[:-1], -1).long()
        v = grid[c % 8] * (1 - 2 * (c // 8))
    else:
        c = codes.long()
        v = grid[(c % 128).clamp(max=126)] * (1 - 2 * (c // 128))
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "product":
        n, kb = case["n"], case["k"] // 32
        r, c = torch.meshgrid(torch.arange(n, device="cuda"), torch.arange(kb, device="cuda"), indexing="ij")
        at = (r // 128 * (-(-kb // 4)) + c // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + c % 4
        return _near64(s["x"], case["fmt"], 1) @ _decode64(s["w_codes"], s["w_scales"][at], case["fmt"]).T
    if op == "linear":
        x, w, g, fmt = s["x"], s["w"], s["grad"], case["fmt"]
        return (_near64(x, fmt, 1) @ _near64(w, fmt, 1).T, _near64(g, "mxfp8", 1) @ _near64(w, "mxfp8", 0),
                _near64(g, "mxfp8", 0).T @ _near64(x, "mxfp8", 0))
    if op == "swiglu":
        n = case["n"]
        gate, up = (s["ins"][0][:, :n], s["ins"][0][:, n:]) if case["packed"] else s["ins"]
        dy, g8, u8 = s["grad"].double(), _near64(gate, "mxfp8", 1), _near64(up, "mxfp8", 1)
        gate, up = gate.detach().double(), up.detach().double()
        y, e = gate * up / (1 + torch.exp(-gate)), 1 + torch.exp(-g8)
        dgate, dup = dy * u8 * (e + g8 * (e - 1)) / (e * e), dy * g8 / e
        return (y, torch.cat((dgate, dup), 1)) if case["packed"] else (y, dgate, dup)
    if op == "cache":
        return _near64(s["k"], "mxfp4", 2), _near64(s["v"], "mxfp4", 2)
    lens, news = _lengths(case)
    group, page, first, outs = case["heads"] // case["kv"], case["page"], 0, []
    for i, (length, new) in enumerate(zip(lens, news)):
        at = s["table"][i, :-(-length // page)].long()
        k, v = (_decode64(c[at], e[at], "mxfp4").transpose(0, 1).flatten(1, 2)[:, :length].repeat_interleave(group, 0)
                for c, e in (s["cache"][:2], s["cache"][2:]))
        q = s["q"][first:first + new].double().transpose(0, 1)              # [heads, new, d]
        far = torch.arange(length, device="cuda") - (length - new + torch.arange(new, device="cuda"))[:, None]
        hidden = (far > 0) | ((far <= -case["window"]) if case["window"] else (far > length))
        w = torch.softmax((q @ k.mT / math.sqrt(case["d"])).masked_fill(hidden, -math.inf), -1)
        outs.append(torch.nan_to_num(w @ v).transpose(0, 1))               # a query without a key gives zeros
        first += new
    return torch.cat(outs)
