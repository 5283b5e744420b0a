"""Cases of the decode-time operators on block-scaled weights and caches.

Three operators that one decode step of a transformer layer calls in turn:

* ``gemv``    y = x W^T with few rows x (bf16 / fp32) and 4-bit block-scaled W;
* ``append``  per-head RMS norm of queries and keys, position rotation, and the
              keys and values quantized into the rows of a paged cache;
* ``attend``  one query token per sequence against such a cache through a page
              table, optionally a sliding window with first tokens that stay
              visible.

``run`` computes each in its plain form (elementary torch operations in binary32)
or, where ``own`` is true, through the package's calls.
"""
import math

import torch

own = False

# element formats: signed grid of every code, scale format, block, rule
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
_E3M0 = [0.0] + [2.0 ** (c - 3) for c in range(1, 8)]
_E2M3 = [m / 8 for m in range(8)] + [2.0 ** (e - 1) * (1 + m / 8) for e in (1, 2, 3) for m in range(8)]
_E8M0 = [2.0 ** (c - 127) for c in range(255)] + [math.nan]
_UE4M3 = [m * 2.0 ** -9 for m in range(8)] + [2.0 ** (c // 8 - 7) * (1 + (c % 8) / 8) for c in range(8, 127)]
_UE4M3 += [math.nan] * (256 - len(_UE4M3))


def _signed(mag):
    return mag + [-v for v in mag]


# name: (grid over codes, emax, largest magnitude, scale format, block, asymmetric)
_FMT = {
    "mxfp4": (_signed(_E2M1), 2, 6.0, "e8m0", 32, False),
    "nvfp4": (_signed(_E2M1), 2, 6.0, "ue4m3", 16, False),
    "mxfp4_b128": (_signed(_E2M1), 2, 6.0, "e8m0", 128, False),
    "e3m0": (_signed(_E3M0), 4, 16.0, "e8m0", 32, False),
    "mxfp6": (_signed(_E2M3), 2, 7.5, "e8m0", 32, False),
    "int4": ([float(c if c < 8 else c - 16) for c in range(16)], 2, 7.0, "e8m0", 32, False),
    "int4a_g128": ([float(c) for c in range(16)], 3, 15.0, "e8m0", 128, True),
}
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_tables = {}


def _table(values, dtype, device):
    key = (tuple(values[:40]), len(values), dtype, device)
    if key not in _tables:
        _tables[key] = torch.tensor(values, dtype=dtype, device=device)
    return _tables[key]


def _scale_table(fmt, dtype, device):
    return _table(_E8M0 if _FMT[fmt][3] == "e8m0" else _UE4M3, dtype, device)


def _round_codes(fmt, v):
    """Nearest code of every element of v, ties to the even code, saturating."""
    grid, _, _, _, _, asym = _FMT[fmt]
    if fmt.startswith("int4"):
        r = torch.round(v)  # half to even
        return r.clamp(0, 15).to(torch.uint8) if asym else (r.clamp(-7, 7).to(torch.int16) & 15).to(torch.uint8)
    half = len(grid) // 2
    mids = _table([(a + b) / 2 for a, b in zip(grid[: half - 1], grid[1:half])], torch.float32, v.device)
    a = v.abs()
    lo = torch.bucketize(a, mids, right=False, out_int32=True)
    hi = torch.bucketize(a, mids, right=True, out_int32=True)
    c = torch.where(lo % 2 == 0, lo, hi)
    return (c + half * torch.signbit(v)).to(torch.uint8)


def _pack(fmt, codes):
    return codes if fmt == "mxfp6" else codes[..., 0::2] | (codes[..., 1::2] << 4)


def _unpack(fmt, packed):
    return packed if fmt == "mxfp6" else torch.stack([packed & 15, packed >> 4], -1).flatten(-2)


def _quantize(fmt, x, t_scale):
    """(codes, scale codes, offsets) of x [..., C] in blocks along C."""
    grid, emax, top, sfmt, block, asym = _FMT[fmt]
    b = x.float().unflatten(-1, (-1, block))
    off = None
    if asym:
        off = b.amin(-1).to(torch.bfloat16)
        b = b - off.float()[..., None]
    amax = b.abs().amax(-1)
    if sfmt == "e8m0":
        e = torch.frexp(amax)[1] - 1 - emax
        if asym:  # no overflow: the next exponent where the largest would not fit
            e = e + (amax > top * _scale_table(fmt, torch.float32, x.device)[(e + 127).clamp(0, 254).long()])
        e = torch.where(amax > 0, e, -127).clamp(-127, 127)
        sc = (e + 127).to(torch.uint8)
        inv = _table([2.0 ** (127 - c) for c in range(255)], torch.float32, x.device)[sc.long()]
    else:
        sc = (amax / top / t_scale).clamp(max=448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        inv = 1.0 / (_scale_table(fmt, torch.float32, x.device)[sc.long()] * t_scale)
    v = torch.where(torch.isfinite(inv)[..., None] & (amax > 0)[..., None], b * inv[..., None], 0.0)
    return _round_codes(fmt, v.flatten(-2)), sc, off


def _values(fmt, packed, scales, t_scale, off, dtype):
    """x_hat of packed codes and scale codes in blocks along the last axis."""
    grid, _, _, _, block, asym = _FMT[fmt]
    q = _table(grid, dtype, packed.device)[_unpack(fmt, packed).int()].unflatten(-1, (-1, block))
    q = q * _scale_table(fmt, dtype, packed.device)[scales.int()][..., None]
    if t_scale is not None:
        q = q * t_scale.to(dtype)
    if asym:
        q = q + off.to(dtype)[..., None]
    return q.flatten(-2)


def _chunk_index(rows, s, device):
    """Place of scale (r, j) in 512-byte chunks of 128 rows x 4 scales."""
    r, j = torch.arange(rows, device=device)[:, None], torch.arange(s, device=device)[None]
    return (r // 128 * (s // 4) + j // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + j % 4


def _case(name, **k):
    return dict(name=name, **k)


def listed():
    return [
        # the attention output projection of one token at batch 1: latency counts
        _case("gemv mxfp4 1x4096x4096", op="gemv", fmt="mxfp4", m=1, n=4096, k=4096, dtype="bf16", chunked=False),
        # the up projection of one token, weights in the GEMM operand's scale layout
        _case("gemv nvfp4 1x14336x4096", op="gemv", fmt="nvfp4", m=1, n=14336, k=4096, dtype="bf16", chunked=True),
        # the down projection of a few sequences decoded together, group scales with offsets
        _case("gemv int4a_g128 4x4096x14336", op="gemv", fmt="int4a_g128", m=4, n=4096, k=14336, dtype="bf16", chunked=False),
        # an output head with many rows, a batch of sixteen: the largest matrix
        _case("gemv mxfp4 16x65536x8192", op="gemv", fmt="mxfp4", m=16, n=65536, k=8192, dtype="bf16", chunked=False),
        # sizes that fit no tile, binary32 activations
        _case("gemv mxfp4 3x1000x1056 fp32", op="gemv", fmt="mxfp4", m=3, n=1000, k=1056, dtype="fp32", chunked=False),
        # the tokens of one decode step
        _case("append mxfp4 8 tokens", op="append", fmt="mxfp4", tokens=8, heads=32, kv=8, dim=128, rot=128, dtype="bf16",
              rows=256, norm=True, interleaved=False, far=131072),
        # a prompt's tokens at once
        _case("append nvfp4 8192 tokens", op="append", fmt="nvfp4", tokens=8192, heads=32, kv=8, dim=128, rot=128,
              dtype="bf16", rows=8192, norm=True, interleaved=False, far=8192),
        # a ragged chunk of a prompt, binary32, short heads rotated in part and in neighbouring pairs
        _case("append mxfp6 333 tokens fp32", op="append", fmt="mxfp6", tokens=333, heads=14, kv=2, dim=64, rot=32,
              dtype="fp32", rows=512, norm=True, interleaved=True, far=32768),
        # one sequence of ordinary length: latency counts
        _case("attend mxfp4 1 x 1000", op="attend", fmt="mxfp4", seqs=1, longest=1000, heads=32, kv=8, dim=128, page=16,
              window=0, sinks=0, dtype="bf16"),
        # a full decode batch of ragged lengths: the largest cache
        _case("attend mxfp4 64 x 8192", op="attend", fmt="mxfp4", seqs=64, longest=8192, heads=32, kv=8, dim=128, page=64,
              window=0, sinks=0, dtype="bf16"),
        # one long context, split over its length
        _case("attend nvfp4 1 x 131072", op="attend", fmt="nvfp4", seqs=1, longest=131072, heads=32, kv=8, dim=128, page=64,
              window=0, sinks=0, dtype="bf16"),
        # a sliding window with first tokens that stay, 6-bit cache, binary32 queries
        _case("attend mxfp6 window 16 x 4000", op="attend", fmt="mxfp6", seqs=16, longest=4000, heads=14, kv=2, dim=64, page=16,
              window=1000, sinks=4, dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemv", "append", "attend"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "gemv":
        fmt = rng.choice(["mxfp4", "nvfp4", "mxfp4_b128", "e3m0", "int4", "int4a_g128"])
        block = max(32, _FMT[fmt][4])
        k = block * max(1, _log(rng, 128, 16384) // block)
        n = min(_log(rng, 64, 32768), (1 << 28) // k)
        chunked = rng.random() < 0.3
        if chunked:
            k, n = k + -k % (4 * block), n + -n % 128
        return dict(op=op, fmt=fmt, m=_log(rng, 1, 16), n=n, k=k, dtype=dtype, chunked=chunked)
    fmt = rng.choice(["mxfp4", "nvfp4", "mxfp6", "int4"])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 4, 7, 8])
    dim = rng.choice([64, 128, 128, 256])
    if op == "append":
        tokens = _log(rng, 1, 4096)
        return dict(op=op, fmt=fmt, tokens=tokens, heads=heads, kv=kv, dim=dim, rot=rng.choice([dim, dim, dim // 2]), dtype=dtype,
                    rows=tokens + _log(rng, 1, 200), norm=rng.random() < 0.7, interleaved=rng.random() < 0.4,
                    far=_log(rng, 100, 131072))
    longest = _log(rng, 1, 65536)
    seqs = max(1, min(_log(rng, 1, 64), (1 << 27) // (longest * kv * dim)))
    window = rng.choice([0, 0, _log(rng, 1, longest)])
    return dict(op=op, fmt=fmt, seqs=seqs, longest=longest, heads=heads, kv=kv, dim=dim, page=rng.choice([16, 32, 64, 128]),
                window=window, sinks=rng.choice([0, 4]) if window else 0, dtype=dtype)


def _block(case):
    return _FMT[case["fmt"]][4]


def _t_scale(fmt, amax, device):
    return torch.tensor([amax / (6.0 * 448.0)], device=device) if _FMT[fmt][3] == "ue4m3" else None


def _cache(case, rows, gen, dev):
    """Codes and scales of rows x (kv * dim) keys and values as a run of a model leaves them."""
    s = {}
    for which, gain in (("k", 1.5), ("v", 1.0)):
        x = torch.randn(rows, case["kv"] * case["dim"], generator=gen, device=dev) * gain
        ts = _t_scale(case["fmt"], 8.0, dev)
        codes, sc, _ = _quantize(case["fmt"], x, ts)
        s[which + "_codes"], s[which + "_scales"], s[which + "_ts"] = _pack(case["fmt"], codes).contiguous(), sc.contiguous(), ts
    return s


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = _TYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "gemv":
        m, n, k, fmt = case["m"], case["n"], case["k"], case["fmt"]
        # activations: Laplace with a few columns fifty times as large
        u = torch.rand(m, k, generator=gen, device=dev) - 0.5
        x = -torch.sign(u) * torch.log1p(-2 * u.abs() * (1 - 1e-6))
        x[:, torch.randperm(k, generator=gen, device=dev)[: max(1, k // 1024)]] *= 50.0
        s["x"] = x.to(dt)
        s["ts"] = _t_scale(fmt, 0.12, dev)
        w = torch.randn(n, k, generator=gen, device=dev) * 0.02
        codes, sc, off = _quantize(fmt, w, s["ts"])
        s["codes"], s["off"] = _pack(fmt, codes).contiguous(), off
        if case["chunked"]:
            flat = torch.empty(sc.numel(), dtype=torch.uint8, device=dev)
            at = _chunk_index(n, k // _block(case), dev).flatten()
            flat[at] = sc.flatten()
            sc = flat  # offsets stay row-major
        s["scales"] = sc.contiguous()
        return s
    d, kv, heads = case["dim"], case["kv"], case["heads"]
    if case["op"] == "append":
        t = case["tokens"]
        # one fused projection's output: queries, keys and values side by side
        s["qkv"] = torch.randn(t, (heads + 2 * kv) * d, generator=gen, device=dev).to(dt)
        s["gq"] = 1 + 0.1 * torch.randn(d, generator=gen, device=dev) if case["norm"] else None
        s["gk"] = 1 + 0.1 * torch.randn(d, generator=gen, device=dev) if case["norm"] else None
        s["freq"] = torch.tensor([500000.0 ** (-2 * i / case["rot"]) for i in range(case["rot"] // 2)], device=dev)
        s["pos"] = torch.randint(0, case["far"], (t,), generator=gen, device=dev)
        s["slots"] = torch.randperm(case["rows"], generator=gen, device=dev)[:t].contiguous()
        if t > 100:  # padding tokens are not stored
            s["slots"][torch.randperm(t, generator=gen, device=dev)[: t // 100]] = -1
        s.update(_cache(case, case["rows"], gen, dev))
        return s
    per = -(-case["longest"] // case["page"])
    lengths = torch.randint(case["longest"] // 2, case["longest"] + 1, (case["seqs"],), generator=gen, device=dev)
    lengths[0] = case["longest"]
    if case["seqs"] > 4:
        lengths[3] = 0  # a free place of the batch
    s["lengths"] = lengths.int()
    pages = case["seqs"] * per + 3
    s["table"] = torch.randperm(pages, generator=gen, device=dev)[: case["seqs"] * per].reshape(case["seqs"], per).int()
    s["q"] = (torch.randn(case["seqs"], heads, d, generator=gen, device=dev) * 1.5).to(dt)
    s.update(_cache(case, pages * case["page"], gen, dev))
    return s


def _config(fmt, chunked=0, given=False):
    import microscaling_block_quantization_b200 as mx
    elem = {"e3m0": mx.E3M0, "mxfp6": mx.E2M3, "int4": mx.INT4, "int4a_g128": mx.INT4}.get(fmt, mx.E2M1)
    if _FMT[fmt][3] == "ue4m3":
        return mx.Config(elem=elem, block=_FMT[fmt][4], scale_fmt=mx.SCALE_UE4M3, rule=mx.RULE_NEAREST,
                         tensor_scale=mx.TS_GIVEN, sf_layout=int(chunked))
    return mx.Config(elem=elem, block=_FMT[fmt][4], asymmetric=int(_FMT[fmt][5]),
                     rule=mx.RULE_CEIL if _FMT[fmt][5] else mx.RULE_FLOOR, sf_layout=int(chunked))


def _handle(s):
    """The package's view of a state's weight or cache, made once as a program does when it loads them."""
    if "handle" not in s:
        import microscaling_block_quantization_b200 as mx
        case = s["case"]
        if case["op"] == "gemv":
            off = None if s["off"] is None else s["off"].view(torch.int16)
            s["handle"] = mx.Quantized(_config(case["fmt"], case["chunked"]), case["n"], case["k"], s["codes"], s["scales"],
                                       s["ts"], None, off, None)
        else:
            cfg, rows, cols = _config(case["fmt"]), s["k_codes"].shape[0], case["kv"] * case["dim"]
            page = case.get("page", 1)
            k, v = (mx.Quantized(cfg, rows, cols, s[w + "_codes"], s[w + "_scales"], s[w + "_ts"], None, None, None) for w in "kv")
            s["handle"] = mx.KVCache(cfg, rows // page, page, case["kv"], case["dim"], k, v)
    return s["handle"]


def _own(s):
    import microscaling_block_quantization_b200 as mx
    case, h = s["case"], _handle(s)
    if case["op"] == "gemv":
        return mx.gemv(s["x"], h)
    d, kv, heads = case["dim"], case["kv"], case["heads"]
    if case["op"] == "append":
        q, k, v = s["qkv"].split([heads * d, kv * d, kv * d], 1)
        q_out, k_out = mx.kv_append(h, q, k, v, s["slots"], s["pos"], q_gain=s["gq"], k_gain=s["gk"], eps=1e-6,
                                    inv_freq=s["freq"], interleaved=case["interleaved"], k_out=True)
        return q_out, k_out, mx.dequantize(h.k, torch.bfloat16), mx.dequantize(h.v, torch.bfloat16)
    return mx.attn_decode(h, s["q"], s["table"], s["lengths"], window=case["window"], sinks=case["sinks"], lse=True)


def _norm_rotate(case, x, gain, cos, sin):
    """Rows of heads [T, H, D] in binary32: RMS norm over D, then the rotation of the first `rot` entries."""
    if gain is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gain
    r = case["rot"]
    if case["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., : r // 2], x[..., r // 2: r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., r:]], -1)


def run(s):
    if own:
        return _own(s)
    case, fmt = s["case"], s["case"]["fmt"]
    dt = _TYPES[case["dtype"]]
    if case["op"] == "gemv":
        n, nb = case["n"], case["k"] // _block(case)
        sc, off = s["scales"], s["off"]
        if case["chunked"]:
            sc = sc[_chunk_index(n, nb, sc.device)]
        w = _values(fmt, s["codes"], sc, s["ts"], off, torch.float32)
        return (s["x"].float() @ w.T).to(dt)
    d, kv, heads = case["dim"], case["kv"], case["heads"]
    if case["op"] == "append":
        t = case["tokens"]
        q, k, v = s["qkv"].split([heads * d, kv * d, kv * d], 1)
        angle = s["pos"].double()[:, None, None] * s["freq"].double()
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
        q = _norm_rotate(case, q.float().unflatten(-1, (heads, d)), s["gq"], cos, sin).flatten(1).to(dt)
        k = _norm_rotate(case, k.float().unflatten(-1, (kv, d)), s["gk"], cos, sin).flatten(1).to(dt)
        keep = s["slots"] >= 0
        to = s["slots"][keep]
        for which, x in (("k", k), ("v", v)):
            codes, sc, _ = _quantize(fmt, x[keep], s[which + "_ts"])
            s[which + "_codes"][to] = _pack(fmt, codes)
            s[which + "_scales"][to] = sc
        return (q.view(t, heads, d), k.view(t, kv, d),
                *(_values(fmt, s[w + "_codes"], s[w + "_scales"], s[w + "_ts"], None, torch.float32).to(torch.bfloat16) for w in "kv"))
    b, page, table = case["seqs"], case["page"], s["table"]
    at = (table.long()[:, :, None] * page + torch.arange(page, device=table.device)).flatten(1)
    i = torch.arange(at.shape[1], device=at.device)[None]
    n = s["lengths"].long()[:, None]
    seen = i < n
    if case["window"]:
        seen &= (i >= n - case["window"]) | (i < case["sinks"])
    k, v = (_values(fmt, s[w + "_codes"][at], s[w + "_scales"][at], s[w + "_ts"], None, torch.float32).unflatten(-1, (kv, d))
            for w in "kv")
    q = s["q"].float().view(b, kv, heads // kv, d)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) / math.sqrt(d)
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.where(seen[:, None, None], torch.exp(score - top), 0.0)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, 1.0)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)
    return out.reshape(b, heads, d).to(dt), lse.reshape(b, heads)


def _row_bytes(case, cols):
    """Codes and scales of one row."""
    per = 1.0 if case["fmt"] == "mxfp6" else 0.5
    return cols * per + cols / _block(case) * (3 if _FMT[case["fmt"]][5] else 1)


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "gemv":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": n * _row_bytes(case, k) + m * (n + k) * size, "flops": 2.0 * m * n * k}
    cols, q = case["kv"] * case["dim"], case["heads"] * case["dim"]
    if case["op"] == "append":
        t, stored = case["tokens"], case["tokens"] - (case["tokens"] // 100 if case["tokens"] > 100 else 0)
        # the projection in; queries, keys and cache rows out; then the whole cache read back as values
        moved = t * (q + 2 * cols) * size + t * (q + cols) * size + 2 * stored * _row_bytes(case, cols)
        return {"bytes": moved + 2 * case["rows"] * (_row_bytes(case, cols) + 2 * cols), "flops": t * (q + cols) * 10.0}
    # lengths lie evenly between half of the longest and the longest
    mean = 0.75 * case["longest"]
    if case["window"]:
        mean = min(mean, case["window"] + case["sinks"])
    tokens = max(1.0, case["longest"] if case["seqs"] == 1 and not case["window"] else case["seqs"] * mean)
    return {"bytes": 2 * tokens * _row_bytes(case, cols) + 2 * case["seqs"] * q * size, "flops": 4.0 * tokens * q}


def exact(case, seed):
    """The operators' definitions in 64 bits on the inputs that prepare() makes."""
    s = prepare(case, seed)
    fmt, f64 = case["fmt"], torch.float64
    grid, _, top, sfmt, block, asym = _FMT[fmt]
    steps = torch.tensor(_E8M0 if sfmt == "e8m0" else _UE4M3, dtype=f64, device="cuda")
    points = torch.tensor(grid, dtype=f64, device="cuda")

    def decode(codes, scales, ts, off=None):
        c = codes.long()
        if fmt != "mxfp6":
            c = torch.cat([(c % 16)[..., None], (c // 16)[..., None]], -1).reshape(*c.shape[:-1], -1)
        x = points[c].reshape(*c.shape[:-1], -1, block) * steps[scales.long()].unsqueeze(-1)
        x = x if ts is None else x * ts.double()
        x = x if off is None else x + off.double().unsqueeze(-1)
        return x.reshape(*c.shape)

    if case["op"] == "gemv":
        n, nb = case["n"], case["k"] // block
        sc, off = s["scales"], s["off"]
        if case["chunked"]:
            # chunk (i, j) holds rows 128 i + 32 a + r and scales 4 j + b at place 16 r + 4 a + b
            sc = sc.view(n // 128, nb // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(n, nb)
        x = s["x"].double()
        part = [x @ decode(s["codes"][i:i + 8192], sc[i:i + 8192], s["ts"], None if off is None else off[i:i + 8192]).T
                for i in range(0, n, 8192)]
        return torch.cat(part, 1)
    d, kv, heads = case["dim"], case["kv"], case["heads"]
    if case["op"] == "append":
        dt = _TYPES[case["dtype"]]
        r = case["rot"]
        turn = torch.polar(torch.ones((), dtype=f64, device="cuda"), s["pos"].double()[:, None] * s["freq"].double())[:, None]

        def head(x, gain, h):
            x = x.double().reshape(-1, h, d)
            if gain is not None:
                x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / d + 1e-6) * gain.double()
            z = x[..., :r]
            z = torch.complex(*((z[..., 0::2], z[..., 1::2]) if case["interleaved"] else z.chunk(2, -1))) * turn
            z = torch.stack([z.real, z.imag], -1 if case["interleaved"] else -2).reshape(*x.shape[:2], r)
            return torch.cat([z, x[..., r:]], -1)

        qkv = s["qkv"]
        q = head(qkv[:, : heads * d], s["gq"], heads)
        k = head(qkv[:, heads * d: (heads + kv) * d], s["gk"], kv)
        to, out = s["slots"], []
        # the stored rows are the quantized roundings of k and v to the input's type
        for w, x in (("k", k.reshape(len(to), -1).to(dt)), ("v", qkv[:, (heads + kv) * d:])):
            kept = decode(s[w + "_codes"], s[w + "_scales"], s[w + "_ts"])
            b = x.double().reshape(len(to), -1, block)
            big = b.abs().amax(-1)
            if sfmt == "e8m0":
                step = torch.pow(2.0, torch.floor(torch.log2(big)) - _FMT[fmt][1])
                step = torch.where(2 ** torch.round(torch.log2(big)) == big, big / 2.0 ** _FMT[fmt][1], step)
                u = torch.where(step.unsqueeze(-1) > 0, b / step.unsqueeze(-1), 0.0)
            else:
                # the format is defined by its decisions in binary32: the scale is the E4M3 rounding of
                # (big / 6) / s_T, and an element is decided at x times the reciprocal of scale times s_T
                code = (big.float() / top / s[w + "_ts"]).clamp(max=448).to(torch.float8_e4m3fn)
                step = code.double() * s[w + "_ts"].double()
                u = (b.float() * (1 / (code.float() * s[w + "_ts"])).unsqueeze(-1)).double()
                u = torch.where(step.unsqueeze(-1) > 0, u, 0.0)
            if fmt == "int4":
                y = torch.round(u).clamp(-7, 7)
            else:
                # spacing of the grid around u: half to even on the multiples of it
                low, mant = 1.0, 3 if fmt == "mxfp6" else 1
                gap = torch.pow(2.0, torch.floor(torch.log2(u.abs().clamp(min=low))) - mant)
                y = (torch.round(u / gap) * gap).clamp(-top, top)
            y = (y * step.unsqueeze(-1)).reshape(len(to), -1)
            kept[to[to >= 0]] = y[to >= 0]
            out.append(kept)
        return q, k, out[0], out[1]
    outs, lses = [], []
    for b in range(case["seqs"]):
        n = int(s["lengths"][b])
        at = torch.arange(n, device="cuda")
        if case["window"]:
            at = at[(at < case["sinks"]) | (at >= n - case["window"])]
        rows = s["table"][b].long()[at // case["page"]] * case["page"] + at % case["page"]
        if not len(rows):
            outs.append(torch.zeros(heads, d, dtype=f64, device="cuda"))
            lses.append(torch.full((heads,), -math.inf, dtype=f64, device="cuda"))
            continue
        k, v = (decode(s[w + "_codes"][rows], s[w + "_scales"][rows], s[w + "_ts"]).view(-1, kv, d).repeat_interleave(heads // kv, 1)
                for w in "kv")
        a = torch.einsum("hd,lhd->hl", s["q"][b].double(), k) * d ** -0.5
        lses.append(torch.logsumexp(a, -1))
        outs.append(torch.einsum("hl,lhd->hd", torch.softmax(a, -1), v))
    return torch.stack(outs), torch.stack(lses)
