"""GPU parity of decode attention over a paged block-scaled cache.

The reference is binary64 on the dequantized cache.  Tolerances, with u = 2^-24:
a score is a sum of D products in binary32, |error| <= (D / 16 + 16) 2 u |scale| sum |q k| =: e
(the matrix instruction may truncate), so each weight is off by a factor
within exp(2 e) (its own score and the normaliser's), plus the exponential's
2 ulp and, for the sum over n tokens in tiles of 16, (n / 16 + 64) 2 u.  A weight
is rounded to 11 bits (half a step 2^-12) for bf16 results; for binary32 its
remainder is kept (2^-23).  Against sum p |v| that is
  tol = sum p |v| (2 e + (n / 16 + 64) 2 u + w) + half a step of the result,
w = 2^-12 or 2^-23, plus the flush of weights below 2^-32 of the largest: n 2^-32 max |v|."""
import dataclasses
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    from microscaling_block_quantization_b200 import build
    build.build()
    import microscaling_block_quantization_b200 as m
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return m


def configs(mx):
    nv = mx.Config(block=16, scale_fmt=mx.SCALE_UE4M3, rule=mx.RULE_NEAREST, tensor_scale=mx.TS_GIVEN)
    return {
        "mxfp4": mx.MXFP4,
        "mxfp4_b16": mx.Config(block=16),
        "mxfp4_b64": mx.Config(block=64),
        "nvfp4": nv,
        "ue5m3_b32": dataclasses.replace(nv, block=32, scale_fmt=mx.SCALE_UE5M3),
        "e2m3": mx.Config(elem=mx.E2M3),
        "e2m3_b16": mx.Config(elem=mx.E2M3, block=16),
        "e3m2": mx.Config(elem=mx.E3M2),
        "e3m2_b64": mx.Config(elem=mx.E3M2, block=64),
        "e3m0": mx.Config(elem=mx.E3M0),
        "e3m0_b16": mx.Config(elem=mx.E3M0, block=16),
        "int4": mx.Config(elem=mx.INT4, rule=mx.RULE_CEIL),
        "int4_b16": mx.Config(elem=mx.INT4, rule=mx.RULE_CEIL, block=16),
    }


NAMES = ["mxfp4", "mxfp4_b16", "mxfp4_b64", "nvfp4", "ue5m3_b32", "e2m3", "e2m3_b16", "e3m2", "e3m2_b64", "e3m0", "e3m0_b16", "int4", "int4_b16"]


def make(mx, cfg, lengths, Hq, H, D, page, dtype, seed=0, extra=3, vgain=1.0, qgain=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    per = max(1, -(-max(lengths + [1]) // page))
    pages = len(lengths) * per + extra
    ts = dict(k_tensor_scale=torch.tensor([0.003], device="cuda"), v_tensor_scale=torch.tensor([0.002], device="cuda")) if cfg.tensor_scale else {}
    c = mx.kv_cache(pages, page, H, D, cfg, **ts)
    for t, gain in ((c.k, 1.0), (c.v, vgain)):
        x = torch.randn(pages * page, H * D, generator=g, device="cuda") * gain
        q = mx.quantize(x.bfloat16(), cfg, stats=False, tensor_scale=t.tensor_scale)
        t.codes.copy_(q.codes)
        t.scales.copy_(q.scales)
    table = torch.randperm(pages, generator=g, device="cuda")[:len(lengths) * per].reshape(len(lengths), per).int()
    q = (torch.randn(len(lengths), Hq, D, generator=g, device="cuda") * qgain).to(dtype)
    return c, q, table, torch.tensor(lengths, dtype=torch.int32, device="cuda")


def visible(n, window, sinks):
    t = torch.arange(n, device="cuda")
    return t if not window else t[(t < sinks) | (t >= n - window)]


def check(mx, c, q, table, lengths, out, lse, scale=None, window=0, sinks=0):
    D, H, page = c.head_dim, c.kv_heads, c.page_size
    scale = D ** -0.5 if scale is None else scale
    k, v = (mx.dequantize(t).view(-1, H, D) for t in (c.k, c.v))
    G = q.shape[1] // H
    wide = q.dtype == torch.float32 or out.dtype == torch.float32
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    for b in range(q.shape[0]):
        n = max(0, min(int(lengths[b]), table.shape[1] * page))
        t = visible(n, window, sinks)
        pg = table[b].long()[t // page]
        ok = (pg >= 0) & (pg < c.pages)
        rows = (pg * page + t % page)[ok]
        o, ls = out[b].double().view(H * G, D), lse[b].double()
        if not len(rows):
            assert bool((o == 0).all()) and bool((ls == -math.inf).all())
            continue
        kb, vb = (x[rows].double().repeat_interleave(G, 1) for x in (k, v))
        qb = q[b].double()
        s = torch.einsum("hd,lhd->hl", qb, kb) * scale
        e = (torch.einsum("hd,lhd->hl", qb.abs(), kb.abs()) * abs(scale)).amax(1) * (D / 16 + 16) * 2.0 ** -23
        p = torch.softmax(s, 1)
        ref = torch.einsum("hl,lhd->hd", p, vb)
        mag = torch.einsum("hl,lhd->hd", p, vb.abs())
        L = len(rows)
        w = (2 * e + (L / 16 + 64) * 2.0 ** -23 + (2.0 ** -23 if wide else 2.0 ** -12))[:, None]
        tol = mag * w + L * 2.0 ** -32 * vb.abs().amax() + 1e-38
        err = (o - ref).abs()
        assert bool((err <= tol + (ref.abs() + tol) * half).all()), (b, float((err / (tol + ref.abs() * half)).max()))
        want = torch.logsumexp(s, 1)
        assert bool(((ls - want).abs() <= e + (L / 16 + 64) * 2.0 ** -23 + want.abs() * 2.0 ** -22).all())


def run(mx, args, **k):
    out, lse = mx.attn_decode(*args, lse=True, **k)
    check(mx, *args, out, lse, **{n: k[n] for n in ("scale", "window", "sinks") if n in k})
    return out, lse


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("name", NAMES)
def test_cache_formats(mx, name, D, dtype):
    run(mx, make(mx, configs(mx)[name], [100, 37], 8, 2, D, 16, dtype, qgain=1.5))


@pytest.mark.parametrize("name,D", [("mxfp4_b128", 128), ("mxfp4_b128", 256), ("mxfp4_b64", 64)])
def test_long_blocks(mx, name, D):
    cfg = mx.Config(block=128) if name == "mxfp4_b128" else configs(mx)[name]
    run(mx, make(mx, cfg, [77, 1, 130], 3, 3, D, 7, torch.bfloat16))


@pytest.mark.parametrize("Hq,H", [(1, 1), (8, 8), (5, 5), (7, 1), (14, 2), (32, 8), (16, 2), (9, 1), (20, 1), (64, 2), (48, 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_head_groups(mx, Hq, H, dtype):
    run(mx, make(mx, mx.MXFP4, [50, 333], Hq, H, 64, 16, dtype))


@pytest.mark.parametrize("page", [1, 3, 16, 17, 64, 100, 1000])
def test_lengths_and_pages(mx, page):
    """Lengths around tile and page borders, empty and one-token sequences; pages that end inside a tile."""
    run(mx, make(mx, mx.MXFP4, [0, 1, 2, 15, 16, 17, 31, 32, 33, 100, 257, 0, 640], 4, 2, 64, page, torch.bfloat16))


@pytest.mark.parametrize("seqs,n", [(1, 130), (1, 300), (2, 700), (1, 2000), (1, 3000), (1, 40000), (3, 9000), (40, 700), (100, 900)])
@pytest.mark.parametrize("name", ["mxfp4", "nvfp4"])
def test_split_sequences(mx, name, seqs, n):
    lengths = [n - 37 * i * (n // 200) // 8 for i in range(seqs)]
    run(mx, make(mx, configs(mx)[name], lengths, 8, 2, 128, 64, torch.bfloat16, qgain=2.0))
    run(mx, make(mx, configs(mx)[name], lengths, 8, 2, 128, 64, torch.float32, qgain=2.0))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name,D", [("e2m3", 256), ("e3m2", 128), ("mxfp4", 256), ("int4", 64), ("nvfp4", 256)])
def test_many_sequences_joined_in_a_cta(mx, name, D, dtype):
    """A CTA's warps share a sequence, as many as their rings leave room for; fewer tiles than warps too."""
    for seqs, n in ((40, 900), (40, 20), (90, 250)):
        args = make(mx, configs(mx)[name], [n] * (seqs - 2) + [0, 7], 12, 2, D, 32, dtype)
        run(mx, args)
        run(mx, args[:3] + (args[3].clamp(max=33),))


@pytest.mark.parametrize("Hq,H,name", [(4, 1, "mxfp4"), (14, 2, "nvfp4"), (9, 1, "e2m3")])
def test_ragged_batches(mx, Hq, H, name):
    """Long, short and empty sequences of one batch; batches shorter than the table allows."""
    for dtype in (torch.bfloat16, torch.float32):
        for lengths in ([9000, 0, 1, 16, 8000, 17, 0, 0, 5000, 33], [0, 0, 6000], [6000, 0, 0], [1] * 40 + [9000] + [100] * 40,
                        [40000, 3], [700, 2900] * 20):
            c, q, table, ls = make(mx, configs(mx)[name], lengths, Hq, H, 64, 64, dtype)
            run(mx, (c, q, table, ls))
            run(mx, (c, q, table, ls), window=300, sinks=5)
            run(mx, (c, q, table, ls.clamp(max=20)))     # fewer tiles than splits
            run(mx, (c, q, table, ls * 0))
            out = mx.attn_decode(c, q, table, ls)
            for b in (0, len(lengths) - 1):              # as each sequence by itself, but for the order of the sums
                one = mx.attn_decode(c, q[b:b + 1], table[b:b + 1], ls[b:b + 1])
                assert bool((out[b] - one[0]).abs().max() <= 0.02 * one.abs().max())


@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (100, 1), (50, 1000), (1000, 4), (7, 0), (33, 17)])
def test_window_and_sinks(mx, window, sinks):
    run(mx, make(mx, mx.MXFP4, [0, 1, 5, 40, 116, 117, 500, 2000], 4, 2, 64, 16, torch.float32), window=window, sinks=sinks)


def test_table_entries_outside_the_cache(mx):
    """The tokens of a bad entry are not visible; lengths beyond the table and below zero are clamped."""
    c, q, table, lengths = make(mx, mx.MXFP4, [60, 60, 60, 60], 2, 1, 64, 16, torch.bfloat16)
    table[0, 1], table[1, 0], table[2] = -1, c.pages, 2 ** 31 - 1
    lengths[3] = 10 ** 6
    run(mx, (c, q, table, lengths))
    lengths[:] = -5
    run(mx, (c, q, table, lengths))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_large_and_drifting_values(mx, dtype):
    """A running maximum and value scales that grow along the sequence, by far more than either margin; huge and tiny values."""
    for D, name in ((64, "mxfp4"), (128, "mxfp4"), (128, "mxfp4_b16"), (64, "e3m2"), (256, "e2m3")):
        c, q, table, lengths = make(mx, configs(mx)[name], [600, 300], 8, 2, D, 16, dtype, extra=0)
        rows = c.pages * c.page_size
        order = torch.empty(rows, device="cuda")
        for b in range(2):
            t = torch.arange(table.shape[1] * 16, device="cuda")
            order[table[b].long()[t // 16] * 16 + t % 16] = t.float()
        g = torch.Generator(device="cuda").manual_seed(5)
        x = torch.randn(rows, 2 * D, generator=g, device="cuda")
        for up in (1.0, -1.0):
            for t, gain in ((c.k, torch.exp2(up * order / 200)), (c.v, torch.exp2(up * order / 15))):
                z = mx.quantize((x * gain[:, None]).bfloat16(), c.cfg, stats=False)
                t.codes.copy_(z.codes)
                t.scales.copy_(z.scales)
            run(mx, (c, q, table, lengths))
        for gain in (2.0 ** 60, 2.0 ** -60):
            z = mx.quantize((x * gain).bfloat16(), c.cfg, stats=False)
            c.v.codes.copy_(z.codes)
            c.v.scales.copy_(z.scales)
            run(mx, (c, q, table, lengths))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("name", ["mxfp4", "mxfp4_b16", "mxfp4_b64", "e2m3", "int4"])
def test_values_near_the_ends_of_the_range(mx, name, dtype):
    """Values near the largest and the smallest binary32 numbers, in one stretch and in many: sums of them are not formed."""
    for seqs, n in ((20, 40), (20, 100), (1, 5000)):
        c, q, table, lengths = make(mx, configs(mx)[name], [n] * seqs, 4, 2, 128, 16, dtype)
        x = torch.randn(c.pages * c.page_size, 256, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
        for gain in (2.0 ** 122, 2.0 ** -118):
            z = mx.quantize((x * gain).bfloat16(), c.cfg, stats=False)
            c.v.codes.copy_(z.codes)
            c.v.scales.copy_(z.scales)
            run(mx, (c, q, table, lengths))


def test_scales_differ_between_blocks(mx):
    """One block of the head far larger than the others: the small ones keep their relative accuracy."""
    c, q, table, lengths = make(mx, mx.MXFP4, [200], 4, 1, 128, 16, torch.float32)
    x = torch.randn(c.pages * 16, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    x[:, :32] *= 2.0 ** 30
    z = mx.quantize(x.bfloat16(), c.cfg, stats=False)
    c.v.codes.copy_(z.codes)
    c.v.scales.copy_(z.scales)
    out, lse = mx.attn_decode(c, q, table, lengths, lse=True)
    k, v = (mx.dequantize(t).double() for t in (c.k, c.v))
    rows = table[0].long().repeat_interleave(16)[:200] * 16 + torch.arange(200, device="cuda") % 16
    p = torch.softmax(q[0].double() @ k[rows].T / math.sqrt(128), 1)
    ref, mag = p @ v[rows], p @ v[rows].abs()
    assert bool(((out[0].double() - ref).abs() <= mag * 2.0 ** -17).all())


def test_not_a_number_in_the_cache(mx):
    """NaN scales reach the result only where their token is visible."""
    c, q, table, lengths = make(mx, mx.MXFP4, [40, 40, 40], 4, 2, 64, 16, torch.bfloat16)
    rows = lambda b, t: int(table[b, t // 16]) * 16 + t % 16  # noqa: E731
    ks, vs = c.k.scales.view(-1, 2, 2), c.v.scales.view(-1, 2, 2)
    ks[rows(0, 45)], vs[rows(0, 40)] = 255, 255              # behind the end
    vs[rows(1, 39), 1, 0] = 255                              # one block of one head's last value
    ks[rows(2, 3), 0] = 255
    out, lse = mx.attn_decode(c, q, table, lengths, lse=True)
    nan = torch.isnan(out)
    assert not bool(nan[0].any())
    assert bool(nan[1, 2:, :32].all()) and int(nan[1].sum()) == 2 * 32
    assert bool(nan[2, :2].all()) and int(nan[2].sum()) == 2 * 64 and bool(torch.isnan(lse[2, :2]).all())
    check(mx, c, q[:1], table[:1], lengths[:1], out[:1], lse[:1])


def test_strides_outputs_and_types(mx):
    c, q, table, lengths = make(mx, mx.MXFP4, [90, 500], 6, 2, 64, 16, torch.bfloat16)
    want, _ = run(mx, (c, q, table, lengths))
    buf = torch.empty(2, 6 * 64 + 11, dtype=torch.bfloat16, device="cuda")
    buf[:, 5:389] = q.flatten(1)
    wide = torch.full((2, table.shape[1] + 3), -7, dtype=torch.int32, device="cuda")
    wide[:, 1:1 + table.shape[1]] = table
    out = torch.full((2, 400), 7.0, dtype=torch.bfloat16, device="cuda")
    got = mx.attn_decode(c, buf[:, 5:389], wide[:, 1:1 + table.shape[1]], lengths, out=out[:, 3:387])
    assert torch.equal(got, want.flatten(1)) and bool((out[:, 387:] == 7).all()) and bool((out[:, :3] == 7).all())
    o32, l32 = mx.attn_decode(c, q, table, lengths, out_dtype=torch.float32, lse=True)
    check(mx, c, q, table, lengths, o32, l32)
    run(mx, (c, q, table, lengths), scale=0.0)
    run(mx, (c, q, table, lengths), scale=-0.3)
    run(mx, (c, q, table, lengths), scale=2.0)


def test_repeatable_graphs_and_streams(mx):
    args = make(mx, mx.MXFP4, [5000, 100, 0, 3000], 8, 2, 128, 64, torch.bfloat16)
    want = mx.attn_decode(*args)
    assert all(torch.equal(mx.attn_decode(*args), want) for _ in range(3))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [mx.attn_decode(*args, stream=s) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graphs = []
    for _ in range(2):                                       # two graphs, replayed at the same time
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, mx.attn_decode(*args)))
    for _ in range(3):
        for (g, o), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for _, o in graphs)
    c, q, table, lengths = args                              # new lengths in a captured call
    lengths.copy_(torch.tensor([17, 4000, 1, 0], dtype=torch.int32))
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], mx.attn_decode(*args))


def test_cache_past_32_bit_offsets(mx):
    pages, page = (1 << 16) + 1, 64                          # times 1024 elements: more than 2^32
    c = mx.kv_cache(pages, page, 8, 128, mx.Config(elem=mx.E2M3))
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device="cuda")
    x = torch.randn(192, 1024, device="cuda").bfloat16()
    small = mx.kv_cache(3, page, 8, 128, c.cfg)
    z = mx.quantize(x, c.cfg, stats=False)
    for t, s in ((c.k, small.k), (c.v, small.v)):
        s.codes.copy_(z.codes)
        s.scales.copy_(z.scales)
        for i, pg in enumerate(table[0].tolist()):
            t.codes.view(pages, -1)[pg] = z.codes.view(3, -1)[i]
            t.scales.view(pages, -1)[pg] = z.scales.view(3, -1)[i]
    q = torch.randn(1, 16, 128, device="cuda").bfloat16()
    n = torch.tensor([170], dtype=torch.int32, device="cuda")
    assert torch.equal(mx.attn_decode(c, q, table, n), mx.attn_decode(small, q, torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda"), n))


def test_no_sequences_and_no_pages(mx):
    c, q, table, lengths = make(mx, mx.MXFP4, [5], 2, 1, 64, 16, torch.bfloat16)
    assert mx.attn_decode(c, q[:0], table[:0], lengths[:0]).shape == (0, 2, 64)
    out, lse = mx.attn_decode(c, q, table[:, :0], lengths, lse=True)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_refusals_of_the_binding(mx):
    c, q, table, lengths = make(mx, mx.MXFP4, [50, 70], 4, 2, 64, 16, torch.bfloat16)
    good = dict(q=q, page_table=table, lengths=lengths)
    call = lambda **k: mx.attn_decode(c, **{**good, **k})  # noqa: E731
    for k in (dict(q=q.cpu()), dict(q=q[..., :32]), dict(q=q[0]), dict(page_table=table.long()), dict(page_table=table[:1]),
              dict(page_table=table.cpu()), dict(page_table=table.T.contiguous().T), dict(lengths=lengths.long()), dict(lengths=lengths[:1]),
              dict(out=torch.zeros(1, 4, 64, device="cuda")), dict(out=torch.zeros(2, 4, 64)), dict(workspace=torch.zeros(9, device="cuda")),
              dict(out=torch.zeros(2, 4, 64, device="cuda"), out_dtype=torch.bfloat16), dict(window=1 << 40)):
        with pytest.raises(ValueError):
            call(**k)
    for k in (dict(q=q.half()), dict(scale="x"), dict(out_dtype=torch.float16), dict(lengths=None), dict(window=1.5)):
        with pytest.raises(TypeError):
            call(**k)
    for k in (dict(window=-1), dict(sinks=-1), dict(scale=math.inf), dict(q=torch.zeros(2, 3, 64, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(mx.MXError) as e:
            call(**k)
        assert e.value.code == -1
    c, q, table, lengths = make(mx, mx.MXFP4, [9000], 4, 2, 64, 16, torch.bfloat16)
    with pytest.raises(mx.MXError) as e:
        mx.attn_decode(c, q, table, lengths, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    assert e.value.code == -5
    n = mx.lib().mx_attn_workspace_bytes(c.ref(), 1, 4, table.shape[1], 0, 0)
    own = torch.full((n,), 255, dtype=torch.uint8, device="cuda")         # any contents
    assert torch.equal(mx.attn_decode(c, q, table, lengths, workspace=own), mx.attn_decode(c, q, table, lengths))
