"""GPU parity of mx_kv_append: norm, rotation and quantized store of new tokens.

The rotated heads are checked against binary64.  Error of an output
a cos - b sin: the norm's factor carries the sum of squares (8 multiply-adds a
lane and up to 5 shuffle additions, 13 roundings, halved by the root), its
mean, eps, a root good to 2 ulp (4 half steps) and two products: 14 half steps of
binary32; cosine and sine 2 ulp each plus the fraction's rounding (pi half
steps), below 8; the products and the sum 3.  |error| <= 25 2^-24 (|a| + |b|), then
the output's rounding.  The cache rows are checked bit for bit against
mx_quantize of the rounded keys and of the values."""
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
        "mxfp4_oas": mx.Config(rule=mx.RULE_OAS),
        "mxfp4_ceil_b64": mx.Config(rule=mx.RULE_CEIL, block=64),
        "mxfp4_round_up": mx.Config(round=mx.ROUND_CEIL),
        "nvfp4": nv,
        "nvfp4_unscaled": dataclasses.replace(nv, tensor_scale=mx.TS_NONE),
        "ue5m3_b128": dataclasses.replace(nv, block=128, scale_fmt=mx.SCALE_UE5M3),
        "pow2_ue4m3": mx.Config(block=16, scale_fmt=mx.SCALE_UE4M3),
        "e2m3": mx.Config(elem=mx.E2M3),
        "e3m2_b16": mx.Config(elem=mx.E3M2, block=16),
        "e2m3_nearest": mx.Config(elem=mx.E2M3, block=32, scale_fmt=mx.SCALE_UE4M3, rule=mx.RULE_NEAREST),
        "e3m2_round_up": mx.Config(elem=mx.E3M2, round=mx.ROUND_CEIL),
        "e3m0": mx.Config(elem=mx.E3M0),
        "int4": mx.Config(elem=mx.INT4, rule=mx.RULE_CEIL),
    }


NAMES = ["mxfp4", "mxfp4_oas", "mxfp4_ceil_b64", "mxfp4_round_up", "nvfp4", "nvfp4_unscaled", "ue5m3_b128", "pow2_ue4m3", "e2m3",
         "e3m2_b16", "e2m3_nearest", "e3m2_round_up", "e3m0", "int4"]


def inputs(T, Hq, H, D, dtype, rot, seed=0, rows=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    qkv = torch.randn(T, (Hq + 2 * H) * D, generator=g, device="cuda").to(dtype)
    rows = rows or T + 7
    return dict(qkv=qkv, q=qkv[:, :Hq * D], k=qkv[:, Hq * D:(Hq + H) * D], v=qkv[:, (Hq + H) * D:],
                slots=torch.randperm(rows, generator=g, device="cuda")[:T].contiguous(),
                positions=torch.randint(0, 200000, (T,), generator=g, device="cuda"),
                q_gain=1 + 0.2 * torch.randn(D, generator=g, device="cuda"), k_gain=1 + 0.2 * torch.randn(D, generator=g, device="cuda"),
                inv_freq=torch.tensor([10000.0 ** (-2 * i / rot) for i in range(rot // 2)], device="cuda") if rot else None, rows=rows)


def cache_of(mx, cfg, rows, H, D):
    ts = dict(k_tensor_scale=torch.tensor([0.002], device="cuda"), v_tensor_scale=torch.tensor([0.0013], device="cuda")) if cfg.tensor_scale else {}
    c = mx.kv_cache(rows, 1, H, D, cfg, device="cuda", **ts)
    for t in (c.k, c.v):
        t.codes.fill_(0x5A if cfg.elem not in mx.FP6 else 0x1A)
        t.scales.fill_(0x33)
    return c


def reference(x, H, D, gain, eps, positions, inv_freq, interleaved):
    """(value, |a| + |b|) of rotated heads in binary64."""
    x = x.double().reshape(-1, H, D)
    if gain is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gain.double()
    y, mag = x.clone(), x.abs()
    if inv_freq is not None:
        r = 2 * inv_freq.numel()
        f = positions.double()[:, None, None] * inv_freq.double()
        a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
        ya, yb, m = a * f.cos() - b * f.sin(), b * f.cos() + a * f.sin(), a.abs() + b.abs()
        if interleaved:
            y[..., 0:r:2], y[..., 1:r:2], mag[..., 0:r:2], mag[..., 1:r:2] = ya, yb, m, m
        else:
            y[..., :r // 2], y[..., r // 2:r], mag[..., :r // 2], mag[..., r // 2:r] = ya, yb, m, m
    return y, mag


def check_heads(got, ref, mag):
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    tol = mag * 25 * 2.0 ** -24
    assert bool(((got.double() - ref).abs() <= tol + (ref.abs() + tol) * half + 1e-38).all())


def check_cache(mx, cache, x, which, slots):
    """The rows hold the quantization of x at the slots inside, and 0x5A / 0x33 elsewhere."""
    t = cache.k if which == "k" else cache.v
    rows = cache.pages * cache.page_size
    keep = (slots >= 0) & (slots < rows)
    codes, scales = t.codes.view(rows, -1), t.scales.view(rows, -1)
    if int(keep.sum()):
        xq = x.reshape(x.shape[0], -1)[keep].contiguous()
        q = mx.quantize(xq, cache.cfg, stats=False, tensor_scale=t.tensor_scale)
        assert torch.equal(codes[slots[keep]], q.codes.view(xq.shape[0], -1))
        assert torch.equal(scales[slots[keep]], q.scales.view(xq.shape[0], -1))
    rest = torch.ones(rows, dtype=torch.bool, device=slots.device)
    rest[slots[keep]] = False
    assert bool((codes[rest] == (0x5A if cache.cfg.elem not in mx.FP6 else 0x1A)).all()) and bool((scales[rest] == 0x33).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", NAMES)
def test_cache_formats(mx, name, dtype):
    cfg = configs(mx)[name]
    s = inputs(37, 4, 2, 128, dtype, 128)
    c = cache_of(mx, cfg, s["rows"], 2, 128)
    q, k = mx.kv_append(c, s["q"], s["k"], s["v"], s["slots"], s["positions"], q_gain=s["q_gain"], k_gain=s["k_gain"],
                        inv_freq=s["inv_freq"], k_out=True)
    for got, x, h, g in ((q, s["q"], 4, s["q_gain"]), (k, s["k"], 2, s["k_gain"])):
        check_heads(got, *reference(x, h, 128, g, 1e-6, s["positions"], s["inv_freq"], False))
    check_cache(mx, c, k, "k", s["slots"])
    check_cache(mx, c, s["v"], "v", s["slots"])


@pytest.mark.parametrize("T,Hq,H,D,rot", [(1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (3, 7, 1, 64, 32), (5, 3, 3, 256, 256),
                                          (2, 16, 2, 256, 64), (9, 5, 5, 64, 16), (4, 8, 8, 128, 0), (2500, 6, 2, 64, 64),
                                          (3000, 4, 1, 128, 96)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_head_layouts(mx, T, Hq, H, D, rot, interleaved):
    for dtype in (torch.bfloat16, torch.float32):
        s = inputs(T, Hq, H, D, dtype, rot, seed=T)
        c = cache_of(mx, mx.MXFP4, s["rows"], H, D)
        gk = s["k_gain"] if Hq % 2 else None           # a norm of queries alone, or of both
        q, k = mx.kv_append(c, s["q"], s["k"], s["v"], s["slots"], s["positions"], q_gain=s["q_gain"], k_gain=gk, eps=1e-5,
                            inv_freq=s["inv_freq"], interleaved=interleaved, k_out=True)
        check_heads(q, *reference(s["q"], Hq, D, s["q_gain"], 1e-5, s["positions"], s["inv_freq"], interleaved))
        check_heads(k, *reference(s["k"], H, D, gk, 1e-5, s["positions"], s["inv_freq"], interleaved))
        check_cache(mx, c, k, "k", s["slots"])
        check_cache(mx, c, s["v"], "v", s["slots"])


def test_padding_and_foreign_slots(mx):
    s = inputs(20, 2, 1, 64, torch.bfloat16, 64, rows=30)
    s["slots"][[0, 5, 19]] = torch.tensor([-1, 30, 1 << 45], device="cuda")
    s["slots"][7] = -(1 << 50)
    c = cache_of(mx, mx.MXFP4, 30, 1, 64)
    _, k = mx.kv_append(c, s["q"], s["k"], s["v"], s["slots"], s["positions"], inv_freq=s["inv_freq"], k_out=True)
    check_cache(mx, c, k, "k", s["slots"])
    check_cache(mx, c, s["v"], "v", s["slots"])


def test_strides_alignment_and_in_place(mx):
    """Tokens and heads at odd places, outputs into slices, and outputs over the inputs: the same results."""
    s = inputs(11, 4, 2, 64, torch.bfloat16, 64)
    args = dict(q_gain=s["q_gain"], k_gain=s["k_gain"], inv_freq=s["inv_freq"])
    c = cache_of(mx, mx.MXFP4, s["rows"], 2, 64)
    q, k = mx.kv_append(c, s["q"], s["k"], s["v"], s["slots"], s["positions"], k_out=True, **args)
    odd = torch.empty(11, 8 * 64 + 5, dtype=torch.bfloat16, device="cuda")
    odd[:, 3:3 + 512] = s["qkv"]
    c2 = cache_of(mx, mx.MXFP4, s["rows"], 2, 64)
    out = torch.full((11, 300), 7.0, dtype=torch.bfloat16, device="cuda")
    q2, k2 = mx.kv_append(c2, odd[:, 3:259], odd[:, 259:387].unflatten(1, (2, 64)), odd[:, 387:515], s["slots"], s["positions"],
                          q_out=out[:, 1:257], k_out=True, **args)
    assert torch.equal(q2, q.flatten(1)) and torch.equal(k2, k) and bool((out[:, 257:] == 7).all()) and bool((out[:, 0] == 7).all())
    assert torch.equal(c2.k.codes, c.k.codes) and torch.equal(c2.v.codes, c.v.codes) and torch.equal(c2.k.scales, c.k.scales)
    c3 = cache_of(mx, mx.MXFP4, s["rows"], 2, 64)
    own = s["qkv"].clone()
    mx.kv_append(c3, own[:, :256], own[:, 256:384], own[:, 384:], s["slots"], s["positions"], q_out=own[:, :256], k_out=own[:, 256:384], **args)
    assert torch.equal(own[:, :256], q.flatten(1)) and torch.equal(own[:, 256:384], k.flatten(1)) and torch.equal(c3.k.codes, c.k.codes)


def test_without_queries_norm_or_rotation(mx):
    s = inputs(6, 1, 2, 128, torch.float32, 0)
    c = cache_of(mx, mx.Config(elem=mx.E2M3), s["rows"], 2, 128)
    q, k = mx.kv_append(c, None, s["k"], s["v"], s["slots"])
    assert q is None and k is None
    check_cache(mx, c, s["k"], "k", s["slots"])
    check_cache(mx, c, s["v"], "v", s["slots"])


def test_special_values(mx):
    s = inputs(8, 1, 1, 64, torch.bfloat16, 0)
    k, v = s["k"].clone(), s["v"].clone()
    k[0, 3], k[1, 40], v[2, 5], v[3], k[4] = math.inf, math.nan, -math.inf, 0.0, 0.0
    v[5] = 2.0 ** -130
    v[6, 0] = -0.0
    for name in ("mxfp4", "nvfp4", "e2m3", "int4", "e3m2_b16"):
        c = cache_of(mx, configs(mx)[name], s["rows"], 1, 64)
        mx.kv_append(c, None, k, v, s["slots"])
        check_cache(mx, c, k, "k", s["slots"])
        check_cache(mx, c, v, "v", s["slots"])
    # the norm of a zero head is zero, of one with an infinity NaN
    c = cache_of(mx, mx.MXFP4, s["rows"], 1, 64)
    _, ko = mx.kv_append(c, None, k, v, s["slots"], k_gain=s["k_gain"], k_out=True)
    assert bool((ko[4] == 0).all()) and bool(torch.isnan(ko[0, 0, 3])) and bool(torch.isnan(ko[1]).all())


def test_far_positions(mx):
    """The angle of a position keeps its fraction of a turn far out."""
    s = inputs(4, 2, 1, 64, torch.float32, 64)
    s["positions"] = torch.tensor([0, 1, 1 << 20, (1 << 24) + 1], device="cuda")
    c = cache_of(mx, mx.MXFP4, s["rows"], 1, 64)
    q, _ = mx.kv_append(c, s["q"], s["k"], s["v"], s["slots"], s["positions"], inv_freq=s["inv_freq"])
    check_heads(q, *reference(s["q"], 2, 64, None, 0, s["positions"], s["inv_freq"], False))


def test_cache_past_32_bit_offsets(mx):
    rows = (1 << 22) + 64                                # times 1024 elements: more than 2^32
    s = inputs(3, 8, 8, 128, torch.bfloat16, 128)
    slots = torch.tensor([rows - 1, 1 << 22, 5], device="cuda")
    c = mx.kv_cache(rows, 1, 8, 128, mx.Config(elem=mx.E2M3))
    _, k = mx.kv_append(c, s["q"], s["k"], s["v"], slots, s["positions"], inv_freq=s["inv_freq"], k_out=True)
    for t, x in ((c.k, k.flatten(1)), (c.v, s["v"])):
        q = mx.quantize(x.contiguous(), c.cfg, stats=False)
        assert torch.equal(t.codes.view(rows, 1024)[slots], q.codes.view(3, 1024))
        assert torch.equal(t.scales.view(rows, 32)[slots], q.scales.view(3, 32))
        assert int(t.codes.count_nonzero()) == int(q.codes.count_nonzero())


def test_graph_and_streams(mx):
    s = inputs(9, 4, 2, 128, torch.bfloat16, 128)
    args = dict(q_gain=s["q_gain"], k_gain=s["k_gain"], inv_freq=s["inv_freq"])
    c = cache_of(mx, mx.MXFP4, s["rows"], 2, 128)
    q, _ = mx.kv_append(c, s["q"], s["k"], s["v"], s["slots"], s["positions"], **args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    c2 = cache_of(mx, mx.MXFP4, s["rows"], 2, 128)
    torch.cuda.synchronize()
    q2, _ = mx.kv_append(c2, s["q"], s["k"], s["v"], s["slots"], s["positions"], stream=side, **args)
    side.synchronize()
    assert torch.equal(q, q2) and torch.equal(c.k.codes, c2.k.codes)
    c3 = cache_of(mx, mx.MXFP4, s["rows"], 2, 128)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q3, _ = mx.kv_append(c3, s["q"], s["k"], s["v"], s["slots"], s["positions"], **args)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(q3, q) and torch.equal(c3.v.codes, c.v.codes) and torch.equal(c3.v.scales, c.v.scales)


def test_no_tokens(mx):
    s = inputs(2, 4, 2, 64, torch.bfloat16, 64)
    c = cache_of(mx, mx.MXFP4, 8, 2, 64)
    q, k = mx.kv_append(c, s["q"][:0], s["k"][:0], s["v"][:0], s["slots"][:0], s["positions"][:0], inv_freq=s["inv_freq"], k_out=True)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)


def test_refusals_of_the_binding(mx):
    s = inputs(4, 2, 1, 64, torch.bfloat16, 64)
    c = cache_of(mx, mx.MXFP4, s["rows"], 1, 64)
    good = dict(q=s["q"], k=s["k"], v=s["v"], slots=s["slots"], positions=s["positions"], inv_freq=s["inv_freq"])
    call = lambda **k: mx.kv_append(c, **{**good, **k})  # noqa: E731
    wide = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    for k in (dict(k=s["k"].cpu()), dict(v=s["v"].float()), dict(v=s["v"][:3]), dict(k=wide), dict(k=wide[:, ::2]), dict(q=s["q"].cpu()),
              dict(slots=s["slots"].int()), dict(slots=s["slots"][:3]), dict(slots=s["slots"].cpu()), dict(positions=None),
              dict(positions=s["positions"].int()), dict(inv_freq=s["inv_freq"].double()), dict(q_gain=torch.ones(63, device="cuda")),
              dict(k_gain=torch.ones(64, dtype=torch.bfloat16, device="cuda")), dict(q_out=s["q"].float()), dict(k_out=s["v"][:3]),
              dict(v=s["v"][:1].expand(4, 64))):
        with pytest.raises(ValueError):
            call(**k)
    for k in (dict(k=s["k"].half(), v=s["v"].half(), q=s["q"].half()), dict(k=None), dict(eps="x"), dict(k_out=3)):
        with pytest.raises(TypeError):
            call(**k)
    with pytest.raises(mx.MXError) as e:
        call(inv_freq=torch.ones(12, device="cuda"))         # 24 rotated elements
    assert e.value.code == -2
    check_cache(mx, c, s["k"], "k", torch.full_like(s["slots"], -1))    # nothing was written
