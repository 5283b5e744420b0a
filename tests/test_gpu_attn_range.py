"""GPU parity of decode attention where value scales differ by far more than an
f16 weight's range, with the weight of the softmax on the small ones.

The reference is binary64 on the dequantized cache.  Tolerance per element, with
u = 2^-24, as in the other attention tests: e the score's bound, sums of n tokens
and the exponential (n / 16 + 64) 2 u, a weight's rounding w (2^-12 for bf16
results, 2^-23 for binary32), against sum p |v|:
  tol = sum p |v| (2 e + (n / 16 + 64) 2 u + w) + half a step of the result
      + what may be dropped: products below 2^-24 of the largest weight times a
        block's smallest scale s (blocks of zeros aside), of elements up to 28 s (E3M2).
        The block's largest element is 16 s at least (E3M2, E3M0), or 4 s of 6 or 7.5
        (E2M1, E2M3), 3.5 s of 7 (INT4, ceil), 2 s of 6 (nearest scales, which round
        up to 2 below the normal range): n 2^-24 s 28 < n 2^-21 of the smallest of the
        blocks' largest elements.
NVFP4 (weights by themselves): dropped below 2^-35, n 2^-35 max |v|."""
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
        "e2m3": mx.Config(elem=mx.E2M3),
        "e3m2_b16": mx.Config(elem=mx.E3M2, block=16),
        "e3m0": mx.Config(elem=mx.E3M0),
        "int4": mx.Config(elem=mx.INT4, rule=mx.RULE_CEIL),
        "nvfp4": nv,
        "ue5m3_b32": dataclasses.replace(nv, block=32, scale_fmt=mx.SCALE_UE5M3),
    }


NAMES = ["mxfp4", "mxfp4_b16", "mxfp4_b64", "e2m3", "e3m2_b16", "e3m0", "int4", "nvfp4", "ue5m3_b32"]
SPAN = {"nvfp4": 0.1, "ue5m3_b32": 0.35}     # exponents of scales that these formats hold, of +-40


def cache(mx, cfg, score, exps, D, dtype, seed=0):
    """Two sequences (the second with the tokens in reverse order) whose tokens have the given scores against the first
    head's query (the other heads': 0.9, 0.5 and -1 of them) and values scaled by 2^exps (None: zeros)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, H = len(score), 4
    per = -(-n // 16)
    ts = dict(k_tensor_scale=torch.ones(1, device="cuda"), v_tensor_scale=torch.ones(1, device="cuda")) if cfg.tensor_scale else {}
    c = mx.kv_cache(2 * per + 1, 16, 1, D, cfg, **ts)
    q0 = torch.randn(D, generator=g, device="cuda")
    q = torch.stack([q0, 0.9 * q0, 0.5 * q0, -q0])[None].repeat(2, 1, 1).to(dtype)
    k = torch.tensor(score, device="cuda")[:, None] * math.sqrt(D) * q0 / (q0 @ q0) + 0.01 * torch.randn(n, D, generator=g, device="cuda")
    v = torch.randn(n, D, generator=g, device="cuda") * torch.tensor([0.0 if e is None else 2.0 ** e for e in exps], device="cuda")[:, None]
    table = torch.randperm(2 * per + 1, generator=g, device="cuda")[:2 * per].reshape(2, per).int()
    for t, x in ((c.k, k), (c.v, v)):
        full = torch.zeros(c.pages * 16, D, device="cuda")
        for b, y in enumerate((x, x.flip(0))):
            at = torch.arange(n, device="cuda")
            full[table[b].long()[at // 16] * 16 + at % 16] = y
        z = mx.quantize(full, cfg, stats=False, tensor_scale=t.tensor_scale)
        t.codes.copy_(z.codes)
        t.scales.copy_(z.scales)
    return c, q, table, torch.tensor([n, n], dtype=torch.int32, device="cuda")


def check(mx, c, q, table, lengths, out):
    D = c.head_dim
    wide = out.dtype == torch.float32 or q.dtype == torch.float32
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    k, v = (mx.dequantize(t).double() for t in (c.k, c.v))
    alone = c.cfg.elem == mx.E2M1 and c.cfg.scale_fmt == mx.SCALE_UE4M3
    for b in range(2):
        n = int(lengths[b])
        t = torch.arange(n, device="cuda")
        rows = table[b].long()[t // 16] * 16 + t % 16
        kb, vb, qb = k[rows], v[rows], q[b].double()
        s = qb @ kb.T * D ** -0.5
        e = (qb.abs() @ kb.abs().T * D ** -0.5).amax(1) * (D / 16 + 16) * 2.0 ** -23
        p = torch.softmax(s, 1)
        ref, mag = p @ vb, p @ vb.abs()
        w = (2 * e + (n / 16 + 64) * 2.0 ** -23 + (2.0 ** -23 if wide else 2.0 ** -12))[:, None]
        big = vb.abs().unflatten(1, (-1, min(c.cfg.block, 32))).amax(2)
        least = torch.where(big > 0, big, math.inf).amin(0)
        drop = n * 2.0 ** -35 * vb.abs().amax() if alone else \
            n * 2.0 ** -21 * torch.where(least.isfinite(), least, 0.0).repeat_interleave(min(c.cfg.block, 32))
        tol = mag * w + drop + 1e-38
        err = (out[b].double() - ref).abs()
        assert bool((err <= tol + (ref.abs() + tol) * half).all()), (b, float((err / (tol + (ref.abs() + tol) * half)).max()))


LN2 = math.log(2.0)
CASES = {
    "two, 2^26 apart": ([0.0, 60 * LN2], [26, 0]),
    "two, 2^40 apart": ([0.0, 60 * LN2], [40, 0]),
    "two, equal parts": ([0.0, 40 * LN2], [40, 0]),
    "four, mixed": ([0.0, 30 * LN2, 60 * LN2, 58 * LN2], [30, 0, -30, -28]),
    "in another tile": ([60 * LN2] + [0.0] * 34 + [1.0], [-20] + [10] * 34 + [12]),
    "one among many": ([0.0] * 20 + [50 * LN2] + [2.0] * 60, [15] * 20 + [-15] + [14] * 60),
    "blocks of zeros": ([0.0, 3.0, 60 * LN2] + [1.0] * 20, [20, None, -10] + [None, 20] * 10),
    "all zeros but one": ([0.0] * 17 + [-60 * LN2] + [0.0] * 20, [None] * 17 + [30] + [None] * 20),
}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", list(CASES))
@pytest.mark.parametrize("name", NAMES)
def test_the_weight_is_on_small_values(mx, name, case, dtype):
    score, exps = CASES[case]
    exps = [None if e is None else round(e * SPAN.get(name, 1.0)) for e in exps]
    for D in (64, 128, 256):
        args = cache(mx, configs(mx)[name], score, exps, D, dtype)
        check(mx, *args, mx.attn_decode(*args))


@pytest.mark.parametrize("name", NAMES)
def test_scores_and_scales_at_random(mx, name):
    """Tokens of scores within +-45 and values within 2^+-40, in one stretch and in many."""
    g = torch.Generator().manual_seed(7)
    for n, D in ((5, 128), (50, 64), (700, 128), (3000, 256)):
        score = ((torch.rand(n, generator=g) - 0.5) * 90).tolist()
        exps = [round(float(x) * SPAN.get(name, 1.0)) for x in (torch.rand(n, generator=g) - 0.5) * 80]
        for dtype in (torch.bfloat16, torch.float32):
            args = cache(mx, configs(mx)[name], score, exps, D, dtype, seed=n)
            check(mx, *args, mx.attn_decode(*args))


def test_least_scales_of_the_range(mx):
    """Scales at the least code, with codes that are not zero."""
    for name in ("mxfp4", "mxfp4_b64"):
        args = cache(mx, configs(mx)[name], [0.0, 1.0, 2.0] * 9, [-125] * 27, 128, torch.float32)
        out = mx.attn_decode(*args)
        v = mx.dequantize(args[0].v).abs().amax()
        assert float(v) > 0.0 and float(out.abs().amax()) > 0.01 * float(v)
