"""GPU parity of the matrix-vector products on 4-bit block-scaled weights.

y = x W^T is checked against the dequantized weights (the CPU oracle's, or the
library's dequantizer, itself bit-exact with the oracle) multiplied in
binary64.  The kernel's products are exact; its sums are binary32: within a
block by the matrix instruction, then over blocks, chunks and splits.  With
n additions on the longest path of binary32 sums, |error| <= n 2^-24 sum |x W|
(a multiply-add rounds once); one more rounding each for the tensor scale and
the output.  The matrix instruction may truncate instead of rounding, 2^-23
per addition.  A sum passes 16 products per instruction pair, K / 32 blocks,
the K splits: (K / 32 + 64) 2^-23 covers them for the K here.  Block offsets
add one term per block to the same sums."""
import pytest
import torch

from microscaling_block_quantization_b200 import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    from microscaling_block_quantization_b200 import build
    build.build()
    import microscaling_block_quantization_b200 as m
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return m


def weights(mx, cfg, n, k, seed=3, sigma=0.02):
    w = inputs.normal(n, k, sigma=sigma, seed=seed).cuda()
    return mx.quantize(w, cfg, stats=False)


def reference(mx, x, qw):
    """(x W^T, sum |x| |W|) in binary64, W from the dequantizer in its own steps."""
    w = mx.dequantize(qw, torch.float32).double()
    x = x.double()
    bound = x.abs() @ w.abs().T
    if qw.offsets is not None:
        # an offset block's value is q s + o: its terms, not their sum, pass through the sums
        o = qw.offsets.view(torch.bfloat16).double().abs()
        o = o.view(qw.rows, -1).repeat_interleave(qw.cfg.block, 1)
        bound = bound + 2 * x.abs() @ o.T
    return x @ w.T, bound


def check(mx, x, qw, y):
    ref, bound = reference(mx, x, qw)
    k = x.shape[-1]
    tol = bound * (k / 32 + 64) * 2.0 ** -23
    if y.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + ref.abs() * 2.0 ** -8
    else:
        tol = tol + ref.abs() * 2.0 ** -23
    err = (y.double() - ref).abs()
    assert bool((err <= tol + 1e-38).all()), float((err - tol).max())


def configs(mx):
    return {
        "mxfp4": mx.Config(),
        "mxfp4_chunked": mx.Config(sf_layout=1),
        "nvfp4": mx.NVFP4,
        "nvfp4_chunked": mx.Config(block=16, scale_fmt=1, rule=3, tensor_scale=1, sf_layout=1),
        "ue5m3_b8": mx.Config(block=8, scale_fmt=2, rule=3, tensor_scale=1),
        "ue4m3_b64_chunked": mx.Config(block=64, scale_fmt=1, rule=3, sf_layout=1),
        "ue4m3_b8_chunked": mx.Config(block=8, scale_fmt=1, rule=3, tensor_scale=1, sf_layout=1),
        "pow2_ue4m3_b16": mx.Config(block=16, scale_fmt=1, rule=1),
        "mxfp4_b64": mx.Config(block=64),
        "mxfp4_b128_chunked": mx.Config(block=128, sf_layout=1),
        "mxfp4_b256": mx.Config(block=256),
        "mbs": mx.Config(macro_block=128),
        "mbs_b16": mx.Config(macro_block=128, block=16),
        "e3m0": mx.Config(elem=mx.E3M0, rule=mx.RULE_CEIL),
        "e3m0_b16": mx.Config(elem=mx.E3M0, block=16),
        "int4": mx.Config(elem=mx.INT4, rule=mx.RULE_CEIL),
        "int4_b8": mx.Config(elem=mx.INT4, block=8),
        "int4_asym": mx.Config(elem=mx.INT4, rule=mx.RULE_CEIL, asymmetric=1),
        "int4_asym_b64": mx.Config(elem=mx.INT4, rule=mx.RULE_CEIL, asymmetric=1, block=64),
        "int4_asym_b128_chunked": mx.Config(elem=mx.INT4, rule=mx.RULE_CEIL, asymmetric=1, block=128, sf_layout=1),
        "int4_asym_chunked": mx.Config(elem=mx.INT4, rule=mx.RULE_CEIL, asymmetric=1, sf_layout=1),
        "e2m1_asym": mx.Config(asymmetric=1),
        "e3m0_asym_b256": mx.Config(elem=mx.E3M0, asymmetric=1, block=256),
    }


NAMES = ["mxfp4", "mxfp4_chunked", "nvfp4", "nvfp4_chunked", "ue5m3_b8", "ue4m3_b64_chunked", "ue4m3_b8_chunked",
         "pow2_ue4m3_b16", "mxfp4_b64", "mxfp4_b128_chunked", "mxfp4_b256", "mbs", "mbs_b16", "e3m0", "e3m0_b16", "int4", "int4_b8",
         "int4_asym", "int4_asym_b64", "int4_asym_b128_chunked", "int4_asym_chunked", "e2m1_asym", "e3m0_asym_b256"]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", NAMES)
def test_every_weight_form(mx, name, dtype):
    qw = weights(mx, configs(mx)[name], 384, 1024)
    x = inputs.laplace_outlier_cols(3, 1024, seed=5, n_outlier_cols=2, dtype=dtype).cuda()
    y = mx.gemv(x, qw, torch.float32)
    check(mx, x, qw, y)


def test_against_the_cpu_oracle(mx, orc):
    n, k = 48, 160
    w, x = inputs.normal(n, k, 0.02, 3), inputs.small_normal(5, k, 4)
    r = orc.quantize(orc.Cfg(), w)
    wh = torch.from_numpy(orc.dequantize(orc.Cfg(), r["packed"], r["scales"], None, None, None, n, k)).double()
    y = mx.gemv(x.cuda(), mx.quantize(w.cuda(), mx.MXFP4, stats=False), torch.float32).cpu().double()
    ref, bound = x.double() @ wh.T, x.double().abs() @ wh.abs().T
    assert bool(((y - ref).abs() <= bound * (k / 32 + 64) * 2.0 ** -23).all())


@pytest.mark.parametrize("m", [1, 2, 7, 8, 9, 16, 17, 33])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_of_x(mx, m, dtype):
    qw = weights(mx, mx.MXFP4, 80, 544)
    x = inputs.small_normal(m, 544, 1, dtype=dtype).cuda()
    y = mx.gemv(x, qw)
    assert y.dtype == dtype and y.shape == (m, 80)
    check(mx, x, qw, y)


@pytest.mark.parametrize("n,k", [(1, 32), (15, 64), (16, 96), (17, 160), (33, 1056), (1000, 288), (5, 4128), (129, 32)])
@pytest.mark.parametrize("name", ["mxfp4", "nvfp4", "int4_asym", "ue5m3_b8"])
def test_odd_sizes(mx, name, n, k):
    qw = weights(mx, configs(mx)[name], n, k)
    x = inputs.small_normal(2, k, 1).cuda()
    check(mx, x, qw, mx.gemv(x, qw, torch.float32))


@pytest.mark.parametrize("n,k,m", [(4096, 4096, 1), (14336, 4096, 2), (4096, 14336, 4), (64, 65536, 3), (70000, 256, 1), (32, 131072, 9)])
def test_large_sizes(mx, n, k, m):
    qw = weights(mx, mx.MXFP4, n, k)
    x = inputs.laplace_outlier_cols(m, k, seed=2).cuda()
    check(mx, x, qw, mx.gemv(x, qw, torch.float32))


def test_strided_and_unaligned_rows(mx):
    qw = weights(mx, mx.MXFP4, 40, 256)
    buf = inputs.small_normal(6, 771, 1).cuda()
    for x in (buf[:, 3:259], buf[::2, 8:264], buf[1:2, 5:261]):
        out = torch.full((x.shape[0], 100), 7.0, device="cuda")
        y = mx.gemv(x, qw, out=out[:, 21:61])
        assert y.data_ptr() == out[:, 21:61].data_ptr()
        check(mx, x, qw, y)
        assert bool((out[:, :21] == 7).all()) and bool((out[:, 61:] == 7).all())   # nothing beside the rows
    one = mx.gemv(buf[0, 3:259], qw)
    assert one.shape == (40,) and torch.equal(one, mx.gemv(buf[:1, 3:259], qw)[0])


def test_dynamic_range_of_x(mx):
    """Values 2^-30 of a chunk's largest are exact; a token of tiny or huge values keeps its relative accuracy."""
    qw = weights(mx, mx.MXFP4, 64, 512)
    x = inputs.small_normal(4, 512, 1, dtype=torch.float32)
    x[0] *= 2.0 ** -120
    x[1] *= 2.0 ** 100
    x[2, ::3] *= 2.0 ** -20
    x[3] = 0.0
    for t in (x.cuda(), x.bfloat16().cuda()):
        check(mx, t, qw, mx.gemv(t, qw, torch.float32))
    w = torch.zeros(32, 128)
    w[:, 0], w[:, 1] = 0.0, 1.0
    qw = mx.quantize(w.cuda(), mx.MXFP4, stats=False)
    for dt in (torch.bfloat16, torch.float32):
        t = torch.zeros(1, 128, dtype=dt, device="cuda")
        t[0, 0], t[0, 1] = 2.0 ** 30, 1.0 + 2.0 ** -7      # the largest meets a zero weight
        assert bool((mx.gemv(t, qw, torch.float32) == 1.0 + 2.0 ** -7).all())


def test_special_values(mx):
    w = inputs.normal(32, 256, 0.02, 3)
    w[:, 5] = 0.5
    w[:, 6] = 0.0
    qw = mx.quantize(w.cuda(), mx.MXFP4, stats=False)
    x = inputs.small_normal(4, 256, 1)
    x[0, 5] = float("inf")
    x[1, 6] = float("inf")
    x[2, 7] = float("nan")
    for t in (x.cuda(), x.float().cuda()):
        y = mx.gemv(t, qw, torch.float32)
        assert bool((y[0] == float("inf")).all())            # inf times a positive weight
        assert bool(torch.isnan(y[1]).all())                 # inf times zero
        assert bool(torch.isnan(y[2]).all())
        check(mx, t[3:], qw, y[3:])
    w[9, 40] = float("nan")                                  # a block with the NaN scale code
    y = mx.gemv(x[3:].cuda(), mx.quantize(w.cuda(), mx.MXFP4, stats=False), torch.float32)
    assert bool(torch.isnan(y[0, 9])) and int(torch.isnan(y).sum()) == 1


def test_ragged_last_chunk_ignores_the_next_rows_scales(mx):
    """K = 160: the last 128-column chunk holds one block; the next row's blocks are NaN."""
    w = inputs.normal(32, 160, 0.02, 3)
    w[1::2, :] = float("nan")
    for name in ("mxfp4", "nvfp4", "ue5m3_b8", "int4_asym"):
        cfg = configs(mx)[name]
        ts = torch.ones(1, device="cuda") if cfg.tensor_scale else None
        if cfg.tensor_scale:
            import dataclasses
            cfg = dataclasses.replace(cfg, tensor_scale=mx.TS_GIVEN)
        y = mx.gemv(inputs.small_normal(1, 160, 1).cuda(), mx.quantize(w.cuda(), cfg, stats=False, tensor_scale=ts), torch.float32)
        assert bool(torch.isfinite(y[0, 0::2]).all()) and bool(torch.isnan(y[0, 1::2]).all())


def test_repeatable_streams_and_graph(mx):
    qw = weights(mx, mx.NVFP4, 1000, 2080)
    x = inputs.small_normal(3, 2080, 1).cuda()
    y = mx.gemv(x, qw)
    for _ in range(3):
        assert torch.equal(mx.gemv(x, qw), y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ys = [[mx.gemv(x, qw, stream=s) for s in streams] for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(v, y) for pair in ys for v in pair)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        yg = mx.gemv(x, qw)
    x2 = inputs.small_normal(3, 2080, 9).cuda()
    want = mx.gemv(x2, qw)
    x.copy_(x2)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(yg, want)


def test_after_a_quantizer_on_the_same_stream(mx):
    """The weights are written by the launch just before: the product waits for them."""
    x = inputs.small_normal(1, 4096, 1).cuda()
    ws = [inputs.normal(2048, 4096, 0.02, s).cuda() for s in (1, 2)]
    want = [mx.gemv(x, mx.quantize(w, mx.MXFP4, stats=False)) for w in ws]
    torch.cuda.synchronize()
    q = mx.quantize(ws[0], mx.MXFP4, stats=False)
    for i in range(6):
        mx.quantize(ws[i % 2], mx.MXFP4, out=q, stats=False)
        assert torch.equal(mx.gemv(x, q), want[i % 2])


def test_empty(mx):
    qw = weights(mx, mx.MXFP4, 16, 64)
    assert mx.gemv(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), qw).shape == (0, 16)
    none = mx.Quantized(mx.MXFP4, 4, 0, qw.codes, qw.scales, qw.tensor_scale, None, None, None)
    assert bool((mx.gemv(torch.empty(3, 0, device="cuda"), none) == 0).all())


def test_refusals_of_the_binding(mx):
    """Wrong shapes, types, strides, devices and buffers raise before any launch."""
    qw = weights(mx, mx.MXFP4, 32, 128)
    x = torch.zeros(2, 128, dtype=torch.bfloat16, device="cuda")
    for bad, kind in ((x[:, :96], ValueError), (x[None], ValueError), (x.half(), TypeError), (x.cpu(), ValueError),
                      (torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda")[:, ::2], ValueError),
                      (x[:1].expand(3, 128), ValueError), (None, TypeError)):
        with pytest.raises(kind):
            mx.gemv(bad, qw)
    out = torch.zeros(2, 32, device="cuda")
    for bad, kind in ((out[:1], ValueError), (out.half(), TypeError), (out.cpu(), ValueError), (out.T.contiguous().T, ValueError)):
        with pytest.raises(kind):
            mx.gemv(x, qw, out=bad)
    with pytest.raises(ValueError):
        mx.gemv(x, qw, torch.bfloat16, out=out)
    with pytest.raises(TypeError):
        mx.gemv(x, qw, torch.float16)
    import dataclasses
    for change in (dict(codes=qw.codes[:-16]), dict(scales=qw.scales[:-1]), dict(codes=qw.codes.cpu()), dict(rows=33),
                   dict(codes=torch.zeros(2 * 32 * 64, dtype=torch.uint8, device="cuda")[::2])):
        with pytest.raises(ValueError):
            mx.gemv(x, dataclasses.replace(qw, **change))
    with pytest.raises(mx.MXError) as e:
        mx.gemv(x, dataclasses.replace(qw, cfg=mx.Config(hadamard=32)))
    assert e.value.code == -2
    assert torch.equal(mx.gemv(x, qw), torch.zeros(2, 32, dtype=torch.bfloat16, device="cuda"))
