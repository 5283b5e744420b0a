"""What the matrix-vector product's f16 pieces keep of the activations."""
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [256, 1056])
def test_one_value_of_every_significand(mx, K, dtype):
    """x with one value that is not zero, of a full significand: y is that value times one weight.  bf16: one piece, exact,
    and the product, of 8 and 2 bits, too.  binary32: the value's second piece has 11 of the at most 12 bits left, one unit
    of 2^-23 is lost at most; the product's two parts are added with one rounding, 2^-24 of the result."""
    w = mx.quantize(inputs.normal(64, K, 0.02, 3).cuda(), mx.MXFP4, stats=False)
    wd = mx.dequantize(w).double()
    g = torch.Generator(device="cuda").manual_seed(1)
    M = 512
    value = (1 + torch.rand(M, generator=g, device="cuda")) * torch.exp2(torch.randint(-60, 60, (M,), generator=g, device="cuda").float())
    value[0] = 1 + 2049 * 2.0 ** -23                         # 2049 units beside an f16
    value = value.to(dtype)
    at = torch.randint(0, K, (M,), generator=g, device="cuda")
    x = torch.zeros(M, K, dtype=dtype, device="cuda")
    x[torch.arange(M, device="cuda"), at] = value
    y = torch.cat([mx.gemv(b, w, torch.float32) for b in x.split(16)]).double()
    want = value.double()[:, None] * wd.T[at]
    lost = 0.0 if dtype == torch.bfloat16 else 2.0 ** -23 + 2.0 ** -24 * (1 + 2.0 ** -23)
    assert bool(((y - want).abs() <= lost * want.abs()).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cfg", [dict(asymmetric=1, elem=4, rule=1), dict(asymmetric=1, elem=4, rule=1, block=128), dict(asymmetric=1)])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_not_finite_x_with_offsets(mx, bad, cfg, dtype):
    """(q s) x and o x are summed apart: an infinite x gives infinities or NaN, in its own token alone."""
    w = mx.quantize(inputs.normal(96, 512, 0.02, 3).cuda(), mx.Config(**cfg), stats=False)
    x = inputs.small_normal(3, 512, 1).cuda().to(dtype)
    fine = mx.gemv(x, w)
    x[1, 300] = bad
    y = mx.gemv(x, w)
    assert not bool(torch.isfinite(y[1]).any())
    assert torch.equal(y[0], fine[0]) and torch.equal(y[2], fine[2]) and bool(torch.isfinite(fine).all())
