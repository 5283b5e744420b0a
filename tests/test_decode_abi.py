"""The decode-time operators reject what they do not take on the host, before
any launch (no GPU needed: fake pointers are never read)."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def mx():
    from microscaling_block_quantization_b200 import build
    build.build()
    import microscaling_block_quantization_b200 as m
    m.lib()
    return m


P = C.c_void_p


def gemv(mx, cfg, M=1, N=64, K=256, x=4096, xd=0, ldx=None, codes=4096, scales=4096, ts=4096, macro=4096, off=4096,
         y=4096, yd=0, ldy=None):
    p = lambda v: None if v is None else P(v)  # noqa: E731
    return mx.mx_gemv(cfg, p(x), xd, K if ldx is None else ldx, M, p(codes), p(scales), p(ts), p(macro), p(off), N, K,
                      p(y), yd, N if ldy is None else ldy, None)


@pytest.mark.parametrize("cfg,rc", [
    (dict(elem=2), -2), (dict(elem=3), -2),                  # FP6 elements
    (dict(axis=1), -2), (dict(axis=2), -2),                  # blocks not along K
    (dict(hadamard=32), -2),                                 # rotated weights
    (dict(asymmetric=1, block=16), -2),                      # offsets of small blocks
    (dict(block=24), -2), (dict(elem=7), -1),
    (dict(rule=3), -1),
])
def test_gemv_configurations(mx, cfg, rc):
    assert gemv(mx, mx.Config(**cfg)) == rc


@pytest.mark.parametrize("args,rc", [
    (dict(K=40), -1), (dict(M=-1), -1), (dict(M=(1 << 17) + 1), -1), (dict(N=-1), -1),
    (dict(ldx=255), -1), (dict(ldy=63), -1), (dict(xd=2), -1), (dict(yd=7), -1),
    (dict(x=None), -1), (dict(codes=None), -1), (dict(scales=None), -1), (dict(y=None), -1),
    (dict(codes=4104), -3), (dict(scales=4104), -3), (dict(x=4097), -3), (dict(x=4098, xd=1), -3), (dict(y=4097), -3),
    (dict(N=1 << 24, K=256), -1),                            # 2^32 weights
    (dict(M=0), 0), (dict(N=0, ldy=0), 0),
])
def test_gemv_arguments(mx, args, rc):
    assert gemv(mx, mx.MXFP4, **args) == rc


def test_gemv_optional_operands(mx):
    assert gemv(mx, mx.NVFP4, ts=None) == -1
    assert gemv(mx, mx.NVFP4, ts=4098) == -3
    assert gemv(mx, mx.Config(macro_block=128), macro=None) == -1
    assert gemv(mx, mx.Config(macro_block=128), macro=4104) == -3
    assert gemv(mx, mx.Config(asymmetric=1), off=None) == -1
    assert gemv(mx, mx.Config(asymmetric=1), off=4104) == -3


def test_gemv_binding_refusals(mx):
    import torch
    q = mx.Quantized(mx.MXFP4, 4, 64, *(torch.zeros(16, dtype=torch.uint8) for _ in range(2)), torch.ones(1), None, None, None)
    with pytest.raises(ValueError):
        mx.gemv(torch.zeros(1, 64), q)                       # not on a CUDA device
