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


def cache(mx, pages=4, page_size=16, kv=2, dim=64, k=4096, v=4096, ks=4096, vs=4096, kt=4096, vt=4096):
    return C.byref(mx.mx_kv_cache(k, v, ks, vs, kt, vt, pages, page_size, kv, dim))


def append(mx, cfg, c, q=4096, k=4096, v=4096, dt=0, ldq=None, ldk=128, ldv=128, T=3, Hq=4, gq=4096, gk=4096, eps=1e-6,
           freq=4096, rot=64, inter=0, pos=4096, slots=4096, qo=4096, ldqo=256, ko=None, ldko=128):
    p = lambda x: None if x is None else P(x)  # noqa: E731
    return mx.mx_kv_append(cfg, c, p(q), p(k), p(v), dt, 256 if ldq is None else ldq, ldk, ldv, T, Hq, p(gq), p(gk), eps,
                           p(freq), rot, inter, p(pos), p(slots), p(qo), ldqo, p(ko), ldko, None)


CACHE_CONFIGS = [
    (dict(block=8), -2), (dict(block=256), -2), (dict(block=128), -2),      # 128 is longer than the head
    (dict(axis=2), -2), (dict(axis=1, block=8), -2), (dict(sf_layout=1), -2), (dict(asymmetric=1), -2), (dict(macro_block=128), -2),
    (dict(hadamard=32), -2), (dict(rule=4), -2), (dict(round=2), -2),
    (dict(block=16, scale_fmt=1, rule=3, tensor_scale=1), -2), (dict(block=16, scale_fmt=1, rule=3, tensor_scale=3), -2),
    (dict(elem=9), -1), (dict(rule=3), -1),
]
CACHES = [
    (dict(dim=96), -2), (dict(kv=0), -1), (dict(page_size=0), -1), (dict(pages=-1), -1), (dict(pages=1 << 30, page_size=2), -1),
    (dict(k=None), -1), (dict(v=None), -1), (dict(ks=None), -1), (dict(vs=None), -1),
    (dict(k=4104), -3), (dict(v=4104), -3), (dict(ks=4104), -3), (dict(vs=4100), -3),
]


@pytest.mark.parametrize("cfg,rc", CACHE_CONFIGS)
def test_append_configurations(mx, cfg, rc):
    assert append(mx, mx.Config(**cfg), cache(mx)) == rc


@pytest.mark.parametrize("args,rc", CACHES)
def test_append_caches(mx, args, rc):
    assert append(mx, mx.MXFP4, cache(mx, **args)) == rc


@pytest.mark.parametrize("args,rc", [
    (dict(dt=2), -1), (dict(T=-1), -1), (dict(Hq=-1), -1), (dict(inter=2), -1), (dict(rot=80), -1), (dict(rot=24), -2),
    (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1),
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(qo=None), -1), (dict(slots=None), -1), (dict(pos=None), -1),
    (dict(freq=None), -1), (dict(ldq=255), -1), (dict(ldk=127), -1), (dict(ldv=0), -1), (dict(ldqo=255), -1), (dict(ko=4096, ldko=1), -1),
    (dict(q=4097), -3), (dict(k=4097), -3), (dict(v=4098, dt=1), -3), (dict(ko=4097), -3), (dict(gq=4100), -3), (dict(gk=4104), -3),
    (dict(freq=4098), -3), (dict(pos=4100), -3), (dict(slots=4100), -3), (dict(T=0), 0),
])
def test_append_arguments(mx, args, rc):
    assert append(mx, mx.MXFP4, cache(mx), **args) == rc


def test_append_tensor_scales(mx):
    nv = mx.Config(block=16, scale_fmt=1, rule=3, tensor_scale=2)
    assert append(mx, nv, cache(mx, kt=None)) == -1 and append(mx, nv, cache(mx, vt=None)) == -1
    assert append(mx, nv, cache(mx, vt=4098)) == -3
    assert append(mx, nv, None) == -1


def test_append_binding_refusals(mx):
    import torch
    c = mx.kv_cache(2, 4, 1, 64, device="cpu")
    with pytest.raises(ValueError):
        mx.kv_append(c, None, torch.zeros(1, 64), torch.zeros(1, 64), torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError):
        mx.kv_cache(2, 4, 1, 64, mx.Config(block=16, scale_fmt=1, rule=3, tensor_scale=2), device="cpu")
    small = mx.kv_cache(2, 4, 1, 64, device="cpu")
    small.k.codes = small.k.codes[:8]
    with pytest.raises(ValueError):
        small.ref()


def attn(mx, cfg, c, q=4096, qd=0, ldq=256, S=2, Hq=4, tab=4096, ldt=3, mp=3, ln=4096, scale=0.1, win=0, sinks=0, out=4096, od=0,
         ldo=256, lse=None, ws=4096, wb=1 << 40):
    p = lambda x: None if x is None else P(x)  # noqa: E731
    return mx.mx_attn_decode(cfg, c, p(q), qd, ldq, S, Hq, p(tab), ldt, mp, p(ln), scale, win, sinks, p(out), od, ldo, p(lse),
                             p(ws), wb, None)


@pytest.mark.parametrize("cfg,rc", CACHE_CONFIGS)
def test_attention_configurations(mx, cfg, rc):
    assert attn(mx, mx.Config(**cfg), cache(mx)) == rc


@pytest.mark.parametrize("args,rc", CACHES)
def test_attention_caches(mx, args, rc):
    assert attn(mx, mx.MXFP4, cache(mx, **args)) == rc


@pytest.mark.parametrize("args,rc", [
    (dict(S=1 << 20, Hq=4096, ldq=1 << 20, ldo=1 << 20), -1),
    (dict(qd=2), -1), (dict(od=3), -1), (dict(S=-1), -1), (dict(S=(1 << 20) + 1), -1), (dict(Hq=0), -1), (dict(Hq=3), -1),
    (dict(mp=-1), -1), (dict(mp=1 << 28, ldt=1 << 28), -1), (dict(win=-1), -1), (dict(sinks=-2), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(q=None), -1), (dict(out=None), -1), (dict(ln=None), -1), (dict(tab=None), -1),
    (dict(ldq=255), -1), (dict(ldo=255), -1), (dict(ldt=2), -1),
    (dict(q=4097), -3), (dict(q=4098, qd=1), -3), (dict(out=4097), -3), (dict(tab=4098), -3), (dict(ln=4098), -3), (dict(lse=4098), -3),
    (dict(mp=1000, ldt=1000, ws=None), -5), (dict(mp=1000, ldt=1000, wb=1000), -5), (dict(mp=1000, ldt=1000, ws=4104), -3),
    (dict(S=0), 0),
])
def test_attention_arguments(mx, args, rc):
    assert attn(mx, mx.MXFP4, cache(mx), **args) == rc


def test_attention_workspace_size(mx):
    L = mx.lib()
    c = cache(mx, pages=1 << 12, page_size=64, dim=128)
    assert L.mx_attn_workspace_bytes(c, 0, 4, 10, 0, 0) == 0 and L.mx_attn_workspace_bytes(None, 1, 4, 10, 0, 0) == 0
    assert L.mx_attn_workspace_bytes(c, 1, 4, 1, 0, 0) == 0                       # one page: not split
    long, short = L.mx_attn_workspace_bytes(c, 1, 4, 1 << 12, 0, 0), L.mx_attn_workspace_bytes(c, 1, 4, 1 << 12, 5000, 4)
    assert L.mx_attn_workspace_bytes(c, 1, 4, 1 << 12, 200, 4) == 0               # joined within a CTA
    assert L.mx_attn_workspace_bytes(c, 128, 4, 16, 0, 0) == 0
    assert long > short > 0 and long % (4 * (8 + 512)) == 0


def test_attention_binding_refusals(mx):
    import torch
    c = mx.kv_cache(2, 4, 1, 64, device="cpu")
    with pytest.raises(ValueError):
        mx.attn_decode(c, torch.zeros(1, 1, 64), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
