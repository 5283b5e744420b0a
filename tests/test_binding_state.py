"""What the binding keeps beside a configuration or a cache: safe between
threads, and no part of what is copied or pickled (no GPU needed)."""
import ctypes as C
import gc
import threading
import time

import pytest


@pytest.fixture(scope="module")
def mx():
    from microscaling_block_quantization_b200 import build
    build.build()
    import microscaling_block_quantization_b200 as m
    m.lib()
    return m


def test_first_use_of_a_configuration_by_several_threads(mx, monkeypatch):
    """Threads that meet in a configuration's first use get one struct, which stays."""
    make = mx.Config.c

    def slow(self):
        s = make(self)
        time.sleep(0.05)                     # the others arrive before it is kept
        return s

    monkeypatch.setattr(mx.Config, "c", slow)
    cfg = mx.Config(block=16, seed=77)
    got, gate = [], threading.Barrier(8)

    def use():
        gate.wait()
        got.append((cfg.address(), cfg.ref()))

    threads = [threading.Thread(target=use) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    addresses = {a for a, _ in got}
    assert len(got) == 8 and addresses == {cfg.address()}
    del got
    gc.collect()
    other = [mx.Config(block=128).c() for _ in range(100)]   # would take a freed struct's place
    held = mx.mx_config.from_address(cfg.address())
    assert (held.block, held.seed) == (16, 77) and len(other) == 100
    s = mx.mx_sizes()
    assert mx.lib().mx_query_sizes(cfg.ref(), 4, 64, C.byref(s)) == 0 and s.n_scales == 16


def test_used_configurations_are_copied_and_pickled(mx):
    import copy
    import dataclasses
    import io
    import pickle

    import torch
    cfg = mx.Config(elem=mx.E2M3, block=16, seed=5)
    cfg.ref()
    for other in (pickle.loads(pickle.dumps(cfg)), copy.deepcopy(cfg), copy.copy(cfg), dataclasses.replace(cfg)):
        assert other == cfg and hash(other) == hash(cfg) and other is not cfg
        assert mx.mx_config.from_address(other.address()).seed == 5 and other.address() != cfg.address()
    assert vars(cfg) == dataclasses.asdict(cfg) and mx.Config(**vars(cfg)) == cfg
    with pytest.raises(dataclasses.FrozenInstanceError):
        cfg.block = 32
    # what holds one
    q = mx.Quantized(cfg, 2, 32, torch.arange(64, dtype=torch.uint8), torch.zeros(4, dtype=torch.uint8), None, None, None, None)
    file = io.BytesIO()
    torch.save(q, file)
    file.seek(0)
    for other in (copy.deepcopy(q), pickle.loads(pickle.dumps(q)), torch.load(file, weights_only=False)):
        assert other.cfg == cfg and torch.equal(other.codes, q.codes) and other.codes.data_ptr() != q.codes.data_ptr()


def given(mx):
    return mx.Config(block=16, scale_fmt=mx.SCALE_UE4M3, rule=mx.RULE_NEAREST, tensor_scale=mx.TS_GIVEN)


def small_cache(mx, cfg=None):
    import torch
    ts = dict(k_tensor_scale=torch.ones(1), v_tensor_scale=torch.ones(1)) if cfg and cfg.tensor_scale else {}
    return mx.kv_cache(2, 4, 1, 64, cfg or mx.MXFP4, device="cpu", **ts)


def pointers(c):
    s = c.ref()._obj
    return [s.k_codes, s.v_codes, s.k_scales, s.v_scales, s.k_tensor_scale, s.v_tensor_scale]


def held(c):
    return [t.data_ptr() for t in (c.k.codes, c.v.codes, c.k.scales, c.v.scales, c.k.tensor_scale, c.v.tensor_scale)]


def test_a_used_cache_follows_its_tensors(mx):
    """New buffers, tensor scales and sizes of a cache that was used are the ones of the next call."""
    import copy
    import pickle

    import torch
    c = small_cache(mx, given(mx))
    assert pointers(c) == held(c)
    c.k = copy.deepcopy(c.v)
    c.v.codes = c.v.codes.clone()
    c.v.tensor_scale = torch.ones(1)
    assert pointers(c) == held(c)
    for other in (copy.deepcopy(c), pickle.loads(pickle.dumps(c))):
        assert pointers(other) == held(other) and not set(held(other)) & set(held(c))


def calls(mx, c):
    import torch
    zeros = torch.zeros
    return [lambda: mx.kv_append(c, None, zeros(1, 64), zeros(1, 64), zeros(1, dtype=torch.int64)),
            lambda: mx.attn_decode(c, zeros(1, 1, 64), zeros(1, 2, dtype=torch.int32), zeros(1, dtype=torch.int32))]


@pytest.mark.parametrize("change,error,text", [
    (lambda c: setattr(c.k, "codes", c.k.codes[:100]), ValueError, "k: buffers too small"),
    (lambda c: setattr(c.v, "codes", c.v.codes.repeat(2)[::2]), ValueError, "v: buffers too small"),
    (lambda c: setattr(c.k, "scales", c.k.scales[:31]), ValueError, "k: buffers too small"),
    (lambda c: setattr(c, "pages", 3), ValueError, "buffers too small"),
    (lambda c: setattr(c, "head_dim", 128), ValueError, "buffers too small"),
    (lambda c: setattr(c.v, "tensor_scale", None), TypeError, "v: a float32 tensor scale"),
    (lambda c: setattr(c.k, "tensor_scale", c.k.tensor_scale.double()), TypeError, "k: a float32 tensor scale"),
    (lambda c: setattr(c.k, "tensor_scale", c.k.tensor_scale[:0]), TypeError, "k: a float32 tensor scale"),
])
def test_a_changed_cache_is_checked_at_every_call(mx, change, error, text):
    c = small_cache(mx, given(mx))
    for call in calls(mx, c):
        with pytest.raises(ValueError, match="CUDA"):        # all that is wrong before the change
            call()
    change(c)
    for call in calls(mx, c) + [c.ref]:
        with pytest.raises(error, match=text):
            call()


def test_a_cache_of_another_element_type_is_checked(mx):
    c = small_cache(mx)
    c.ref()
    c.cfg = mx.Config(elem=mx.E2M3)                          # a byte a code
    for call in calls(mx, c) + [c.ref]:
        with pytest.raises(ValueError, match="buffers too small"):
            call()


@pytest.mark.parametrize("dim", [0, -64])
def test_a_cache_without_a_head_length_is_refused(mx, dim):
    import torch
    c = small_cache(mx)
    c.head_dim = dim
    q = torch.zeros(1, 0)
    for call in calls(mx, c) + [lambda: mx.kv_append(c, q, q, q, torch.zeros(1, dtype=torch.int64)),
                                lambda: mx.attn_decode(c, q, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))]:
        with pytest.raises(ValueError, match="head_dim"):
            call()


def quantized(mx, cfg, rows=128, cols=256):
    import torch
    s = mx.query_sizes(cfg, rows, cols)
    z = lambda n, t=torch.uint8: torch.zeros(max(n, 1), dtype=t)  # noqa: E731
    return mx.Quantized(cfg, rows, cols, z(s.codes_bytes), z(s.n_scales), torch.ones(1), z(s.n_macro) if cfg.macro_block else None,
                        z(s.n_offsets, torch.int16) if cfg.asymmetric else None, None)


def cut(name, by=1):
    def change(q):
        t = getattr(q, name)
        setattr(q, name, t[:t.numel() - by])
    return change


def strided(name):
    def change(q):
        setattr(q, name, getattr(q, name).repeat_interleave(2)[::2])
    return change


@pytest.mark.parametrize("out", [False, True])
@pytest.mark.parametrize("cfg,change,error,text", [
    ({}, cut("codes"), ValueError, "codes must be contiguous and hold 16384"),
    ({}, cut("scales"), ValueError, "scales must be contiguous and hold 1024"),
    ({}, strided("codes"), ValueError, "codes must be contiguous"),
    (dict(elem=2), lambda q: setattr(q, "codes", q.codes[:16384]), ValueError, "codes must be contiguous and hold 32768"),
    (dict(axis=1), cut("scales"), ValueError, "scales must be contiguous and hold 1024"),
    (dict(axis=2), cut("scales"), ValueError, "scales must be contiguous and hold 32"),
    (dict(sf_layout=1), cut("scales"), ValueError, "scales must be contiguous and hold 1024"),
    (dict(macro_block=128), cut("macro"), ValueError, "macro must be contiguous and hold 256"),
    (dict(asymmetric=1), cut("offsets"), ValueError, "offsets must be contiguous and hold 2048"),
    (dict(block=16, scale_fmt=1, rule=3, tensor_scale=1), cut("tensor_scale"), TypeError, "tensor_scale must be float32"),
    (dict(block=16, scale_fmt=1, rule=3, tensor_scale=2), lambda q: setattr(q, "tensor_scale", q.tensor_scale.double()), TypeError,
     "tensor_scale must be float32"),
])
def test_dequantize_checks_its_buffers(mx, cfg, change, error, text, out):
    import torch
    q = quantized(mx, mx.Config(**cfg))
    more = dict(out=torch.zeros(128, 256)) if out else {}
    with pytest.raises(ValueError, match="codes must be a CUDA tensor"):         # all that is wrong before the change
        mx.dequantize(q, **more)
    change(q)
    with pytest.raises(error, match=text):
        mx.dequantize(q, **more)


def test_dequantize_checks_its_result(mx):
    import torch
    q = quantized(mx, mx.MXFP4)
    for bad in (torch.zeros(128, 255), torch.zeros(256, 128).T, torch.zeros(128, 512)[:, ::2]):
        with pytest.raises(ValueError, match="out must be contiguous"):
            mx.dequantize(q, out=bad)


def test_gemv_checks_its_tensor_scale(mx):
    import torch
    q = quantized(mx, given(mx), 64, 256)
    for change in (lambda: setattr(q, "tensor_scale", q.tensor_scale.double()), lambda: setattr(q, "tensor_scale", torch.ones(0))):
        with pytest.raises(ValueError, match="CUDA"):
            mx.gemv(torch.zeros(1, 256), quantized(mx, given(mx), 64, 256))
        change()
        with pytest.raises(TypeError, match="tensor_scale must be float32"):
            mx.gemv(torch.zeros(1, 256), q)


def test_a_binding_built_for_another_torch_is_not_loaded(mx, monkeypatch):
    import sysconfig

    import torch
    from microscaling_block_quantization_b200 import build
    assert build.up_to_date()
    mine = build.binding_path()
    assert torch.__version__ in mine and mine.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    monkeypatch.setattr(mx, "_compiled", None)
    assert mx._binding().__file__ == mine
    monkeypatch.setattr(mx, "_compiled", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert not build.up_to_date()
    with pytest.raises(RuntimeError, match="missing"):
        mx.gemv(torch.zeros(1, 256), quantized(mx, mx.MXFP4))


def test_dequantize_needs_no_binding(mx, monkeypatch):
    import torch
    monkeypatch.setattr(mx, "_compiled", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(ValueError, match="codes must be a CUDA tensor"):
        mx.dequantize(quantized(mx, mx.MXFP4))


def test_a_stream_of_another_device_is_refused(mx):
    import types

    import torch
    stream = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    zeros, c = torch.zeros, small_cache(mx)
    for call in (lambda: mx.gemv(zeros(1, 256), quantized(mx, mx.MXFP4), stream=stream),
                 lambda: mx.kv_append(c, None, zeros(1, 64), zeros(1, 64), zeros(1, dtype=torch.int64), stream=stream),
                 lambda: mx.attn_decode(c, zeros(1, 1, 64), zeros(1, 2, dtype=torch.int32), zeros(1, dtype=torch.int32), stream=stream)):
        with pytest.raises(ValueError, match="the stream is on cuda:1, expected cpu"):
            call()
