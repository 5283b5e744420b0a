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
