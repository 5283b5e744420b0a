"""Calls on a cache whose buffers were replaced after its first use go to the new ones."""
import copy

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


def test_replaced_buffers(mx):
    cfg = mx.Config(block=16, scale_fmt=mx.SCALE_UE4M3, rule=mx.RULE_NEAREST, tensor_scale=mx.TS_GIVEN)
    scales = [torch.tensor([x], device="cuda") for x in (0.01, 0.02)]
    c = mx.kv_cache(3, 16, 2, 64, cfg, k_tensor_scale=scales[0], v_tensor_scale=scales[1])
    k, v, q = (torch.randn(20, 2, 64, device="cuda").bfloat16() for _ in range(3))
    slots = torch.arange(20, device="cuda")
    table, n = torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda"), torch.tensor([20], dtype=torch.int32, device="cuda")
    mx.kv_append(c, None, k, v, slots)
    first = mx.attn_decode(c, q[:1], table, n)
    old, before = (c.k, c.v), copy.deepcopy((c.k, c.v))
    fresh = mx.kv_cache(3, 16, 2, 64, cfg, k_tensor_scale=scales[0] * 2, v_tensor_scale=scales[1] * 2)
    c.k, c.v = fresh.k, fresh.v
    mx.kv_append(c, None, k, v, slots)
    again = mx.attn_decode(c, q[:1], table, n)
    for t, u in zip(old, before):                            # left as they were
        assert torch.equal(t.codes, u.codes) and torch.equal(t.scales, u.scales)
    for t, x, s in ((c.k, k, scales[0] * 2), (c.v, v, scales[1] * 2)):
        want = mx.quantize(x.flatten(1), cfg, stats=False, tensor_scale=s)
        assert torch.equal(t.codes[:want.codes.numel()], want.codes) and torch.equal(t.scales[:want.scales.numel()], want.scales)
    kh, vh = (mx.dequantize(t)[:20].view(20, 2, 64).double() for t in (c.k, c.v))
    p = torch.softmax(torch.einsum("hd,lhd->hl", q[0].double(), kh) / 8, 1)
    want = torch.einsum("hl,lhd->hd", p, vh)
    # half a step of bf16, and the weights' 2^-12 of sum p |v|
    tol = want.abs() * 2.0 ** -8 + torch.einsum("hl,lhd->hd", p, vh.abs()) * 2.0 ** -11
    assert bool(((again[0].double() - want).abs() <= tol).all())
    assert torch.equal(first, again)                         # scales twice as large, scale codes half: the same values


def test_dequantize_without_the_compiled_binding(mx, monkeypatch):
    for cfg in (mx.MXFP4, mx.NVFP4, mx.Config(elem=mx.E2M3), mx.Config(axis=mx.AXIS_COL)):
        q = mx.quantize(torch.randn(64, 256, device="cuda").bfloat16(), cfg, stats=False)
        for dtype in (torch.float32, torch.bfloat16):
            want = mx.dequantize(q, dtype)
            with monkeypatch.context() as m:
                m.setattr(mx, "_compiled", None)
                m.setattr(torch, "__version__", "0.0.1")
                got = mx.dequantize(q, dtype)
            assert torch.equal(got, want)
