"""One decode step of an attention layer on block-scaled storage, run as it is
used: the fused projection (mx_gemv), norm, rotation and cache append
(mx_kv_append), attention over the cache (mx_attn_decode) and the output
projection (mx_gemv), several steps in a row, eager and captured, against the
same steps in binary64 on the dequantized weights and on the cache rows that
the steps wrote.  A stage is compared with the exact result of its own inputs,
to the rounding of its bf16 output (2^-8 relative to the row's largest terms)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

HQ, H, D, HID, PAGE, SEQS = 8, 2, 64, 512, 16, 3


@pytest.fixture(scope="module")
def mx():
    from microscaling_block_quantization_b200 import build
    build.build()
    import microscaling_block_quantization_b200 as m
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return m


class Layer:
    def __init__(self, mx, weight_cfg, cache_cfg):
        g = torch.Generator(device="cuda").manual_seed(3)
        w = torch.randn((HQ + 2 * H) * D, HID, generator=g, device="cuda") * HID ** -0.5
        o = torch.randn(HID, HQ * D, generator=g, device="cuda") * (HQ * D) ** -0.5
        self.wqkv, self.wo = (mx.quantize(t.bfloat16(), weight_cfg, stats=False) for t in (w, o))
        self.cache = mx.kv_cache(SEQS * 8, PAGE, H, D, cache_cfg)
        self.table = torch.randperm(SEQS * 8, generator=g, device="cuda").reshape(SEQS, 8).int()
        self.gq = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
        self.gk = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
        self.freq = torch.tensor([10000.0 ** (-2 * i / D) for i in range(D // 2)], device="cuda")
        self.lengths = torch.zeros(SEQS, dtype=torch.int32, device="cuda")

    def step(self, mx, x):
        """x: [SEQS, HID] bf16; every sequence grows by one token."""
        pos = self.lengths.long()
        slots = self.table.gather(1, (pos // PAGE)[:, None])[:, 0].long() * PAGE + pos % PAGE
        self.lengths += 1
        qkv = mx.gemv(x, self.wqkv)
        q, k, v = qkv.split([HQ * D, H * D, H * D], 1)
        qr, kr = mx.kv_append(self.cache, q, k, v, slots, pos, q_gain=self.gq, k_gain=self.gk, inv_freq=self.freq, k_out=True)
        a = mx.attn_decode(self.cache, qr, self.table, self.lengths)
        return qkv, qr, kr, slots, a, mx.gemv(a.flatten(1), self.wo)


def near(got, ref, mag, rel=2.0 ** -8):
    assert bool(((got.double() - ref).abs() <= rel * (ref.abs() + 0.25 * mag)).all()), float(((got.double() - ref).abs() / (ref.abs() + 0.25 * mag)).max())


def check_step(mx, layer, x, out):
    qkv, qr, kr, slots, a, y = out
    w, o = mx.dequantize(layer.wqkv).double(), mx.dequantize(layer.wo).double()
    near(qkv, x.double() @ w.T, (x.double().abs() @ w.abs().T) * 2.0 ** -6)
    pos = layer.lengths.double() - 1
    for src, got, n, gain in ((qkv[:, :HQ * D], qr, HQ, layer.gq), (qkv[:, HQ * D:(HQ + H) * D], kr, H, layer.gk)):
        z = src.double().view(SEQS, n, D)
        z = z / torch.sqrt((z * z).mean(-1, keepdim=True) + 1e-6) * gain.double()
        f = pos[:, None, None] * layer.freq.double()
        lo, hi = z.chunk(2, -1)
        near(got, torch.cat([lo * f.cos() - hi * f.sin(), hi * f.cos() + lo * f.sin()], -1),
             2.0 ** -12 * (lo.abs() + hi.abs()).repeat(1, 1, 2))
    for t, rows in ((layer.cache.k, kr.flatten(1)), (layer.cache.v, qkv[:, (HQ + H) * D:])):
        z = mx.quantize(rows.contiguous(), layer.cache.cfg, stats=False)
        n = layer.cache.pages * PAGE
        assert torch.equal(t.codes.view(n, -1)[slots], z.codes.view(SEQS, -1)) and torch.equal(t.scales.view(n, -1)[slots], z.scales.view(SEQS, -1))
    k, v = (mx.dequantize(t).double().view(-1, H, D) for t in (layer.cache.k, layer.cache.v))
    for b in range(SEQS):
        t = torch.arange(int(layer.lengths[b]), device="cuda")
        rows = layer.table[b].long()[t // PAGE] * PAGE + t % PAGE
        kb, vb = (z[rows].repeat_interleave(HQ // H, 1) for z in (k, v))
        p = torch.softmax(torch.einsum("hd,lhd->hl", qr[b].double(), kb) / math.sqrt(D), 1)
        # sum p |v| times 2^-11: the weights' rounding is 2^-12 of it; a score is off by e <= (64 / 16 + 16) 2^-23
        # sum |q k| / 8 < 20 2^-23 64 (heads of norm 8 sqrt(1.3)), so its exponential by 2 e < 2^-12
        near(a[b], torch.einsum("hl,lhd->hd", p, vb), torch.einsum("hl,lhd->hd", p, vb.abs()) * 2.0 ** -1)
    af = a.flatten(1).double()
    near(y, af @ o.T, (af.abs() @ o.abs().T) * 2.0 ** -6)


@pytest.mark.parametrize("weights,cache", [("mxfp4", "mxfp4"), ("nvfp4", "e2m3"), ("int4_g128", "int4")])
def test_steps(mx, weights, cache):
    wc = {"mxfp4": mx.MXFP4, "nvfp4": mx.NVFP4, "int4_g128": mx.Config(elem=mx.INT4, rule=mx.RULE_CEIL, asymmetric=1, block=128)}[weights]
    cc = {"mxfp4": mx.MXFP4, "e2m3": mx.Config(elem=mx.E2M3), "int4": mx.Config(elem=mx.INT4, rule=mx.RULE_CEIL)}[cache]
    layer = Layer(mx, wc, cc)
    g = torch.Generator(device="cuda").manual_seed(4)
    layer.lengths.copy_(torch.tensor([0, 15, 31], dtype=torch.int32))
    for _ in range(4):                                       # page borders inside
        x = torch.randn(SEQS, HID, generator=g, device="cuda").bfloat16()
        check_step(mx, layer, x, layer.step(mx, x))


def test_captured_steps(mx):
    """A captured step replayed gives what eager steps give, the cache included."""
    g = torch.Generator(device="cuda").manual_seed(4)
    xs = torch.randn(6, SEQS, HID, generator=g, device="cuda").bfloat16()
    eager, captured = Layer(mx, mx.MXFP4, mx.MXFP4), Layer(mx, mx.MXFP4, mx.MXFP4)
    want = [eager.step(mx, x)[-1] for x in xs]
    x = xs[0].clone()
    captured.step(mx, x)                                     # warm-up, then from the start again
    captured.lengths.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = captured.step(mx, x)[-1]
    captured.lengths.zero_()
    for i in range(6):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
    assert torch.equal(eager.cache.k.codes, captured.cache.k.codes) and torch.equal(eager.cache.v.codes, captured.cache.v.codes)


FIRST = """
import sys
sys.path.insert(0, {root!r})
import torch
import microscaling_block_quantization_b200 as mx
g = torch.Generator(device="cuda").manual_seed(0)
qw = mx.quantize(torch.randn(96, 256, generator=g, device="cuda").bfloat16(), mx.NVFP4, stats=False)
x = torch.randn(2, 256, generator=g, device="cuda").bfloat16()
c = mx.kv_cache(8, 16, 1, 64)
k = torch.randn(100, 64, generator=g, device="cuda").bfloat16()
slots = torch.arange(100, device="cuda")
q = torch.randn(1, 2, 64, generator=g, device="cuda").bfloat16()
table, n = torch.arange(8, device="cuda", dtype=torch.int32)[None], torch.tensor([100], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y = mx.gemv(x, qw)
    mx.kv_append(c, None, k, k, slots)
    a = mx.attn_decode(c, q, table, n)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(y, mx.gemv(x, qw)) and torch.equal(a, mx.attn_decode(c, q, table, n)) and float(a.float().abs().sum()) > 0
print("same")
"""


def test_first_calls_of_a_process_inside_a_capture(mx):
    """Nothing that a first call sets up is forbidden while a graph is captured."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=root)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
