"""The decoder layer of examples/decoder_layer.py: the operators together.

Against 64-bit arithmetic without the cache's rounding: a code is off by up to
2^-4 of its value, about 2.6 % root mean square, and scores of order 1 move
weights by as much; the attention's output is then off by a few per cent, 10 %
at most in the Frobenius norm.  What follows each stage is compared given the
stage's own inputs, so that no expert choice hangs on the rounding."""
import os
import sys

import pytest
import torch

import layer_reference as ref
from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))
pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _reference_attention(layer, x):
    """x bfloat16 [n, H] of one sequence -> the output projection's result [n, H]."""
    hq, hkv, d = layer.heads
    n = x.shape[0]
    _, h = ref.norm(x.cpu(), None, layer.norm1.cpu(), 1e-6)

    def weights(lin):
        return ref.nvfp4(lin.q.cpu(), lin.s.cpu()) * lin.ts.cpu().double()[:, None]
    t = (h @ weights(layer.qkv).T).view(n, hq + 2 * hkv, d)
    rope = layer.cache.rope[:n].cpu()
    t[:, :hq + hkv] = ref.rotate(t[:, :hq + hkv], rope, False)
    o = torch.zeros((n, hq, d), dtype=torch.float64)
    g = hq // hkv
    for kv in range(hkv):
        o[:, kv * g:(kv + 1) * g] = ref.attend(t[:, kv * g:(kv + 1) * g], t[:, hq + kv], t[:, hq + hkv + kv], n, n, d ** -0.5)[0]
    return o.view(n, -1) @ weights(layer.out).T


@pytest.mark.parametrize("n,head_dim,q_heads,kv_heads", [(1, 64, 8, 2), (75, 64, 8, 2), (140, 128, 4, 4)])
def test_prompt_through_the_layer(n, head_dim, q_heads, kv_heads):
    from decoder_layer import DecoderLayer, Session
    layer = DecoderLayer(head_dim=head_dim, q_heads=q_heads, kv_heads=kv_heads, seed=3)
    x = torch.randn((n, layer.H), generator=torch.Generator().manual_seed(n)).bfloat16().to(DEV)
    s = Session(layer, 1, 256)
    s.kv_len += n
    r = torch.zeros_like(x)
    y = layer(x, r, s.one * n, s.kv_len, s.pages, n)
    assert layer.check() == 0 and torch.isfinite(y).all()
    want = x.cpu().double() + _reference_attention(layer, x)
    err = (r.cpu().double() - want).norm() / (want - x.cpu().double()).norm()
    assert err < 0.1, float(err)
    # the experts' inputs, from the residual that the layer left
    _, h = ref.norm(r.cpu(), None, layer.norm2.cpu(), 1e-6)
    h = h.bfloat16()
    logits = layer.router(h.to(DEV))
    torch.testing.assert_close(logits.cpu().double(), h.double() @ (ref.nvfp4(layer.router.q.cpu(), layer.router.s.cpu()) *
                               layer.router.ts.cpu().double()[:, None]).T, rtol=2 ** -10, atol=2 ** -10)


def test_captured_decode_equals_eager_and_chunks_carry_on():
    from decoder_layer import DecoderLayer, Session
    layer = DecoderLayer(seed=5)
    s = Session(layer, 3, 200)
    gen = torch.Generator().manual_seed(1)
    s.prefill(torch.randn((3, 130, layer.H), generator=gen).bfloat16().to(DEV), chunk=50)
    assert layer.check() == 0 and s.kv_len.tolist() == [130] * 3
    state = [t.clone() for t in (layer.cache.k, layer.cache.v, layer.cache.k_scale, layer.cache.v_scale, s.kv_len)]
    xs = torch.randn((5, 3, layer.H), generator=gen).bfloat16().to(DEV)
    eager = [s.decode(x, torch.zeros_like(x)).clone() for x in xs]
    assert s.kv_len.tolist() == [135] * 3
    for t, old in zip((layer.cache.k, layer.cache.v, layer.cache.k_scale, layer.cache.v_scale, s.kv_len), state):
        t.copy_(old)
    s.capture()
    for x, want in zip(xs, eager):
        s.x.copy_(x)
        s.graph.replay()
        assert torch.equal(s.y, want)
    assert layer.check() == 0 and s.kv_len.tolist() == [135] * 3


def test_the_command_runs(capsys, monkeypatch):
    import decoder_layer
    monkeypatch.setattr(sys, "argv", ["decoder_layer.py", "--batch", "2", "--prompt", "70", "--tokens", "4"])
    assert decoder_layer.main() == 0
    assert "status 0, 2 sequences of 74 tokens" in capsys.readouterr().out
