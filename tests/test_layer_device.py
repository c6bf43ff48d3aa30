"""The layer operators launch on the current device: tensors or a stream of another
one are refused before anything is called.  The device is changed by pretending
(another number for the current device, a stand-in for the library that only counts
calls), so that nothing runs where it does not belong."""
import types

import pytest
import torch

from quantized_moe_routed_gb300 import KVCache, MoeError, Nvfp4Linear, add_rms_norm, binding, layer

DEV = "cuda:0"


class _Stream(types.SimpleNamespace):
    """What the binding reads of a stream."""


@pytest.mark.parametrize("current,tensors,stream,ok", [
    (0, 0, None, True), (0, 1, None, False), (1, 0, None, False), (1, 1, 1, True), (0, 0, 1, False), (1, 0, 0, False),
    (1, 1, 0, False)])
def test_stream_handles_belong_to_the_current_device(monkeypatch, current, tensors, stream, ok):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 100 + index, raising=False)
    dev = torch.device("cuda", tensors)
    st = None if stream is None else _Stream(device=torch.device("cuda", stream), cuda_stream=200 + stream)
    if ok:
        assert layer._handle(st, dev) == (100 + tensors if stream is None else 200 + stream)
        return
    with pytest.raises(MoeError) as ei:
        layer._handle(st, dev)
    assert ei.value.status == binding.MOE_ERR_INVALID_ARG


class _Recorder:
    """A library whose functions do nothing but count."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.mark.gpu
@pytest.mark.parametrize("wrong", ["tensors", "stream"])
def test_every_call_refuses_another_device(monkeypatch, wrong):
    x = torch.zeros((2, 128), dtype=torch.bfloat16, device=DEV)
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    lin = Nvfp4Linear(torch.zeros((16, 64), dtype=torch.uint8, device=DEV), torch.zeros((16, 8), dtype=torch.uint8, device=DEV),
                      torch.ones(1, device=DEV))
    cache = KVCache(2, 2, 1, 64)
    ws = cache.new_workspace()
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    step = (i32(0, 2), i32(2), torch.zeros((1, 1), dtype=torch.int32, device=DEV), ws, 2)
    q, k = x.view(2, 2, 64), torch.zeros((2, 1, 64), dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    if wrong == "tensors":
        st = None
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    else:
        st = _Stream(device=torch.device("cuda", 1), cuda_stream=0)
    rec = _Recorder()
    monkeypatch.setattr(layer, "_library", lambda: rec)
    # (outputs given where they can be, so that none is allocated under the pretended stream)
    out = torch.empty_like(x)
    calls = [lambda: add_rms_norm(x, w, out=out, stream=st), lambda: lin(x, out=torch.empty((2, 16), device=DEV), stream=st),
             lambda: cache.append(k, k, *step, stream=st), lambda: cache.attend(q, *step, out=out.view(2, 2, 64), stream=st),
             lambda: cache.check(ws, stream=st), lambda: cache.new_workspace(stream=st)]
    for call in calls:
        with pytest.raises(MoeError) as ei:
            call()
        assert ei.value.status == binding.MOE_ERR_INVALID_ARG
    assert rec.calls == []
