"""The operators for speculative decoding together, as a decoding loop uses them: a tree's
append and attention, tokens sampled from the logits of what it gives, the compaction to a
path, a fork, and the decoding that goes on from there; eagerly and as a captured graph;
and the example that runs them with the experts."""
import math
import os
import sys

import pytest
import torch

import layer_reference as ref
import speculate_reference as spec
import test_gpu_layer_kv as base
import test_gpu_speculate_tree as trees
from conftest import ROOT
from quantized_moe_routed_gb300 import Nvfp4Linear, rope_table, sample
from quantized_moe_routed_gb300.inputs import quantize_nvfp4

sys.path.insert(0, os.path.join(ROOT, "examples"))
pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAGE = 64


def i32(*a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("n,L,Hq,Hkv,D", [(5, 40, 4, 2, 64), (20, 70, 8, 2, 128), (40, 150, 8, 1, 128)])
def test_a_step_from_tree_to_fork(n, L, Hq, Hkv, D):
    """Every stage against its definition, given what the stage before left."""
    B, V = 2, 600
    step = base.Step([n] * B, [L, L + 13], seed=n, spare=8, max_pages=(L + 13) // PAGE + 2)
    bufs = base._pool(step, Hkv, D, seed=n, exps=(-8, -6))
    used = set(step.pages.flatten().tolist())
    free = [p for p in range(step.n_pages) if p not in used]
    parents = spec.random_trees(step.ql, n)
    rope = rope_table(400, D, device=DEV)
    g = torch.Generator().manual_seed(n)
    qkv = torch.randn((step.N, Hq + 2 * Hkv, D), generator=g).bfloat16().to(DEV)
    w, s, ts = quantize_nvfp4(torch.randn((V, Hq * D), generator=g) * 0.3)
    head = Nvfp4Linear(w.to(DEV), s.to(DEV), ts.reshape(1).float().to(DEV))
    u = torch.rand(step.N, generator=g)
    cache = base._cache(bufs, Hq, Hkv, D, rope=rope)
    ws = cache.new_workspace()
    q_off, kv_len, pages = step.dev()
    args = (q_off, kv_len, pages, ws)
    q, k, v = qkv.split((Hq, Hkv, Hkv), dim=1)

    q = cache.append(k, v, *args, max_q=n, q=q, parents=parents.to(DEV))
    out = cache.attend(q, *args, max_q=n, parents=parents.to(DEV))
    now = tuple(t.cpu() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale))
    trees._check(step, now, q.cpu(), out, parents, 1 / math.sqrt(D))

    logits = head(out.view(step.N, -1))
    tokens = sample(logits, u.to(DEV), temperature=0.8, top_k=20, top_p=0.9)
    for i in range(step.N):
        want, _, near = spec.sample(logits[i].cpu(), float(u[i]), float(torch.tensor(0.8)), 20, float(torch.tensor(0.9)))
        assert int(tokens[i]) == want or near < 2.0 ** -34

    keeps = [sorted(spec.path(parents[b * n:(b + 1) * n].tolist(), n - 1)) for b in range(B)]
    table = torch.full((B, n), -1, dtype=torch.int32)
    for b, path in enumerate(keeps):
        table[b, :len(path)] = torch.tensor(path, dtype=torch.int32)
    lens = cache.compact(table.to(DEV), i32(*map(len, keeps)), *args, max_q=n)
    *want, wl = spec.compact(now, step.pages, step.q_off.tolist(), step.L, keeps, [len(p) for p in keeps])
    assert lens.tolist() == wl
    got = (ref.e4m3(cache.k.cpu()), ref.e4m3(cache.v.cpu()), cache.k_scale.cpu().double(), cache.v_scale.cpu().double())
    assert all(bool(((a == b) | (a.isnan() & b.isnan())).all()) for a, b in zip(got, want))

    # two samples of the first sequence and one of the second, a token more each
    new_pages, new_len = cache.fork(i32(0, 0, 1), i32(-1, free[0], free[1]), lens, pages, ws)
    kv = torch.randn((3, Hq + 2 * Hkv, D), generator=g).bfloat16().to(DEV)
    q, k, v = kv.split((Hq, Hkv, Hkv), dim=1)
    new_len = new_len + 1
    last = (i32(0, 1, 2, 3), new_len, new_pages, ws)
    need = [(x + PAGE - 1) // PAGE for x in new_len.tolist()]
    assert all(int(new_pages[c, m - 1]) >= 0 for c, m in enumerate(need))
    q = cache.append(k, v, *last, max_q=1, q=q)
    out = cache.attend(q, *last, max_q=1)
    assert cache.check(ws) == 0
    after = base.Step([1, 1, 1], new_len.tolist(), seed=0)
    after.pages = new_pages.cpu()
    now = tuple(t.cpu() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale))
    base._check_attend(after, now, q.cpu(), out, 1 / math.sqrt(D))


def _model(**kw):
    from speculative_decoding import Model
    return Model(V=500, n_pages=64, positions=512, T_max=256, **kw)


@pytest.mark.parametrize("prompts,samples,prompt", [(1, 1, 2), (1, 1, 65), (2, 3, 70), (3, 1, 129)])
def test_the_example_decodes(prompts, samples, prompt):
    from speculative_decoding import DEPTH, Speculation
    torch.manual_seed(prompt)
    model = _model()
    x = torch.randint(0, model.V, (prompts, prompt), device=DEV)
    s = Speculation(model, x, samples, steps=12)
    before = s.kv_len.clone()
    out = s.run(6)
    s.capture()
    out = [a + b for a, b in zip(out, s.run(6))]
    assert model.layer.check() == 0
    assert all(12 <= len(t) <= 12 * (DEPTH + 1) and all(0 <= a < model.V for a in t) for t in out)
    assert (s.kv_len - before).tolist() == [len(t) for t in out]     # every token but the last is in the cache, and the root


def test_a_captured_step_gives_what_an_eager_one_gives():
    from speculative_decoding import Speculation
    outs = []
    for captured in (False, True):
        torch.manual_seed(5)
        model = _model(seed=2)
        s = Speculation(model, torch.randint(0, model.V, (1, 40), device=DEV), 1, steps=20, temperature=0.5)
        if captured:
            s.capture()
        outs.append(s.run(20))
        assert model.layer.check() == 0
    assert outs[0] == outs[1]


def test_the_example_runs_from_the_command_line(monkeypatch, capsys):
    import speculative_decoding
    monkeypatch.setattr(sys, "argv", ["speculative_decoding.py", "--prompts", "2", "--samples", "2", "--prompt", "30", "--steps", "5"])
    assert speculative_decoding.main() == 0
    assert "status 0" in capsys.readouterr().out
