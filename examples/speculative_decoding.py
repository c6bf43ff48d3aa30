"""Speculative decoding of the decoder layer of decoder_layer.py with a tree of drafted
tokens: embedding -> the layer over all of a tree's tokens, each seeing its own path (append
and attention of a tree) -> output head -> a token sampled at every node -> the path
along which the drafts are what was sampled is kept, the cache compacted to it.  Several
samples of each prompt go on from one prefill (fork).

Drafts come from a table of the tokens that followed each token last.  A step is captured once as
a CUDA graph and replayed: lengths, drafts and accepted paths stay on the device.
Weights are random.

    python examples/speculative_decoding.py --prompts 4 --samples 2 --prompt 100 --steps 50
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from decoder_layer import DecoderLayer, Session  # noqa: E402
from quantized_moe_routed_gb300 import Nvfp4Linear, add_rms_norm, sample  # noqa: E402
from quantized_moe_routed_gb300.inputs import quantize_nvfp4  # noqa: E402
from quantized_moe_routed_gb300.layer import PAGE  # noqa: E402

# Each node's parent and which of that token's followers it drafts: three deep, the
# likelier branches longer.
PARENT = [-1, 0, 0, 1, 1, 2, 3, 3]
FOLLOWER = [0, 0, 1, 0, 1, 0, 0, 1]
DEPTH = 3


class Model:
    """A decoder layer between an embedding and an output head over V tokens."""

    def __init__(self, V=1000, seed=0, **layer):
        self.layer = DecoderLayer(seed=seed, **layer)
        gen = torch.Generator().manual_seed(seed + 1)
        H, dev = self.layer.H, self.layer.device
        self.V, self.embed = V, torch.randn((V, H), generator=gen).bfloat16().to(dev)
        self.norm = torch.ones(H, dtype=torch.bfloat16, device=dev)
        q, s, ts = quantize_nvfp4(torch.randn((V, H), generator=gen) * (4.0 / H ** 0.5))
        self.head = Nvfp4Linear(q.to(dev), s.to(dev), ts.reshape(1).float().to(dev))

    def __call__(self, tokens, q_off, kv_len, pages, max_q, parents=None):
        """tokens int64 [N] -> logits float32 [N, V]."""
        x = self.embed[tokens]
        residual = torch.zeros_like(x)
        y = self.layer(x, residual, q_off, kv_len, pages, max_q, parents=parents)
        return self.head(add_rms_norm(y, self.norm, residual=residual))


class Speculation:
    """C sequences that go on from B prompts, `samples` of each, decoded with trees."""

    def __init__(self, model: Model, prompts, samples: int, steps: int, temperature=0.7, top_p=0.9):
        """prompts int64 [B, n].  Room for `steps` steps of DEPTH + 1 tokens each."""
        self.model, self.settings = model, dict(temperature=temperature, top_p=top_p)
        cache, dev = model.layer.cache, model.layer.device
        B, n = prompts.shape
        longest = n + steps * (DEPTH + 1) + len(PARENT)
        s = Session(model.layer, B, longest)
        step = min(128, model.layer.experts.T_max // B)
        for at in range(0, n - 1, step):  # all but the last token, which is the first tree's root
            part = prompts[:, at:min(at + step, n - 1)]
            m = part.shape[1]
            s.kv_len += m
            model(part.reshape(-1), s.one * m, s.kv_len, s.pages, m)
        # the samples share the prompt's full pages; each has pages of its own from its partly filled one on
        C, width = B * samples, (longest + PAGE - 1) // PAGE
        src = torch.arange(C, device=dev) // samples
        first = (n - 1) // PAGE
        used = set(s.pages.flatten().tolist())
        free = torch.tensor([p for p in range(cache.n_pages) if p not in used], dtype=torch.int32, device=dev)
        own = width - first
        if C * own > len(free):
            raise ValueError(f"{C} samples of {own} pages each, {len(free)} are free")
        mine = free[:C * own].view(C, own)
        self.pages, self.kv_len = cache.fork(src.int(), mine[:, 0].contiguous(), s.kv_len, s.pages, model.layer.cache_ws)
        self.pages[:, first + 1:width] = mine[:, 1:]
        # one step's arrays
        k = len(PARENT)
        self.C, self.root = C, prompts[src, -1].clone()
        self.q_off = torch.arange(C + 1, dtype=torch.int32, device=dev) * k
        self.parent = torch.tensor(PARENT, device=dev)
        self.parents = torch.tensor(PARENT * C, dtype=torch.int32, device=dev)
        self.follower = torch.tensor(FOLLOWER, device=dev)
        self.table = torch.randint(0, model.V, (model.V, 2), device=dev)   # the last two tokens after each
        self.u = torch.zeros(C * k, device=dev)
        self.taken = torch.zeros((C, DEPTH + 1), dtype=torch.int64, device=dev)    # what the step gave: the first
        self.n_taken = torch.zeros(C, dtype=torch.int32, device=dev)               # n_taken of each row
        self.graph = None

    def step(self):
        """One tree for each sequence; between 1 and DEPTH + 1 tokens come of it."""
        model, C, k = self.model, self.C, len(PARENT)
        cache, ws = model.layer.cache, model.layer.cache_ws
        drafts = [self.root]
        for i in range(1, k):
            drafts.append(self.table[drafts[PARENT[i]], FOLLOWER[i]])
        tokens = torch.stack(drafts, 1)
        self.kv_len += k
        logits = model(tokens.view(-1), self.q_off, self.kv_len, self.pages, k, parents=self.parents)
        given = sample(logits, self.u, **self.settings).view(C, k).long()
        # from the root on: the child that drafts what was sampled, if there is one
        at = torch.zeros(C, dtype=torch.int64, device=self.root.device)
        keep, alive, count = [at], torch.ones_like(at, dtype=torch.bool), torch.ones_like(at)
        for _ in range(DEPTH):
            said = given.gather(1, at[:, None])
            child = (self.parent == at[:, None]) & (tokens == said) & alive[:, None]
            alive = child.any(1)
            at = torch.where(alive, child.int().argmax(1), at)
            keep.append(torch.where(alive, at, k))
            count = count + alive
        keep = torch.stack(keep, 1).int()
        self.n_taken.copy_(count)
        self.taken[:] = given.gather(1, keep.long().clamp(max=k - 1))
        for j in range(DEPTH + 1):  # drafts to come: what followed, the last first
            seen = tokens.gather(1, keep[:, j:j + 1].long().clamp(max=k - 1))[:, 0]
            new, was = self.taken[:, j], self.table[seen, 0]
            moves = (j < count) & (new != was)
            self.table[seen, 1] = torch.where(moves, was, self.table[seen, 1])
            self.table[seen, 0] = torch.where(moves, new, self.table[seen, 0])
        self.root.copy_(given.gather(1, at[:, None])[:, 0])
        step = (self.q_off, self.kv_len, self.pages, ws, k)
        self.kv_len.copy_(cache.compact(keep, self.n_taken, *step))

    def capture(self):
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.step()

    def run(self, steps):
        """Tokens of each sequence after `steps` steps: a list of lists."""
        out = [[] for _ in range(self.C)]
        for _ in range(steps):
            self.u.uniform_()
            if self.graph is None:
                self.step()
            else:
                self.graph.replay()
            for c, (row, m) in enumerate(zip(self.taken.tolist(), self.n_taken.tolist())):
                out[c] += row[:m]
        return out


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--prompts", type=int, default=4)
    ap.add_argument("--samples", type=int, default=2)
    ap.add_argument("--prompt", type=int, default=100)
    ap.add_argument("--steps", type=int, default=50)
    args = ap.parse_args()
    longest = args.prompt + args.steps * (DEPTH + 1) + len(PARENT)
    per = longest // PAGE + 2
    model = Model(n_pages=args.prompts * per * (1 + args.samples), positions=longest + len(PARENT),
                  T_max=max(args.prompts * 128, args.prompts * args.samples * len(PARENT)))
    spec = Speculation(model, torch.randint(0, model.V, (args.prompts, args.prompt), device=model.layer.device), args.samples, args.steps)
    spec.capture()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    out = spec.run(args.steps)
    end.record()
    status = model.layer.check()
    given = sum(map(len, out))
    print(f"status {status}, {spec.C} sequences, {given / spec.C / args.steps:.2f} tokens a step, "
          f"{start.elapsed_time(end) / args.steps * 1e3:.0f} us a step")
    return status


if __name__ == "__main__":
    sys.exit(main())
