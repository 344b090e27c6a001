"""Serving a small hybrid stack: gated-delta-rule layers that keep a state, and
softmax-attention layers that keep a paged key/value cache.

Several requests of different lengths are prefilled together, packed and in
chunks, then decoded one token per request and step. Every layer runs on the
library's kernels:

  delta-rule layer   prefill  gdn_chunk_fwd_fused (packed, states carried from
                              chunk to chunk)
                     decode   gdn_recurrent_step
  attention layer    both     gdn_paged_append, then gdn_paged_attn

Random weights; run as ``python examples/hybrid_serving.py`` (needs the built
library and a GPU). It decodes with the state and the cache, prefills the same
tokens again from nothing, and compares the two.
"""
from __future__ import annotations

import sys
from pathlib import Path

import torch
import torch.nn.functional as F

sys.path.insert(0, str(Path(__file__).resolve().parents[1]))

import gated_deltanet_chunkwise_gb300 as gdn  # noqa: E402


def rope_table(rows, rot, device, base=10000.0):
    """cos and sin of every position, made in fp64 and rounded once."""
    half = rot // 2
    freq = base ** (-torch.arange(half, dtype=torch.float64) / half)
    angle = torch.arange(rows, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(device)


class Pages:
    """Free list and page table of one pool, on the host as an engine has it."""

    def __init__(self, pool, page_size, requests, max_pages, device):
        self.page_size = page_size
        self.free = list(range(pool))
        self.count = [0] * requests
        self.table = torch.zeros((requests, max_pages), dtype=torch.int32,
                                 device=device)

    def grow(self, lens):
        for n, length in enumerate(lens):
            while self.count[n] * self.page_size < length:
                self.table[n, self.count[n]] = self.free.pop()
                self.count[n] += 1


class DeltaLayer:
    """Projection, gated delta rule (RMS-normalised, gated output), projection."""

    def __init__(self, width, heads, d, gen, device):
        new = lambda *s: torch.randn(s, generator=gen, device=device,
                                     dtype=torch.bfloat16) / s[0] ** 0.5
        self.heads, self.d = heads, d
        self.w_qkvz = new(width, 4 * heads * d)
        self.w_ab = new(width, 2 * heads).float()
        self.norm = torch.ones(d, device=device)
        self.w_out = new(heads * d, width)

    def start(self, requests, device):
        return torch.zeros((requests, self.heads, self.d, self.d), device=device)

    def project(self, x):
        q, k, v, z = (t.contiguous() for t in (x @ self.w_qkvz).view(
            *x.shape[:-1], 4, self.heads, self.d).unbind(-3))
        a, b = (t.contiguous() for t in (x.float() @ self.w_ab).view(
            *x.shape[:-1], 2, self.heads).unbind(-2))
        return q, k, v, z, a, b

    def prefill(self, x, state, cu):
        """x [1, tokens, width], packed by cu; returns (y, states)."""
        q, k, v, z, a, b = self.project(x)
        o, state = gdn.gdn_chunk_fwd_fused(q, k, v, a, b, state, cu,
                                           norm_weight=self.norm, gate=z)
        return o.flatten(-2) @ self.w_out, state

    def decode(self, x, state):
        """x [requests, width]; the state is updated in place."""
        q, k, v, z, a, b = self.project(x)
        unit = lambda t: F.normalize(t.float(), dim=-1, eps=0.0).to(t.dtype)
        o = gdn.gdn_recurrent_step(unit(q), unit(k), v, -F.softplus(a),
                                   torch.sigmoid(b), state).float()
        o = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + 1e-6) * self.norm
        o = (o * torch.sigmoid(z.float())).to(x.dtype)
        return o.flatten(-2) @ self.w_out


class AttentionLayer:
    """Projection, rotary softmax attention over the paged cache, projection."""

    def __init__(self, width, heads, kv_heads, d, pool, page_size, gen, device):
        new = lambda *s: torch.randn(s, generator=gen, device=device,
                                     dtype=torch.bfloat16) / s[0] ** 0.5
        self.heads, self.kv_heads, self.d = heads, kv_heads, d
        self.w_qkv = new(width, (heads + 2 * kv_heads) * d)
        self.w_out = new(heads * d, width)
        shape = (pool, kv_heads, page_size, d)
        self.k_cache = torch.zeros(shape, dtype=torch.bfloat16, device=device)
        self.v_cache = torch.zeros(shape, dtype=torch.bfloat16, device=device)

    def __call__(self, x, pages, lens, rope, cu=None):
        """x [B, T, width] (packed by cu, or one token per request)."""
        qkv = (x @ self.w_qkv).view(*x.shape[:2], -1, self.d)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 2)
        q = gdn.gdn_paged_append(q, k, v, self.k_cache, self.v_cache,
                                 pages.table, lens, cu, rope=rope, q_out=q)
        o = gdn.gdn_paged_attn(q, self.k_cache, self.v_cache, pages.table, lens,
                               cu)
        return o.flatten(-2) @ self.w_out


class HybridServer:
    """Three delta-rule layers to one attention layer, as hybrid stacks have
    them, serving a fixed set of requests."""

    def __init__(self, requests, max_len, *, width=512, blocks=2, vocab=1000,
                 page_size=16, device="cuda", seed=0):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        per = -(-max_len // page_size)
        self.device, self.vocab = device, vocab
        self.embed = torch.randn((vocab, width), generator=gen, device=device,
                                 dtype=torch.bfloat16)
        self.layers = []
        for _ in range(blocks):
            self.layers += [DeltaLayer(width, 4, 128, gen, device)
                            for _ in range(3)]
            self.layers.append(AttentionLayer(width, 8, 2, 128, requests * per,
                                              page_size, gen, device))
        self.pages = Pages(requests * per, page_size, requests, per, device)
        self.rope = rope_table(max_len, 64, device)  # half of each head turns
        self.states = [layer.start(requests, device)
                       if isinstance(layer, DeltaLayer) else None
                       for layer in self.layers]
        self.lens = torch.zeros(requests, dtype=torch.int32, device=device)
        self.length = [0] * requests

    def _grow(self, new):
        self.length = [a + b for a, b in zip(self.length, new)]
        self.pages.grow(self.length)
        self.lens.copy_(torch.tensor(self.length, dtype=torch.int32))

    def _norm(self, x):
        return F.rms_norm(x, x.shape[-1:])

    def prefill(self, chunks):
        """One chunk of tokens per request (some may be empty); returns the
        logits of all of them, packed."""
        new = [len(c) for c in chunks]
        self._grow(new)
        cu = torch.tensor([0] + new).cumsum(0).to(torch.int32).to(self.device)
        x = self.embed[torch.cat(chunks)][None]
        for i, layer in enumerate(self.layers):
            if isinstance(layer, DeltaLayer):
                y, self.states[i] = layer.prefill(self._norm(x), self.states[i], cu)
            else:
                y = layer(self._norm(x), self.pages, self.lens, self.rope, cu)
            x = x + y
        return self._norm(x)[0].float() @ self.embed.float().t()

    def decode(self, tokens):
        """One token per request; returns the logits [requests, vocab]."""
        self._grow([1] * len(tokens))
        x = self.embed[tokens]
        for i, layer in enumerate(self.layers):
            if isinstance(layer, DeltaLayer):
                y = layer.decode(self._norm(x), self.states[i])
            else:
                y = layer(self._norm(x)[:, None], self.pages, self.lens,
                          self.rope)[:, 0]
            x = x + y
        return self._norm(x).float() @ self.embed.float().t()


def serve(lengths=(70, 1, 200, 33), chunk=64, steps=12, seed=0, device="cuda",
          blocks=2):
    """Prefill in chunks and decode, then prefill everything at once; returns
    the decode steps' logits of both, [steps, requests, vocab]."""
    gen = torch.Generator(device=device)
    gen.manual_seed(seed + 1)
    most = max(lengths) + steps
    server = HybridServer(len(lengths), most, device=device, seed=seed,
                          blocks=blocks)
    prompts = [torch.randint(server.vocab, (n,), generator=gen, device=device)
               for n in lengths]
    last = [None] * len(lengths)
    for at in range(0, max(lengths), chunk):
        chunks = [p[at:at + chunk] for p in prompts]
        logits = server.prefill(chunks)
        ends = torch.tensor([len(c) for c in chunks]).cumsum(0).tolist()
        for n, c in enumerate(chunks):
            if len(c):
                last[n] = logits[ends[n] - 1]
    tokens = torch.stack(last).argmax(-1)
    said, stepped = [], []
    for _ in range(steps):
        said.append(tokens)
        stepped.append(server.decode(tokens))
        tokens = stepped[-1].argmax(-1)
    again = HybridServer(len(lengths), most, device=device, seed=seed,
                         blocks=blocks)
    whole = [torch.cat([p, torch.stack(said)[:, n]])
             for n, p in enumerate(prompts)]
    logits = again.prefill(whole)
    ends = torch.tensor([len(w) for w in whole]).cumsum(0).tolist()
    once = torch.stack([logits[e - steps:e] for e in ends], 1)
    assert gdn.gdn_device_status() == 0
    return torch.stack(stepped), once


def main():
    stepped, once = serve()
    off = ((stepped - once).norm() / once.norm()).item()
    same = (stepped.argmax(-1) == once.argmax(-1)).float().mean().item()
    print(f"{stepped.shape[0]} steps of {stepped.shape[1]} requests: chunked "
          f"prefill and decode against one prefill: logits differ by {off:.2e} "
          f"(2-norm), {100 * same:.0f} % of the tokens agree")


if __name__ == "__main__":
    main()
