"""A semi-CRF tagger of token sequences, trained and then run on a stream.

    tokens -> embed -> [layer_norm -> decay_attention -> residual] x layers -> layer_norm
           -> emissions -> semi-CRF (nll for training, viterbi for tagging)

The encoder's cost is linear in the length, like the CRF's.  Training runs it over whole, ragged
sequences; tagging a stream runs it a token at a time, with one state a layer in a pool.

    python examples/tagger.py            # trains on synthetic segments, tags a stream
"""

from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import semi_markov_crf_amd as crf  # noqa: E402


class Tagger(torch.nn.Module):
    """Encoder and CRF parameters.  Head h of a layer forgets with a time constant of 2^(h + 1)
    positions."""

    def __init__(self, tokens, labels, max_segment, width=64, heads=4, layers=2, seed=0):
        super().__init__()
        gen = torch.Generator().manual_seed(seed)

        def param(*shape, sd):
            return torch.nn.Parameter(sd * torch.randn(*shape, generator=gen))

        self.width, self.heads = width, heads
        self.table = param(tokens, width, sd=width ** -0.5)
        self.layers = torch.nn.ModuleList()
        for _ in range(layers):
            layer = torch.nn.Module()
            layer.norm = torch.nn.Parameter(torch.ones(width))
            layer.qkv = param(width, 3 * width, sd=width ** -0.5)
            layer.out = param(width, width, sd=width ** -0.5 / layers)
            self.layers.append(layer)
        self.norm = torch.nn.Parameter(torch.ones(width))
        self.bias = torch.nn.Parameter(torch.zeros(width))
        self.emit = param(width, labels, sd=width ** -0.5)
        self.trans = torch.nn.Parameter(torch.zeros(labels, labels))
        self.dur = torch.nn.Parameter(torch.zeros(max_segment, labels))
        self.register_buffer("log_decay", -torch.exp2(-1.0 - torch.arange(heads, dtype=torch.float32)))

    def _split(self, y, layer):
        """q, k, v of a layer as views of one projection, [..., heads, width / heads]."""
        qkv = y @ layer.qkv
        return (x.unflatten(-1, (self.heads, -1)) for x in qkv.chunk(3, -1))

    def emissions(self, tokens, lengths):
        """[B, T, labels] for whole sequences; differentiable."""
        x = crf.embed(tokens, self.table, scale=math.sqrt(self.width), lengths=lengths)
        for layer in self.layers:
            q, k, v = self._split(crf.layer_norm(x, layer.norm, lengths=lengths), layer)
            o = crf.decay_attention(q, k, v, self.log_decay, lengths=lengths)
            x = x + o.flatten(-2) @ layer.out
        return crf.layer_norm(x, self.norm, self.bias, lengths=lengths) @ self.emit

    def loss(self, tokens, lengths, labels, seg_start):
        """Mean negative log-likelihood a position; leaves the gradients in .grad."""
        em = self.emissions(tokens, lengths)
        n = float(lengths.sum())
        out = crf.nll(em.detach(), lengths, self.trans.detach(), self.dur.detach(), labels, seg_start)
        em.backward(out["grad_em"] / n)
        self.trans.grad, self.dur.grad = out["grad_trans"] / n, out["grad_dur"] / n
        return float(out["nll"].sum()) / n

    @torch.no_grad()
    def tag(self, tokens, lengths):
        """Labels [B, T] (-1 at padding) of whole sequences."""
        em = self.emissions(tokens, lengths)
        return crf.viterbi(em, lengths, self.trans.detach(), self.dur.detach())[1]

    def new_pool(self, streams):
        """The states of `streams` streams, one array a layer."""
        d = self.width // self.heads
        return [torch.zeros(streams, self.heads, d, d, device=self.table.device) for _ in self.layers]

    @torch.no_grad()
    def step(self, token, pool, slots):
        """Emissions [B, labels] of the next token [B] of the streams in rows `slots` of the pool."""
        x = crf.embed(token[:, None].contiguous(), self.table, scale=math.sqrt(self.width))
        for layer, states in zip(self.layers, pool):
            q, k, v = self._split(crf.layer_norm(x, layer.norm)[:, 0], layer)
            o = crf.decay_attention_step(q, k, v, self.log_decay, states, slots=slots)
            x = x + (o.flatten(-2) @ layer.out)[:, None]
        return (crf.layer_norm(x, self.norm, self.bias) @ self.emit)[:, 0]


def synthetic(seed, B, T, tokens=8, labels=3, max_segment=24, device="cuda"):
    """Segments of random labels and lengths; each label prefers some tokens.  Returns tokens,
    lengths, labels and segment starts."""
    gen = torch.Generator().manual_seed(seed)
    lengths = torch.randint(T // 2, T + 1, (B,), generator=gen, dtype=torch.int32)
    tok = torch.randint(0, tokens, (B, T), generator=gen)
    lab = torch.full((B, T), -1, dtype=torch.int32)
    seg = torch.zeros(B, T, dtype=torch.uint8)
    for b in range(B):
        t, last = 0, -1
        while t < int(lengths[b]):
            k = min(int(torch.randint(4, max_segment + 1, (1,), generator=gen)), int(lengths[b]) - t)
            c = (last + 1 + int(torch.randint(0, labels - 1, (1,), generator=gen))) % labels
            own = torch.rand(k, generator=gen) < 0.4
            tok[b, t:t + k][own] = c
            lab[b, t:t + k], seg[b, t] = c, 1
            t, last = t + k, c
    return tuple(x.to(device) for x in (tok, lengths, lab, seg))


def main(steps=150, quiet=False):
    """Trains, tags, and runs a stream; returns (first loss, last loss, accuracy, largest difference
    of the streamed emissions)."""
    model = Tagger(tokens=8, labels=3, max_segment=24).cuda()
    opt = torch.optim.Adam(model.parameters(), lr=1e-2)
    first = last = None
    for i in range(steps):
        last = model.loss(*synthetic(i, B=16, T=300))
        opt.step()
        opt.zero_grad()
        first = last if first is None else first
        if not quiet and i % 25 == 0:
            print(f"step {i:4d}  nll a position {last:.4f}", flush=True)
    tok, lengths, lab, _ = synthetic(10_000, B=16, T=300)
    accuracy = float((model.tag(tok, lengths) == lab)[lab >= 0].float().mean())

    # the same sequences as streams: rows of the pool in another order
    B, T = tok.shape
    slots = torch.randperm(B, generator=torch.Generator().manual_seed(1)).to(tok.device, torch.int32)
    pool = model.new_pool(B)
    with torch.no_grad():
        whole = model.emissions(tok, torch.full_like(lengths, T))
    stream = torch.stack([model.step(tok[:, t], pool, slots) for t in range(T)], 1)
    off = float((stream - whole).abs().max())
    if not quiet:
        print(f"accuracy {accuracy:.3f}, streamed emissions off by {off:.1e}", flush=True)
    return first, last, accuracy, off


if __name__ == "__main__":
    main()
