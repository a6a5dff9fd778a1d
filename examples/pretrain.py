"""An encoder pretrained on unlabelled tokens, then trained as a semi-CRF tagger, then run on a stream.

    tokens -> embed -> layer_norm -> [gated_recurrence -> residual_norm] x layers
           -> token_nll over the embedding's own table     (the next token: no labels needed)
           -> emissions -> semi-CRF                        (nll for training, viterbi for tagging)

A block is one projection to the recurrence's input, its two gates and the gate of what it adds, the
recurrence, and a residual norm that ends the block and starts the next.

    python examples/pretrain.py            # pretrains and trains on synthetic segments, tags a stream
"""

from __future__ import annotations

import math
import os
import sys

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
for path in (HERE, os.path.dirname(HERE)):
    if path not in sys.path:
        sys.path.insert(0, path)
import semi_markov_crf_amd as crf  # noqa: E402
from tagger import synthetic  # noqa: E402


class Encoder(torch.nn.Module):
    """Channels of a layer forget, at an open gate, with time constants from 2 to 128 positions."""

    def __init__(self, tokens, labels, max_segment, width=64, layers=2, seed=0):
        super().__init__()
        gen = torch.Generator().manual_seed(seed)

        def param(*shape, sd):
            return torch.nn.Parameter(sd * torch.randn(*shape, generator=gen))

        self.width = width
        self.table = param(tokens, width, sd=width ** -0.5)
        self.first = torch.nn.Parameter(torch.ones(width))
        self.layers = torch.nn.ModuleList()
        for _ in range(layers):
            layer = torch.nn.Module()
            layer.into = param(width, 4 * width, sd=width ** -0.5)
            layer.out = param(width, width, sd=width ** -0.5)
            # log_decay = -exp(rate): learned, and below 0
            layer.rate = torch.nn.Parameter(-math.log(2.0) * (1.0 + 6.0 * torch.arange(width) / max(1, width - 1)))
            layer.scale = torch.nn.Parameter(torch.full((width,), 0.5))
            layer.norm = torch.nn.Parameter(torch.ones(width))
            layer.bias = torch.nn.Parameter(torch.zeros(width))
            self.layers.append(layer)
        self.emit = param(width, labels, sd=width ** -0.5)
        self.trans = torch.nn.Parameter(torch.zeros(labels, labels))
        self.dur = torch.nn.Parameter(torch.zeros(max_segment, labels))

    def forward(self, tokens, lengths):
        """[B, T, width]: the normalised residual stream."""
        r = crf.embed(tokens, self.table, scale=math.sqrt(self.width), lengths=lengths)
        y = crf.layer_norm(r, self.first, lengths=lengths)
        for layer in self.layers:
            x, decay, into, out = (y @ layer.into).chunk(4, -1)
            h = crf.gated_recurrence(x, decay, into, -torch.exp(layer.rate), lengths=lengths)
            r, y = crf.residual_norm(r, h @ layer.out, layer.norm, layer.bias, gate=out, scale=layer.scale,
                                     lengths=lengths)
        return y

    def next_token_loss(self, tokens, lengths):
        """Mean negative log-likelihood of each sequence's next token; differentiable."""
        t = torch.arange(tokens.shape[1], device=tokens.device)
        targets = torch.where(t + 1 < lengths[:, None], tokens.roll(-1, 1), -1)
        loss = crf.token_nll(self(tokens, lengths), self.table, targets, lengths=lengths)
        return loss.sum() / (targets >= 0).sum().clamp(min=1)

    def tag_loss(self, tokens, lengths, labels, seg_start):
        """Mean negative log-likelihood of a segmentation a position; leaves the gradients in .grad."""
        em = self(tokens, lengths) @ self.emit
        n = float(lengths.sum())
        out = crf.nll(em.detach(), lengths, self.trans.detach(), self.dur.detach(), labels, seg_start)
        em.backward(out["grad_em"] / n)
        self.trans.grad, self.dur.grad = out["grad_trans"] / n, out["grad_dur"] / n
        return float(out["nll"].sum()) / n

    def new_pool(self, streams):
        """The states of `streams` streams, one array a layer."""
        return [torch.zeros(streams, self.width, device=self.table.device) for _ in self.layers]

    @torch.no_grad()
    def step(self, token, pool, slots):
        """The residual stream [B, width] at the next token [B] of the streams in rows `slots` of the pool."""
        r = crf.embed(token[:, None].contiguous(), self.table, scale=math.sqrt(self.width))
        y = crf.layer_norm(r, self.first)
        for layer, states in zip(self.layers, pool):
            x, decay, into, out = (y @ layer.into).chunk(4, -1)
            h = crf.gated_recurrence_step(x[:, 0], decay[:, 0], into[:, 0], -torch.exp(layer.rate), states, slots=slots)
            r, y = crf.residual_norm(r, (h @ layer.out)[:, None], layer.norm, layer.bias, gate=out, scale=layer.scale)
        return y[:, 0]


def main(pretrain=60, train=100, quiet=False):
    """Pretrains, trains, tags, and runs a stream; returns (next-token losses, tagging losses, accuracy,
    largest difference of the streamed residual stream)."""
    model = Encoder(tokens=8, labels=3, max_segment=24).cuda()
    opt = torch.optim.Adam(model.parameters(), lr=1e-2)
    before, after = [], []
    for i in range(pretrain):
        tok, lengths, _, _ = synthetic(50_000 + i, B=16, T=300)
        loss = model.next_token_loss(tok, lengths)
        opt.zero_grad()
        loss.backward()
        opt.step()
        before.append(float(loss.detach()))
        if not quiet and i % 20 == 0:
            print(f"pretraining step {i:4d}  nll a token {before[-1]:.4f}", flush=True)
    for i in range(train):
        opt.zero_grad()
        after.append(model.tag_loss(*synthetic(i, B=16, T=300)))
        opt.step()
        if not quiet and i % 20 == 0:
            print(f"step {i:4d}  nll a position {after[-1]:.4f}", flush=True)
    tok, lengths, lab, _ = synthetic(10_000, B=16, T=300)
    with torch.no_grad():
        whole = model(tok, torch.full_like(lengths, tok.shape[1]))
        tags = crf.viterbi(model(tok, lengths) @ model.emit, lengths, model.trans.detach(), model.dur.detach())[1]
    accuracy = float((tags == lab)[lab >= 0].float().mean())
    # the same sequences as streams: rows of the pool in another order
    slots = torch.randperm(len(tok), generator=torch.Generator().manual_seed(1)).to(tok.device, torch.int32)
    pool = model.new_pool(len(tok))
    stream = torch.stack([model.step(tok[:, t], pool, slots) for t in range(tok.shape[1])], 1)
    off = float((stream - whole).abs().max())
    if not quiet:
        print(f"accuracy {accuracy:.3f}, streamed off by {off:.1e}", flush=True)
    return before, after, accuracy, off


if __name__ == "__main__":
    main()
