"""The pretraining example: embedding, gated recurrence, residual norm, token loss and the CRF together,
trained for a few steps and run token by token."""

import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("pretrain", os.path.join(ROOT, "examples", "pretrain.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_pretraining_training_and_streaming_run():
    before, after, accuracy, off = load().main(pretrain=6, train=6, quiet=True)
    print(f"\n[pretrain] {before[0]:.4f} {before[-1]:.4f}, {after[0]:.4f} {after[-1]:.4f}, {accuracy:.3f}, {off:.1e}")
    assert len(before) == len(after) == 6 and all(math.isfinite(v) for v in before + after)
    # normalised rows of order 1 from sums of 64 products through two layers, and states that a stream
    # rounds once a token and whole sequences once a tile: fp32 rounding, 2^-24 times a few thousand
    assert off < 1e-3


@pytest.mark.parametrize("which", ["next_token", "tag"])
def test_gradients_against_differences(which):
    """The losses' derivatives along the gradient of the parameters."""
    import torch
    p = load()
    model = p.Encoder(tokens=8, labels=3, max_segment=24, width=32, layers=2).cuda()
    data = p.synthetic(3, B=4, T=120)

    def loss():
        if which == "tag":
            model.zero_grad()
            return model.tag_loss(*data)
        return float(model.next_token_loss(*data[:2]))

    loss()
    if which == "next_token":
        model.zero_grad()
        model.next_token_loss(*data[:2]).backward()
    params = [q for q in model.parameters() if q.grad is not None]
    assert len(params) >= 14                          # all of the encoder's
    grads = [q.grad.clone() for q in params]
    # along the gradient the slope is its norm, far above the rounding of the loss (fp32, about 1e-6 a
    # position); the curvature's share of a central difference is of order h^2
    norm = float(sum((g ** 2).sum() for g in grads)) ** 0.5
    h, ends = 1e-2, []
    for s in (1, -1):
        with torch.no_grad():
            for q, g in zip(params, grads):
                q.add_(g / norm, alpha=s * h)
        ends.append(loss())
        with torch.no_grad():
            for q, g in zip(params, grads):
                q.add_(g / norm, alpha=-s * h)
    slope = (ends[0] - ends[1]) / (2 * h)
    assert abs(slope - norm) < 2e-2 * norm, (slope, norm)
