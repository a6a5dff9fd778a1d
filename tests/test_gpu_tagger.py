"""The example tagger: every encoder operator and the CRF together, trained for a few steps,
then run token by token."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    spec = importlib.util.spec_from_file_location("tagger", os.path.join(ROOT, "examples", "tagger.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_tagger_learns_and_streams():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    first, last, accuracy, off = load().main(steps=60, quiet=True)
    print(f"\n[tagger] nll {first:.4f} -> {last:.4f}, accuracy {accuracy:.3f}, streamed off by {off:.1e}")
    # a tagger that knows nothing gets a third of the labels right
    assert last < 0.8 * first and accuracy > 0.6
    # emissions are sums of 64 products of order 1 from states of some hundred terms: fp32 rounding
    # through two layers, 2^-24 times a few thousand
    assert off < 1e-3


def test_tagger_gradients_against_differences():
    """The loss's derivative along a random direction of the encoder's parameters."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    t = load()
    model = t.Tagger(tokens=8, labels=3, max_segment=24, width=32, heads=2, layers=1).cuda()
    data = t.synthetic(3, B=4, T=120)
    model.loss(*data)
    params = list(model.parameters())
    grads = [p.grad.clone() for p in params]
    torch.manual_seed(0)
    # along the gradient: the slope is its norm, far above the rounding of the loss (fp32, about
    # 1e-6 a position), and the curvature's share of a central difference is of order h^2
    norm = float(sum((g ** 2).sum() for g in grads)) ** 0.5
    h, ends = 1e-2, []
    for s in (1, -1):
        with torch.no_grad():
            for p, g in zip(params, grads):
                p.add_(g / norm, alpha=s * h)
        ends.append(model.loss(*data))
        with torch.no_grad():
            for p, g in zip(params, grads):
                p.add_(g / norm, alpha=-s * h)
    slope = (ends[0] - ends[1]) / (2 * h)
    assert abs(slope - norm) < 2e-2 * norm, (slope, norm)
