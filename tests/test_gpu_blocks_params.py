"""residual_norm: a parameter's gradient has the parameter's type and accuracy, whichever parameters there are."""

import numpy as np
import pytest

import blocks_ref as ref
from test_gpu_blocks import dev, near, put, values
from test_gpu_encoder import crf  # noqa: F401

pytestmark = pytest.mark.gpu

NAMES = ("weight", "bias", "scale", "branch_weight", "branch_bias")


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("wtyp", ["f32", "bf16"])
def test_one_parameter_alone(crf, name, wtyp):  # noqa: F811
    import torch
    rng = np.random.default_rng(NAMES.index(name))
    B, T, N, post = 2, 37, 72, name.startswith("branch")
    x, o, gr, gy = (values(rng, (B, T, N), "bf16") for _ in range(4))
    p = values(rng, N, wtyp, 0.1, 1.0)
    given = {k: p if k == name else None for k in NAMES}
    want, err = ref.residual(x, o, given["weight"], given["bias"], None, given["scale"], post, given["branch_weight"],
                             given["branch_bias"], True, 1e-5, gr, gy)
    leaf = put(p, wtyp).requires_grad_()
    args, kw = (put(x, "bf16"), put(o, "bf16")), dict(norm_branch=post)
    r, y = crf.residual_norm(*args, **{name: leaf}, **kw)
    grads = put(gr, "bf16"), put(gy, "bf16")
    d = torch.autograd.grad([r, y], leaf, grads)[0]
    assert d.dtype is leaf.dtype
    near(d, want["grad_" + name], err["grad_" + name], wtyp, name)
    # and from the gradient by itself, told the same parameter
    stats = crf.residual_norm(*args, **{name: leaf.detach()}, want_stats=True, **kw)[2]
    told = {name: leaf.detach(), **kw}
    e = crf.residual_norm_grad(*grads, *args, told.pop("weight", None), stats, **told)
    assert e["grad_" + name].dtype is leaf.dtype and torch.equal(e["grad_" + name], d)


def test_a_bias_of_another_type_is_refused(crf):  # noqa: F811
    import torch
    x, w = torch.randn(1, 3, 8, device="cuda").bfloat16(), torch.ones(8, device="cuda")
    stats = crf.residual_norm(x, x, w, want_stats=True)[2]
    with pytest.raises(TypeError):
        crf.residual_norm_grad(x, x, x, x, w, stats, bias=w.bfloat16())
    with pytest.raises(ValueError):
        crf.residual_norm_grad(x, x, x, x, w, stats, bias=w[:4])
