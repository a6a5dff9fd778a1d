"""residual_norm's gradients are asked for in the type of the parameters there are, be it the bias alone; on the
CPU, with a stand-in for the library."""

import pytest
import torch

import semi_markov_crf_amd as crf
from semi_markov_crf_amd import _native
from test_current_device import array, calls  # noqa: F401


@pytest.mark.parametrize("name", ["weight", "bias", "scale", "branch_weight", "branch_bias"])
@pytest.mark.parametrize("typ", [torch.float32, torch.bfloat16])
def test_type_of_the_gradients(calls, monkeypatch, name, typ):  # noqa: F811
    asked = []
    monkeypatch.setattr(_native, "call", lambda dev, fn, a, *rest: asked.append((fn, a.wdtype)) or 0)
    x, p = array(2, 3, 8, dtype=torch.bfloat16), array(8, dtype=typ)
    kw = {name: p, "norm_branch": True, "workspace": array(1 << 13, dtype=torch.uint8)}
    kw["workspace"] = kw["workspace"][-kw["workspace"].data_ptr() % 256:]
    d = crf.residual_norm_grad(x, x, x, x, kw.pop("weight", None), array(2, 3, 4), **kw)
    assert asked == [("semicrf_residual_norm_grad", _native.F32 if typ is torch.float32 else _native.BF16)]
    assert d["grad_" + name].dtype is typ
