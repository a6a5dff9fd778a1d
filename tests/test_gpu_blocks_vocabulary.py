"""The token loss over large vocabularies, where its sums are long."""

import numpy as np
import pytest

from blocks_ref import U
from test_gpu_encoder import crf  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_many_words_of_little_weight(crf, typ):  # noqa: F811
    """One word of score 0 and 2^20 - 1 whose exponentials are each below half a step of it, but 3 % of the sum
    together; as many rows as leave a row's vocabulary undivided.  A lane sees an eighth of the words at least,
    32 at a time, whose exponentials are summed (12 U of their sum) before they join: V / 256 additions of U each.
    The two constants to natural logarithms, the logarithm and the eight lanes' sums: 40 U."""
    import torch
    V, N, M = 2 ** 20, 64, 2 ** 16
    dt = torch.bfloat16 if typ == "bf16" else torch.float32
    print(f"\n[token_nll V={V} M={M} {typ}]", flush=True)
    x, table = torch.zeros(1, M, N, device="cuda", dtype=dt), torch.zeros(V, N, device="cuda", dtype=dt)
    x[..., 0] = 1.0
    table[:, 0] = -17.25
    top = 777_777
    table[top, 0] = 0.0
    t = torch.full((1, M), top, device="cuda", dtype=torch.int32)
    loss, lse = crf.token_nll(x, table, t, want_lse=True)
    want = np.log1p((V - 1) * np.exp(-17.25))
    # an exponential of 25 powers of two: its argument rounds by 25 U
    bound = (V / 256 + 12 + 40) * U + 30 * U * want
    for v in (loss, lse):
        assert float((v.double() - want).abs().max()) <= bound, (float(v[0, 0]), want)
