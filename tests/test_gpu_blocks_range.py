"""The token loss's gradients in bfloat16 over the range that the numbers entering their products keep."""

import numpy as np
import pytest

from blocks_ref import U
from test_gpu_blocks import dev, near, put
from test_gpu_encoder import crf, host  # noqa: F401

pytestmark = pytest.mark.gpu


def plain(x, table, t, scale, g):
    z = scale * (x @ table.T)
    top = z.max(1, keepdims=True)
    lse = top[:, 0] + np.log(np.exp(z - top).sum(1))
    p = np.exp(z - lse[:, None])
    e = p.copy()
    p[np.arange(len(x)), t] -= 1.0
    gs = (scale * g)[:, None]
    return z, lse, e, p, gs * (p @ table), (gs * p).T @ x


def held(v, top):
    """What fp16 may be off by at v where the largest value, `top`, is brought to 2^14 or more: half a step of 11 bits
    down to 2^-28 of it, and half of the smallest step below."""
    return np.maximum(2.0 ** -11 * np.abs(v), 2.0 ** -39 * top)


@pytest.mark.parametrize("case", [(50, 40, 300), (300, 72, 700), (600, 130, 90)], ids=str)
def test_gradients_keep_their_range(crf, case):  # noqa: F811
    """Columns of x and of the table down to 2^-27 of the largest, row gradients over 2^20, words whose probability
    falls to 2^-60: gradients to within the rounding of what enters the products, element by element.  p, at most 1
    and brought to 2^15, is held from 2^-40 on, in 11 bits from 2^-29 on; the table exactly to 2^-28 of its largest
    value; x times the row's gradient as fp16 below the largest |x| times the largest gradient."""
    M, N, V = case
    rng = np.random.default_rng(M)

    def exact(v):
        return host(put(v, "bf16"))

    down = np.exp2(-np.linspace(0.0, 27.0, N))
    x = exact(rng.standard_normal((M, N)) * down)
    table = exact(rng.standard_normal((V, N)) * down)
    # the first two columns make the scores: from 0 down to -41 (2^-60)
    x[:, 0], x[:, 1] = 1.0, exact(rng.uniform(-0.5, 0.5, M))
    table[:, 0] = exact(-np.linspace(0.0, 41.0, V)[rng.permutation(V)])
    t = rng.integers(0, V, M).astype(np.int32)
    g = (rng.choice([-1.0, 1.0], M) * np.exp2(rng.uniform(-20.0, 0.0, M))).astype(np.float32)
    g[0] = 1.0
    z, lse, e, p, dx, dW = plain(x, table, t, 1.0, g.astype(np.float64))
    args = [put(x[None], "bf16"), put(table, "bf16"), dev(t[None])]
    glse = crf.token_nll(*args, want_lse=True)[1]
    d = crf.token_nll_grad(dev(g[None]), *args, glse)
    # p before it is held: scores of up to 45 summed in fp32 and scaled, a log sum to the same, an exponential
    depth = N / 32 + 100
    ez = U * (depth + 8) * (np.abs(x) @ np.abs(table).T) + U * 4 * (np.abs(z) + np.abs(lse)[:, None]) + 60 * U
    ep = e * ez + held(p, 0.5) + 2.0 ** -126
    sums = (depth + V / 32 + M / 32) * U
    ga, xa, wa = np.abs(g)[:, None].astype(np.float64), np.abs(x), np.abs(table)
    wh = np.where(wa >= 2.0 ** -28 * wa.max(), 0.0, 2.0 ** -39 * wa.max())
    edx = ga * (ep @ wa + np.abs(p) @ wh + sums * (np.abs(p) @ wa))
    xg = ga * xa
    exg = held(xg, xa.max() * ga.max())        # one scale for all rows, from the two maxima
    edW = ep.T @ (xg + exg) + np.abs(p).T @ exg + sums * (np.abs(p).T @ xg)
    near(d["grad_x"][0], dx, edx, "bf16", "grad_x")
    near(d["grad_table"], dW, edW, "bf16", "grad_table")
