"""More rows and tiles than workgroups: each takes several, and all of them are compared with the definitions."""

import numpy as np
import pytest

import blocks_ref as ref
from test_gpu_blocks import decays, dev, near, put, values
from test_gpu_encoder import crf  # noqa: F401

pytestmark = pytest.mark.gpu

ROWS = [  # rows, N, typ, wtyp, gate, norm_branch, center; workgroups forward and backward, a row at a time each
    (5300, 1024, "bf16", "bf16", True, True, True),          # 2,048 and 1,024 of two wavefronts
    (3000, 1030, "bf16", "f32", True, False, True),          # 1,280 and 768 of four
    (3200, 520, "f32", "f32", False, True, False),           # 1,536 and 512 of four
    (1200, 4100, "bf16", "bf16", True, True, False),         # 512 and 256 of eight, two pieces a lane
    (2200, 2048, "f32", "f32", True, False, True),           # 1,024 and 384 of eight
]


@pytest.mark.parametrize("case", ROWS, ids=lambda c: "-".join(map(str, c)))
def test_residual_norm_of_many_rows(crf, case):  # noqa: F811
    M, N, typ, wtyp, gated, post, center = case
    print(f"\n[residual rows {case}]", flush=True)
    rng = np.random.default_rng(M + N)
    x, o, gr, gy = (values(rng, (M, N), typ) for _ in range(4))
    z = values(rng, (M, N), typ) if gated else None
    w, b, c, bw, bb = (values(rng, N, wtyp, 0.1, mean) for mean in (1.0, 0.0, 0.5, 1.0, 0.0))
    if not post:
        bw = bb = None
    # few rows have gradients at first, so that the sums for the weights show every one of them
    some = np.sort(rng.choice(M, 40, replace=False))
    few = np.isin(np.arange(M), some)[:, None]

    def d3(v):
        return None if v is None else put(v[None], typ)

    kw = dict(gate=d3(z), norm_branch=post, center=center, scale=put(c, wtyp))
    if post:
        kw.update(branch_weight=put(bw, wtyp), branch_bias=put(bb, wtyp))
    xd, od, wd = d3(x), d3(o), put(w, wtyp)
    r, y, stats = crf.residual_norm(xd, od, wd, put(b, wtyp), want_stats=True, **kw)
    want, err = ref.residual(x, o, w, b, z, c, post, bw, bb, center, 1e-5, gr, gy)
    near(r[0], want["r"], err["r"], typ, "r")
    near(y[0], want["y"], err["y"], typ, "y")
    d = crf.residual_norm_grad(d3(gr), d3(gy), xd, od, wd, stats, **kw)
    for k in ("x", "branch") + (("gate",) if gated else ()):
        near(d["grad_" + k][0], want["grad_" + k], err["grad_" + k], typ, k)
    params = ("weight", "bias", "scale") + (("branch_weight", "branch_bias") if post else ())
    for k in params:
        near(d["grad_" + k], want["grad_" + k], err["grad_" + k], wtyp, k)
    d = crf.residual_norm_grad(d3(gr * few), d3(gy * few), xd, od, wd, stats, **kw)
    part = [None if v is None else v[some] for v in (x, o, z, gr, gy)]
    want, err = ref.residual(part[0], part[1], w, b, part[2], c, post, bw, bb, center, 1e-5, part[3], part[4])
    for k in params:
        near(d["grad_" + k], want["grad_" + k], err["grad_" + k], wtyp, k + " of a few rows")
    assert not d["grad_x"][0][dev(~few[:, 0])].any()


TILES = [  # B, T, N, typ: what decides how a gradient's tiles are served
    (30, 450, 513, "bf16"),      # one channel a lane, 510 chains: a workgroup a chain, three tiles each
    (16, 600, 1000, "bf16"),     # 256 chains, a last one of 40 channels
    (3, 12_000, 40, "bf16"),     # three chains of 94 tiles forward and 63 backward, a workgroup each
    (60, 5000, 70, "f32"),       # 120 chains of 40 and 27 tiles, 18 workgroups on each
]


@pytest.mark.parametrize("case", TILES, ids=lambda c: "-".join(map(str, c)))
def test_recurrence_of_many_tiles(crf, case):  # noqa: F811
    """All chains forward; gradients of a few sequences, the others' gradients are zero."""
    B, T, N, typ = case
    print(f"\n[recurrence tiles {case}]", flush=True)
    rng = np.random.default_rng(T + N)
    some = np.unique([0, B // 2, B - 1])
    lengths = rng.integers(T // 2, T + 1, B).astype(np.int32)
    lengths[some[-1]] = T
    x, r, i = (values(rng, (B, T, N), typ) for _ in range(3))
    g = np.zeros((B, T, N), np.float32)
    g[some] = values(rng, (len(some), T, N), typ)
    lam, state = decays(N, "spread"), rng.standard_normal((B, N)).astype(np.float32)
    gs = np.zeros((B, N), np.float32)
    gs[some] = rng.standard_normal((len(some), N))
    args, ln = [put(v, typ, lengths) for v in (x, r, i)] + [dev(lam)], dev(lengths)
    got, end, starts = crf.gated_recurrence(*args, lengths=ln, state=dev(state), want_state=True, want_starts=True)
    d = crf.gated_recurrence_grad(put(g, typ), *args, starts, lengths=ln, state=dev(state), grad_state=dev(gs))
    at = dev(some)
    h, last, eh, elast, _ = ref.recurrence(x[some], r[some], i[some], lam, lengths[some], state[some])
    near(got[at], h, eh, typ, "h")
    near(end[at], last, elast, "f32", "state")
    want, bound = ref.recurrence_grad(g[some], x[some], r[some], i[some], lam, lengths[some], state[some], gs[some])
    for k, v in want.items():
        near(d["grad_" + k] if k == "log_decay" else d["grad_" + k][at], v, bound[k],
             "f32" if k in ("log_decay", "state") else typ, k)
    # and the same bits again, whichever workgroup takes which tile
    import torch
    again = crf.gated_recurrence(*args, lengths=ln, state=dev(state), want_state=True)
    assert torch.equal(again[0], got) and torch.equal(again[1], end)
    e = crf.gated_recurrence_grad(put(g, typ), *args, starts, lengths=ln, state=dev(state), grad_state=dev(gs))
    assert all(torch.equal(d[k], e[k]) for k in d)
