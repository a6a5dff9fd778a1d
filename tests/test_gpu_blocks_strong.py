"""Gated recurrence where decays are strong: what a position leaves of a large state is small and has to be
right by its own size, and so has what follows it.

Bounds as in tests/blocks_ref.py, but for what a decay of more than 1/4 (s < -1/4) makes of the state:
a = exp(s) is within (|s| (G(r) + 3) + 4) U of itself (the gate's error, the exponent's product, the
exponential); where positions are joined, s is summed over up to 8 of them and the product's exponent
rounds once more, |s| (8 + 4) U a position, and products of joined stretches round by 4 U, of which there
are fewer than positions.  All of it scales with what is left, a |h|, not with |h|."""

import numpy as np
import pytest

from blocks_ref import FLUSHED, G, U, gates
from test_gpu_blocks import dev, near
from test_gpu_encoder import crf, draw_lengths, host  # noqa: F401

pytestmark = pytest.mark.gpu


def kept(s, r, a, m, em):
    """Relative to the state before a position, the error [U] of what the position leaves of it."""
    return np.where(s >= -0.25, em * np.abs(m), (np.abs(s) * (G(r) + 15) + 8) * a + FLUSHED)


def recurrence(x, r, i, lam, lengths, state):
    """h, final state, the states before each position, and their bounds [U]."""
    B, T, N = x.shape
    h, eh, before, ebefore = (np.zeros((B, T, N)) for _ in range(4))
    v, e = state.astype(np.float64), np.zeros((B, N))
    w = np.abs(v)
    for t in range(T):
        on = (t < lengths)[:, None]
        before[:, t], ebefore[:, t] = v, e
        _, si, s, a, m, bb, _, em, _, ebu = gates(x[:, t], r[:, t], i[:, t], lam)
        u = bb * si * x[:, t]
        ne = a * e + kept(s, r[:, t], a, m, em) * w + ebu * np.abs(u)
        nw = a * w + np.abs(u)
        v, w, e = np.where(on, a * v + u, v), np.where(on, nw, w), np.where(on, ne + 2 * nw, e)
        h[:, t], eh[:, t] = np.where(on, v, 0.0), np.where(on, e, 0.0)
    return h, v, before, eh, e, ebefore


def recurrence_grad(g, x, r, i, lam, lengths, state, grad_state):
    B, T, N = x.shape
    _, _, before, _, _, ebefore = recurrence(x, r, i, lam, lengths, state)
    out = {k: np.zeros((B, T, N)) for k in ("x", "decay_gate", "input_gate")}
    err = {k: np.zeros((B, T, N)) for k in out}
    out["log_decay"], err["log_decay"], mag = np.zeros(N), np.zeros(N), np.zeros(N)
    E, e = grad_state.astype(np.float64), np.zeros((B, N))
    w = np.abs(E)
    for t in range(T - 1, -1, -1):
        on = (t < lengths)[:, None]
        sr, si, s, a, m, bb, ea, em, eb, _ = gates(x[:, t], r[:, t], i[:, t], lam)
        gt = g[:, t]
        E1, w1 = E + gt, w + np.abs(gt)
        e1 = e + w1
        u, prev, eprev = si * x[:, t], before[:, t], ebefore[:, t]
        q = a * a / bb * u
        ds = E1 * (a * prev - q)
        eds = e1 * np.abs(a * prev - q) + w1 * (a * eprev + ((ea + 4) * a + FLUSHED) * np.abs(prev)
                                               + (2 * ea + eb + G(i[:, t]) + 8) * np.abs(q))
        du, Gi, Gr = E1 * bb, G(i[:, t]), G(r[:, t])
        for k, v, b in (("x", du * si, e1 * bb * si + w1 * bb * si * (eb + Gi + 3)),
                        ("input_gate", du * u * (1 - si),
                         np.abs(u) * (1 - si) * (e1 * bb + w1 * bb * (eb + 2 * Gi + 5))),
                        ("decay_gate", ds * s * (1 - sr),
                         np.abs(s) * (1 - sr) * (eds + np.abs(ds) * (2 * Gr + 4)))):
            out[k][:, t], err[k][:, t] = np.where(on, v, 0.0), np.where(on, b, 0.0)
        out["log_decay"] += np.where(on, ds * sr, 0.0).sum(0)
        err["log_decay"] += np.where(on, eds * sr + np.abs(ds) * sr * (Gr + 2), 0.0).sum(0)
        mag += np.where(on, np.abs(ds) * sr, 0.0).sum(0)
        nw = a * w1
        ne = a * e1 + kept(s, r[:, t], a, m, em) * w1 + 2 * nw
        E, w, e = np.where(on, a * E1, E), np.where(on, nw, w), np.where(on, ne, e)
    err["log_decay"] += int(np.sum(lengths)) * mag           # a sum in any order
    out["state"], err["state"] = E, e
    return out, {k: U * v for k, v in err.items()}


def draw(rng, B, T, N, typ):
    """Decays of up to 150 a position, gates that are open or shut for good, inputs mostly kept out, so that a
    large state is followed by small ones; gradients of all sizes."""
    def held(v):
        return host(dev(np.asarray(v, np.float32), typ))
    shape = (B, T, N)
    lam = np.resize(np.float32([-14.0, -0.3, -20.0, -1.0, -150.0, -8.0, -0.01, -2.0, -60.0]), N)
    r = np.where(rng.random(shape) < 0.7, rng.uniform(4, 9, shape), rng.normal(-5, 3, shape))
    i = np.where(rng.random(shape) < 0.9, rng.uniform(-14, -8, shape), rng.normal(2, 2, shape))
    x, g = rng.standard_normal(shape), rng.standard_normal(shape) * 10.0 ** rng.uniform(-6, 3, shape)
    state = rng.standard_normal((B, N)) * np.where(rng.random((B, N)) < 0.5, 1e3, 1.0)
    gs = rng.standard_normal((B, N)) * 1e3
    return [held(v) for v in (x, r, i, g)] + [lam, state.astype(np.float32), gs.astype(np.float32)]


CASES = [(3, 1, 9, "f32", "full"), (3, 2, 18, "bf16", "full"), (4, 16, 33, "f32", "ragged"),
         (5, 40, 64, "bf16", "ragged"), (3, 150, 65, "f32", "ragged"), (2, 700, 72, "f32", "ragged"),
         (3, 1025, 130, "bf16", "ragged"), (256, 400, 9, "f32", "ragged"), (1, 4500, 27, "f32", "full")]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_recurrence_after_strong_decays(crf, case):  # noqa: F811
    B, T, N, typ, kind = case
    print(f"\n[recurrence, strong decays {case}]", flush=True)
    rng = np.random.default_rng(B * T + N)
    lengths = draw_lengths(rng, B, T, kind)
    x, r, i, g, lam, state, gs = draw(rng, B, T, N, typ)
    h, end, _, eh, eend, _ = recurrence(x, r, i, lam, lengths, state)
    args, ln = [dev(v.astype(np.float32), typ) for v in (x, r, i)] + [dev(lam)], dev(lengths)
    got, gend, starts = crf.gated_recurrence(*args, lengths=ln, state=dev(state), want_state=True, want_starts=True)
    near(got, h, U * eh, typ, "h")
    near(gend, end, U * eend, "f32", "state")
    d = crf.gated_recurrence_grad(dev(g.astype(np.float32), typ), *args, starts, lengths=ln, state=dev(state),
                                  grad_state=dev(gs))
    want, err = recurrence_grad(g, x, r, i, lam, lengths, state, gs)
    for k, v in want.items():
        near(d["grad_" + k], v, err[k], "f32" if k in ("log_decay", "state") else typ, k)


def test_step_after_strong_decays(crf):  # noqa: F811
    rng = np.random.default_rng(4)
    x, r, i, _, lam, state, _ = draw(rng, 40, 1, 90, "f32")
    h, _, _, eh, _, _ = recurrence(x, r, i, lam, np.ones(40, int), state)
    s = dev(state)
    out = crf.gated_recurrence_step(*(dev(v[:, 0].astype(np.float32)) for v in (x, r, i)), dev(lam), s)
    near(out, h[:, 0], U * eh[:, 0], "f32", "h")
    near(s, h[:, 0], U * eh[:, 0], "f32", "state")


def test_a_reset_leaves_what_comes_after(crf):  # noqa: F811
    """A state of 1,000 under decays of exp(-14) and exp(-20), an input far smaller: 3e-7 of what is left in
    float32, where an error of 2^-24 of the state before would be all of it."""
    import torch
    for lam, u in ((-14.0, 1e-4), (-20.0, 1e-5), (-150.0, 1e-9)):
        big = torch.full((1, 1, 2), 200.0, device="cuda")
        x = torch.full((1, 1, 2), u, device="cuda")
        state = torch.full((1, 2), 1e3, device="cuda")
        ld = torch.full((2,), lam, device="cuda")
        want = np.exp(lam) * 1e3 + np.sqrt(-np.expm1(2 * lam)) * float(x[0, 0, 0])
        for h in (crf.gated_recurrence(x, big, big, ld, state=state)[0],
                  crf.gated_recurrence_step(x[0], big[0], big[0], ld, state)):
            assert np.all(np.abs(host(h) - want) <= (abs(lam) + 16) * U * want), lam


@pytest.mark.parametrize("case", [(2, 16, 64, "f32"), (3, 333, 70, "f32"), (2, 900, 129, "bf16"), (1, 5000, 8, "f32")],
                         ids=lambda c: "-".join(map(str, c)))
def test_weak_decays_that_add_up(crf, case):  # noqa: F811
    """No decay is strong, but those of a few positions together are: a state of 1,000 fades to nothing beside inputs
    that are kept out."""
    B, T, N, typ = case
    print(f"\n[recurrence, weak decays {case}]", flush=True)
    rng = np.random.default_rng(T)
    x, r, i, g, _, state, gs = draw(rng, B, T, N, typ)
    i = host(dev(np.full(i.shape, -40.0, np.float32), typ))
    g[:, : T - 1] *= 1e-12
    g = host(dev(g.astype(np.float32), typ))
    lam = np.resize(np.float32([-0.25, -0.2, -0.1, -0.05]), N)
    L = np.full(B, T)
    h, end, _, eh, eend, _ = recurrence(x, r, i, lam, L, state)
    args = [dev(v.astype(np.float32), typ) for v in (x, r, i)] + [dev(lam)]
    got, gend, starts = crf.gated_recurrence(*args, state=dev(state), want_state=True, want_starts=True)
    near(got, h, U * eh, typ, "h")
    near(gend, end, U * eend, "f32", "state")
    d = crf.gated_recurrence_grad(dev(g.astype(np.float32), typ), *args, starts, state=dev(state), grad_state=dev(gs))
    want, err = recurrence_grad(g, x, r, i, lam, L, state, gs)
    for k, v in want.items():
        near(d["grad_" + k], v, err[k], "f32" if k in ("log_decay", "state") else typ, k)
