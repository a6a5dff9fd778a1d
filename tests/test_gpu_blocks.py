"""Gated recurrence, residual norm and token loss against their definitions in 64 bits, through the
package's entry points.  Tolerances are the first-order bounds of tests/blocks_ref.py, with a tenth
more for what is of second order, and half a step of the output's type."""

import numpy as np
import pytest

import blocks_ref as ref
from test_gpu_encoder import close, crf, dev, draw_lengths, host, poison, rounding  # noqa: F401

pytestmark = pytest.mark.gpu

NAN = float("nan")


def near(got, want, bound, typ, what):
    close(got, want, 1.1 * bound + 1.1 * rounding(typ, np.abs(want) + bound) + 1e-37, what)


def values(rng, shape, typ, sd=1.0, mean=0.0):
    """Numbers that the type holds exactly."""
    return host(dev((mean + sd * rng.standard_normal(shape)).astype(np.float32), typ))


def put(x, typ, lengths=None):
    """On the GPU, in a type; padding holds what must not be read."""
    if lengths is not None:
        x = poison(np.array(x), lengths)
    return dev(np.asarray(x, np.float32), typ)


def up_to(lengths, x):
    """Zeros at padding."""
    m = np.arange(x.shape[1])[None] < lengths[:, None]
    return np.where(m[..., None], x, 0.0)


# ---------------------------------------------------------------- gated recurrence

RECURRENCE = [  # B, T, N, typ, lengths, state, log_decay
    (1, 1, 1, "f32", "full", False, "spread"),
    (1, 1, 7, "bf16", "full", True, "spread"),
    (2, 15, 64, "f32", "full", True, "spread"),
    (3, 16, 65, "bf16", "ragged", True, "spread"),
    (3, 17, 130, "f32", "ragged", False, "spread"),
    (5, 33, 333, "bf16", "ragged", True, "strong"),
    (2, 127, 8, "f32", "full", False, "weak"),
    (3, 128, 96, "bf16", "full", True, "spread"),
    (4, 129, 40, "f32", "ragged", True, "spread"),
    (4, 255, 256, "bf16", "ragged", False, "spread"),
    (1, 257, 2, "bf16", "full", True, "weak"),
    (3, 700, 72, "f32", "ragged", True, "weak"),
    (2, 1025, 129, "bf16", "ragged", True, "spread"),
    (1, 5000, 5, "f32", "full", True, "weak"),
    (9, 600, 512, "bf16", "ragged", True, "spread"),
]


def decays(N, kind):
    if kind == "strong":                                     # memories of a few positions at most
        v = -np.exp(np.linspace(-1.0, 5.0, N))
    elif kind == "weak":                                     # up to a million
        v = -np.exp2(-np.linspace(3.0, 20.0, N))
    else:
        v = -np.exp2(-1.0 - 10.0 * np.arange(N) / max(1, N - 1))
    return v.astype(np.float32)


def recurrence_case(case):
    B, T, N, typ, kind, with_state, dk = case
    rng = np.random.default_rng(B * T * 7 + N)
    lengths = draw_lengths(rng, B, T, kind)
    x, r, i, g = (values(rng, (B, T, N), typ) for _ in range(4))
    lam = decays(N, dk)
    state, gs = (rng.standard_normal((2, B, N)).astype(np.float32) if with_state else (None, None))
    return lengths, x, r, i, g, lam, state, gs


@pytest.mark.parametrize("case", RECURRENCE, ids=lambda c: "-".join(map(str, c)))
def test_gated_recurrence_and_its_gradients(crf, case):  # noqa: F811
    B, T, N, typ, kind, with_state, _ = case
    print(f"\n[recurrence {case}]", flush=True)
    lengths, x, r, i, g, lam, state, gs = recurrence_case(case)
    h, end, eh, eend, starts = ref.recurrence(x, r, i, lam, lengths, state)
    xd, rd, id_, gd = (put(v, typ, lengths) for v in (x, r, i, g))
    ld, sd = dev(lam), None if state is None else dev(state)
    ln = dev(lengths)
    got, gend, gstarts = crf.gated_recurrence(xd, rd, id_, ld, lengths=ln, state=sd, want_state=True,
                                              want_starts=True, check_status=True)
    near(got, h, eh, typ, "h")
    near(gend, end, eend, "f32", "state")
    d = crf.gated_recurrence_grad(gd, xd, rd, id_, ld, gstarts, lengths=ln, state=sd,
                                  grad_state=None if gs is None else dev(gs), check_status=True)
    want, err = ref.recurrence_grad(g, x, r, i, lam, lengths, state, gs)
    for k in ("x", "decay_gate", "input_gate"):
        near(d["grad_" + k], want[k], err[k], typ, k)
    near(d["grad_log_decay"], want["log_decay"], err["log_decay"], "f32", "log_decay")
    assert ("grad_state" in d) == with_state
    if with_state:
        near(d["grad_state"], want["state"], err["state"], "f32", "state")


def test_recurrence_views_and_autograd(crf):  # noqa: F811
    """The three inputs as parts of one projection; gradients through autograd, also of the state."""
    import torch
    rng = np.random.default_rng(3)
    B, T, N = 3, 70, 50
    x, r, i, g = (values(rng, (B, T, N), "bf16") for _ in range(4))
    lam, state = decays(N, "spread"), rng.standard_normal((B, N)).astype(np.float32)
    gs = rng.standard_normal((B, N)).astype(np.float32)
    lengths = np.array([70, 41, 0], np.int32)
    whole = put(np.concatenate([x, r, i], -1), "bf16").requires_grad_()
    ld, sd = dev(lam).requires_grad_(), dev(state).requires_grad_()
    h, end = crf.gated_recurrence(*whole.chunk(3, -1), ld, lengths=dev(lengths), state=sd, want_state=True)
    want_h, want_end, eh, eend, _ = ref.recurrence(x, r, i, lam, lengths, state)
    near(h, want_h, eh, "bf16", "h")
    near(end, want_end, eend, "f32", "state")
    d = torch.autograd.grad([h, end], [whole, ld, sd], [put(g, "bf16"), dev(gs)])
    want, err = ref.recurrence_grad(g, x, r, i, lam, lengths, state, gs)
    names = ("x", "decay_gate", "input_gate")
    near(d[0], np.concatenate([want[k] for k in names], -1), np.concatenate([err[k] for k in names], -1), "bf16", "dx")
    near(d[1], want["log_decay"], err["log_decay"], "f32", "log_decay")
    near(d[2], want["state"], err["state"], "f32", "state")


def test_recurrence_gradients_against_differences(crf):  # noqa: F811
    """Central differences of sum(h g) along random directions, in float32."""
    rng = np.random.default_rng(11)
    B, T, N = 2, 40, 24
    x, r, i, g = (rng.standard_normal((B, T, N)).astype(np.float32) for _ in range(4))
    lam = decays(N, "spread")
    args = [x, r, i, lam]
    starts = crf.gated_recurrence(*map(dev, args), want_starts=True)[1]
    d = crf.gated_recurrence_grad(dev(g), *map(dev, args), starts)
    for k, name in enumerate(("grad_x", "grad_decay_gate", "grad_input_gate", "grad_log_decay")):
        D = rng.standard_normal(args[k].shape).astype(np.float32) * (np.abs(lam) if k == 3 else 1.0)
        D = D.astype(np.float32)
        ends, step = [], 2.0 ** -6
        for s in (1, -1):
            moved = [np.float32(a + s * step * D) if j == k else a for j, a in enumerate(args)]
            ends.append((host(crf.gated_recurrence(*map(dev, moved))) * g).sum())
        slope, want = (ends[0] - ends[1]) / (2 * step), (host(d[name]) * D).sum()
        # h rounds by some 2^-22 of its size, over 2 * 40 * 24 terms and a step of 2^-6; the third
        # derivative's share is step^2 of the terms
        size = np.abs(host(d[name]) * D).sum() + 1.0
        assert abs(slope - want) < 2e-3 * size, (name, slope, want, size)


def test_recurrence_limits_of_the_gates(crf):  # noqa: F811
    """Gates so far open or closed that their sigmoid is 0 or 1, and a decay of 0: finite everywhere,
    the state kept or replaced exactly."""
    import torch
    N = 4
    x = torch.tensor([[[1.0, 2.0, 3.0, 4.0]] * 20], device="cuda")
    state = torch.tensor([[5.0, 6.0, 7.0, 8.0]], device="cuda")
    for rv, iv, lam in ((-200.0, 200.0, -1.0), (200.0, -200.0, -1.0), (0.0, 0.0, 0.0), (200.0, 200.0, -1e4),
                        (-1e30, 1e30, -1.0), (1e30, -1e30, -2.0)):
        r, i = torch.full_like(x, rv), torch.full_like(x, iv)
        ld = torch.full((N,), lam, device="cuda")
        h, end, starts = crf.gated_recurrence(x, r, i, ld, state=state, want_state=True, want_starts=True)
        a = float(np.exp(np.float64(lam) * (1 if rv > 0 else 0.5 if rv == 0 else 0)))
        u = np.sqrt(1 - a * a) * (1.0 if iv > 0 else 0.5 if iv == 0 else 0.0) * host(x)[0]
        v = host(state)[0]
        for t in range(20):
            v = a * v + u[t]
            assert np.allclose(host(h)[0, t], v, rtol=1e-5, atol=1e-6), (rv, iv, lam, t)
        d = crf.gated_recurrence_grad(torch.ones_like(x), x, r, i, ld, starts, state=state)
        for k, t in d.items():
            assert bool(torch.isfinite(t).all()), (rv, iv, lam, k)


def test_recurrence_nan_stays_in_its_channel(crf):  # noqa: F811
    import torch
    torch.manual_seed(0)
    x, r, i = (torch.randn(2, 300, 70, device="cuda") for _ in range(3))
    ld = dev(decays(70, "spread"))
    clean, cend = crf.gated_recurrence(x, r, i, ld, want_state=True)
    for k in range(3):
        bad = [v.clone() if j == k else v for j, v in enumerate((x, r, i))]
        bad[k][1, 40, 9] = NAN
        h, end = crf.gated_recurrence(*bad, ld, want_state=True)
        hit = torch.zeros_like(h, dtype=torch.bool)
        hit[1, 40:, 9] = True
        assert bool(h[hit].isnan().all()) and torch.equal(h[~hit], clean[~hit])
        assert bool(end[1, 9].isnan())


def test_recurrence_carries_on(crf):  # noqa: F811
    """Two halves of a sequence, the second from the first one's state: the same numbers, up to the
    rounding of another order of joins; the state may be updated in place."""
    rng = np.random.default_rng(5)
    B, T, N = 2, 600, 96
    x, r, i = (values(rng, (B, T, N), "f32") for _ in range(3))
    lam = decays(N, "spread")
    h, _, eh, _, _ = ref.recurrence(x, r, i, lam, np.full(B, T))
    first, state = crf.gated_recurrence(*(put(v[:, :333], "f32") for v in (x, r, i)), dev(lam), want_state=True)
    second = crf.gated_recurrence(*(put(v[:, 333:], "f32") for v in (x, r, i)), dev(lam), state=state)
    near(first, h[:, :333], eh[:, :333], "f32", "first")
    near(second, h[:, 333:], eh[:, 333:], "f32", "second")


@pytest.mark.parametrize("N", [1, 65, 200, 257])
@pytest.mark.parametrize("T", [1, 16, 17, 100, 128, 129, 900, 3000])
def test_recurrence_state_in_place(crf, T, N):  # noqa: F811
    """The final state may be written over the initial one, whatever the number of tiles."""
    import torch
    from semi_markov_crf_amd import _native, blocks
    torch.manual_seed(T)
    B = 700 if T < 20 or T == 900 else 3
    x, r, i = (torch.randn(B, T, N, device="cuda") for _ in range(3))
    ld, state = dev(decays(N, "weak")), torch.randn(B, N, device="cuda")
    want, end = crf.gated_recurrence(x, r, i, ld, state=state, want_state=True)
    dev_index, a = blocks._recurrence(x, r, i, ld, None, state, None, 3)
    n = _native.load().semicrf_gated_recurrence_bytes(a, 0)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(x)
    rc = _native.call(dev_index, "semicrf_gated_recurrence", a, torch.cuda.current_stream().cuda_stream, ws.data_ptr(),
                      n, out.data_ptr(), state.data_ptr(), None, None)
    torch.cuda.synchronize()
    assert rc == 0 and torch.equal(out, want) and torch.equal(state, end)


@pytest.mark.parametrize("case", [(300, 200, 128, "bf16", "spread"), (256, 500, 33, "f32", "weak"),
                                  (520, 300, 8, "f32", "spread"), (800, 150, 40, "bf16", "spread"),
                                  (1030, 140, 2, "f32", "strong")], ids=lambda c: "-".join(map(str, c)))
def test_recurrence_of_many_sequences(crf, case):  # noqa: F811
    """Chains for every compute unit and more, in rounds that come out even or not.  All but a few
    sequences get no gradient; those few are compared."""
    import torch
    B, T, N, typ, dk = case
    rng = np.random.default_rng(B + T)
    some = np.array([0, 1, B // 2, B - 2, B - 1])
    lengths = rng.integers(0, T + 1, B).astype(np.int32)
    lengths[some[:4]] = T, 0, T - 1, 129
    x, r, i = (values(rng, (B, T, N), typ) for _ in range(3))
    g = np.zeros((B, T, N), np.float32)
    g[some] = values(rng, (5, T, N), typ)
    lam, state, gs = decays(N, dk), rng.standard_normal((B, N)).astype(np.float32), np.zeros((B, N), np.float32)
    gs[some] = rng.standard_normal((5, N))
    args, ln = [put(v, typ, lengths) for v in (x, r, i)] + [dev(lam)], dev(lengths)
    got, end, starts = crf.gated_recurrence(*args, lengths=ln, state=dev(state), want_state=True, want_starts=True)
    h, last, eh, elast, _ = ref.recurrence(x[some], r[some], i[some], lam, lengths[some], state[some])
    at = torch.tensor(some, device="cuda")
    near(got[at], h, eh, typ, "h")
    near(end[at], last, elast, "f32", "state")
    d = crf.gated_recurrence_grad(put(g, typ), *args, starts, lengths=ln, state=dev(state), grad_state=dev(gs))
    want, bound = ref.recurrence_grad(g[some], x[some], r[some], i[some], lam, lengths[some], state[some], gs[some])
    for k, v in want.items():
        near(d["grad_" + k] if k == "log_decay" else d["grad_" + k][at], v, bound[k],
             "f32" if k in ("log_decay", "state") else typ, k)
    assert not got[~(torch.arange(T, device="cuda")[None] < ln[:, None])].any()


def test_recurrence_broadcast_inputs(crf):  # noqa: F811
    """Gates that are one row for all positions or one sequence for all: views with strides of 0, whose
    gradients autograd adds up."""
    import torch
    torch.manual_seed(2)
    B, T, N = 3, 150, 36
    x = torch.randn(B, T, N, device="cuda", requires_grad=True)
    r = torch.randn(1, 1, N, device="cuda", requires_grad=True)
    i = torch.randn(1, T, N, device="cuda", requires_grad=True)
    ld, g = dev(decays(N, "spread")), torch.randn(B, T, N, device="cuda")
    views = [x, r.expand(B, T, N), i.expand(B, T, N)]
    h = crf.gated_recurrence(*views, ld)
    full = [v.detach().contiguous().requires_grad_() for v in views]
    want = crf.gated_recurrence(*full, ld)
    assert torch.equal(h, want)
    d, e = torch.autograd.grad(h, [x, r, i], g), torch.autograd.grad(want, full, g)
    assert torch.equal(d[0], e[0])
    # sums of 450 and 3 rows by torch, in an order of its own
    assert torch.allclose(d[1], e[1].sum((0, 1), keepdim=True), atol=1e-4)
    assert torch.allclose(d[2], e[2].sum(0, keepdim=True), atol=1e-5)


STEP = [(1, 1, 1, "f32"), (1, 3, 1024, "bf16"), (7, 9, 39, "f32"), (64, 64, 130, "bf16"), (300, 301, 257, "f32")]


@pytest.mark.parametrize("case", STEP, ids=lambda c: "-".join(map(str, c)))
def test_recurrence_step(crf, case):  # noqa: F811
    import torch
    B, pool, N, typ = case
    rng = np.random.default_rng(B + N)
    x, r, i = (values(rng, (B, 1, N), typ) for _ in range(3))
    lam, state = decays(N, "spread"), rng.standard_normal((pool, N)).astype(np.float32)
    slots = rng.permutation(pool)[:B].astype(np.int32)
    if B > 4:
        slots[1], slots[3] = -1, pool
    live = (slots >= 0) & (slots < pool)
    at = np.where(live, slots, 0)
    h, _, eh, _, _ = ref.recurrence(x, r, i, lam, np.ones(B, int), state[at])
    h, eh = h[:, 0] * live[:, None], eh[:, 0]
    args = [put(v[:, 0], typ) for v in (x, r, i)] + [dev(lam)]
    pool_in = dev(state)
    pool_out = torch.full_like(pool_in, 7.0)
    out = crf.gated_recurrence_step(*args, pool_in, slots=dev(slots), state_out=pool_out)
    near(out, h, eh, typ, "h")
    want = np.full_like(state, 7.0, dtype=np.float64)
    bound = np.zeros_like(want)
    want[at[live]], bound[at[live]] = h[live], eh[live]
    near(pool_out, want, bound, "f32", "state")
    assert torch.equal(pool_in, dev(state))
    again = crf.gated_recurrence_step(*args, pool_in, slots=dev(slots))         # in place
    assert torch.equal(again, out)
    keep = np.ones(pool, bool)
    keep[at[live]] = False
    assert torch.equal(pool_in[dev(~keep)], pool_out[dev(~keep)])
    assert torch.equal(pool_in[dev(keep)], dev(state)[dev(keep)])
    if pool >= B:
        s = dev(state)
        whole = crf.gated_recurrence_step(*args, s)
        near(whole, ref.recurrence(x, r, i, lam, np.ones(B, int), state[:B])[0][:, 0], ref.recurrence(
            x, r, i, lam, np.ones(B, int), state[:B])[2][:, 0], typ, "rows in order")


# ---------------------------------------------------------------- residual norm

RESIDUAL = [  # B, T, N, typ, wtyp, lengths, gate, scale, norm_branch, center
    (1, 1, 1, "f32", "f32", "full", True, True, False, False),
    (2, 3, 2, "bf16", "bf16", "full", True, False, True, False),
    (3, 9, 3, "f32", "f32", "ragged", False, True, True, True),
    (3, 20, 7, "bf16", "f32", "ragged", True, True, True, True),
    (2, 33, 8, "bf16", "bf16", "full", False, False, False, True),
    (3, 40, 39, "bf16", "bf16", "ragged", True, True, True, True),
    (2, 65, 64, "f32", "f32", "full", True, False, False, True),
    (3, 50, 128, "bf16", "f32", "ragged", False, True, True, False),
    (2, 31, 333, "f32", "f32", "ragged", True, True, True, True),
    (4, 64, 512, "bf16", "bf16", "ragged", True, True, False, False),
    (2, 37, 777, "f32", "f32", "full", False, False, False, False),
    (3, 30, 1024, "bf16", "bf16", "ragged", True, True, True, True),
    (1, 17, 1030, "f32", "f32", "full", True, True, True, False),
    (2, 9, 2048, "bf16", "f32", "ragged", True, True, True, True),
    (1, 5, 4100, "bf16", "bf16", "full", True, True, True, True),
    (1, 6, 8192, "f32", "f32", "full", True, True, True, True),
    (1, 3, 16384, "bf16", "f32", "full", True, True, True, True),
    (1, 3, 16381, "f32", "f32", "full", False, True, True, False),
    (700, 3, 20, "bf16", "bf16", "ragged", True, True, True, True),       # more rows than one pass takes
    (1, 5000, 72, "f32", "f32", "full", True, False, True, False),
]


@pytest.mark.parametrize("case", RESIDUAL, ids=lambda c: "-".join(map(str, c)))
def test_residual_norm_and_its_gradients(crf, case):  # noqa: F811
    import torch
    B, T, N, typ, wtyp, kind, gated, scaled, post, center = case
    print(f"\n[residual {case}]", flush=True)
    rng = np.random.default_rng(B * T + N)
    lengths = draw_lengths(rng, B, T, kind)
    x, o = values(rng, (B, T, N), typ, 2.0), values(rng, (B, T, N), typ, 1.5, 0.3)
    z = values(rng, (B, T, N), typ) if gated else None
    w, b = values(rng, N, wtyp, 0.1, 1.0), values(rng, N, wtyp, 0.1)
    sc = values(rng, N, wtyp, 0.1, 0.5) if scaled else None
    bw, bb = (values(rng, N, wtyp, 0.1, 1.0), values(rng, N, wtyp, 0.1)) if post else (None, None)
    gr, gy = values(rng, (B, T, N), typ), values(rng, (B, T, N), typ)
    eps = 1e-5
    m = np.arange(T)[None] < lengths[:, None]
    rows = [None if v is None else v[m] for v in (x, o, z, gr, gy)]
    want, err = ref.residual(rows[0], rows[1], w, b, rows[2], sc, post, bw, bb, center, eps, rows[3], rows[4])

    def spread(v):
        full = np.zeros((B, T, N))
        full[m] = v
        return full

    par = {k: None if v is None else put(v, wtyp) for k, v in
           (("scale", sc), ("branch_weight", bw), ("branch_bias", bb))}
    xd, od, grd, gyd = (put(v, typ, lengths) for v in (x, o, gr, gy))
    zd = None if z is None else put(z, typ, lengths)
    ln, wd = dev(lengths), put(w, wtyp)
    kw = dict(gate=zd, norm_branch=post, center=center, lengths=ln, check_status=True, **par)
    r, y, stats = crf.residual_norm(xd, od, wd, put(b, wtyp), eps=eps, want_stats=True, **kw)
    near(r, spread(want["r"]), spread(err["r"]), typ, "r")
    near(y, spread(want["y"]), spread(err["y"]), typ, "y")
    d = crf.residual_norm_grad(grd, gyd, xd, od, wd, stats, **kw)
    names = {"x", "branch", "weight", "bias", "scale"} | ({"gate"} if gated else set()) | (
        {"branch_weight", "branch_bias"} if post else set())
    assert set(d) == {"grad_" + k for k in names}
    for k in sorted(names):
        v, e = want["grad_" + k], err["grad_" + k]
        if k in ("x", "branch", "gate"):
            near(d["grad_" + k], spread(v), spread(e), typ, k)
        else:
            near(d["grad_" + k], v, e, wtyp, k)
    only = crf.residual_norm_grad(grd, gyd, xd, od, wd, stats, want_params=False, **kw)
    assert all(torch.equal(only[k], d[k]) for k in only) and "grad_weight" not in only
    # one of the two gradients alone
    for a, c in ((grd, None), (None, gyd)):
        want1, err1 = ref.residual(rows[0], rows[1], w, b, rows[2], sc, post, bw, bb, center, eps,
                                   0 * rows[3] if a is None else rows[3], 0 * rows[4] if c is None else rows[4])
        d = crf.residual_norm_grad(a, c, xd, od, wd, stats, want_params=False, **kw)
        near(d["grad_x"], spread(want1["grad_x"]), spread(err1["grad_x"]), typ, "grad_x of one")


def test_residual_norm_views_and_autograd(crf):  # noqa: F811
    """branch and gate as parts of one projection; only y used, and both used."""
    import torch
    rng = np.random.default_rng(8)
    B, T, N = 2, 30, 40
    x, o, z, gr, gy = (values(rng, (B, T, N), "bf16") for _ in range(5))
    w, sc = values(rng, N, "f32", 0.1, 1.0), values(rng, N, "f32", 0.1, 0.5)
    both = put(np.concatenate([o, z], -1), "bf16").requires_grad_()
    leaves = [put(x, "bf16").requires_grad_(), both, dev(np.float32(w)).requires_grad_(),
              dev(np.float32(sc)).requires_grad_()]
    for grad_r in (np.zeros_like(gr), gr):
        br, gate = leaves[1].chunk(2, -1)
        r, y = crf.residual_norm(leaves[0], br, leaves[2], gate=gate, scale=leaves[3])
        want, err = ref.residual(x, o, w, None, z, sc, False, None, None, True, 1e-5, grad_r, gy)
        if grad_r.any():
            d = torch.autograd.grad([r, y], leaves, [put(grad_r, "bf16"), put(gy, "bf16")])
        else:
            d = torch.autograd.grad(y, leaves, put(gy, "bf16"))
        near(r, want["r"], err["r"], "bf16", "r")
        near(y, want["y"], err["y"], "bf16", "y")
        near(d[0], want["grad_x"], err["grad_x"], "bf16", "x")
        near(d[1], np.concatenate([want["grad_branch"], want["grad_gate"]], -1),
             np.concatenate([err["grad_branch"], err["grad_gate"]], -1), "bf16", "branch and gate")
        near(d[2], want["grad_weight"], err["grad_weight"], "f32", "weight")
        near(d[3], want["grad_scale"], err["grad_scale"], "f32", "scale")


def test_residual_norm_is_the_layer_norm_of_the_sum(crf):  # noqa: F811
    """Without its options: y is layer_norm(x + branch) and a constant row's norm is the bias."""
    import torch
    torch.manual_seed(1)
    x, o = torch.randn(2, 5, 96, device="cuda"), torch.randn(2, 5, 96, device="cuda")
    w, b = torch.randn(96, device="cuda"), torch.randn(96, device="cuda")
    r, y = crf.residual_norm(x, o, w, b)
    assert torch.equal(r, x + o)
    assert torch.allclose(y, crf.layer_norm(r, w, b), atol=1e-5)
    y = crf.residual_norm(torch.zeros_like(x), torch.zeros_like(o), w, b, norm_branch=True)[1]
    assert torch.equal(y, b.expand_as(y))


def test_residual_norm_gradients_against_differences(crf):  # noqa: F811
    rng = np.random.default_rng(21)
    B, T, N = 2, 6, 50
    args = {k: rng.standard_normal((B, T, N)).astype(np.float32) for k in ("x", "branch", "gate")}
    args.update({k: (1 + 0.3 * rng.standard_normal(N)).astype(np.float32)
                 for k in ("weight", "bias", "scale", "branch_weight", "branch_bias")})
    gr, gy = (rng.standard_normal((B, T, N)).astype(np.float32) for _ in range(2))

    def call(a, **kw):
        a = {k: dev(v) for k, v in a.items()}
        return crf.residual_norm(a.pop("x"), a.pop("branch"), a.pop("weight"), a.pop("bias"), norm_branch=True, **a, **kw)

    stats = call(args, want_stats=True)[2]
    a = {k: dev(v) for k, v in args.items() if k != "bias"}
    d = crf.residual_norm_grad(dev(gr), dev(gy), a.pop("x"), a.pop("branch"), a.pop("weight"), stats,
                               norm_branch=True, **a)
    for name in args:
        D = rng.standard_normal(args[name].shape).astype(np.float32)
        ends, step = [], 2.0 ** -7
        for s in (1, -1):
            r, y = call({**args, name: np.float32(args[name] + s * step * D)})
            ends.append((host(r) * gr + host(y) * gy).sum())
        slope, want = (ends[0] - ends[1]) / (2 * step), (host(d["grad_" + name]) * D).sum()
        # roundings of 2^-22 over 600 terms and a step of 2^-7, third derivatives times step^2 / 6
        size = np.abs(host(d["grad_" + name]) * D).sum() + 1.0
        assert abs(slope - want) < 3e-3 * size, (name, slope, want, size)


# ---------------------------------------------------------------- token loss

NLL = [  # B, T, N, V, typ, target bits, lengths, share of targets, scale
    (1, 1, 1, 1, "f32", 32, "full", 1.0, 1.0),
    (1, 1, 8, 2, "bf16", 64, "full", 1.0, 1.0),
    (2, 3, 7, 5, "f32", 64, "full", 1.0, 0.5),
    (3, 40, 64, 127, "bf16", 32, "ragged", 0.5, 1.0),
    (3, 43, 65, 128, "f32", 32, "ragged", 0.5, 1.0),
    (2, 64, 96, 129, "bf16", 64, "full", 1.0, -0.3),
    (1, 128, 100, 300, "f32", 64, "full", 1.0, 2.0),
    (1, 129, 130, 1000, "bf16", 32, "full", 0.9, 1.0),
    (4, 70, 333, 257, "bf16", 32, "ragged", 1.0, 1.0),
    (5, 333, 39, 40, "f32", 32, "ragged", 0.15, 1.0),
    (2, 4500, 24, 60, "bf16", 64, "ragged", 0.3, 1.0),       # listed by several workgroups
    (3, 1500, 64, 3333, "bf16", 32, "ragged", 0.8, 1.0),     # tiles of 256
    (1, 4200, 33, 4100, "f32", 32, "full", 1.0, 1.0),
    (4, 60, 512, 4096, "bf16", 32, "ragged", 1.0, 1.0),
    (2, 30, 1030, 700, "f32", 32, "full", 1.0, 1.0),
]


def nll_case(case):
    B, T, N, V, typ, bits, kind, share, scale = case
    rng = np.random.default_rng(B * T + N + V)
    lengths = draw_lengths(rng, B, T, kind)
    table = values(rng, (V, N), typ, N ** -0.5)
    t = rng.integers(0, V, (B, T))
    x = values(rng, (B, T, N), typ)
    x = host(put(x + 10 * rng.random((B, T, 1)) * table[t], typ))
    t = np.where(rng.random((B, T)) < share, t, -1 - rng.integers(0, 5, (B, T)))
    for b, L in enumerate(lengths):
        t[b, L:] = V + 3                                     # padding is not looked at
    listed = (np.arange(T)[None] < lengths[:, None]) & (t >= 0)
    return rng, lengths, x, table, t.astype(np.int64 if bits == 64 else np.int32), listed


def depth(typ):
    # additions in a row of a sum over n terms by matrix instructions: 32 products of bfloat16 (64 as an
    # allowance for how the instruction adds them up) or 4 of float32 at a time, then the shares of
    # the contracted axis and pieces of the vocabulary
    return (lambda n: n / 32 + 100) if typ == "bf16" else (lambda n: n / 4 + 60)


@pytest.mark.parametrize("case", NLL, ids=lambda c: "-".join(map(str, c)))
def test_token_nll_and_its_gradients(crf, case):  # noqa: F811
    import torch
    B, T, N, V, typ, bits, kind, share, scale = case
    print(f"\n[token_nll {case}]", flush=True)
    rng, lengths, x, table, t, listed = nll_case(case)
    g = (rng.random((B, T)) - 0.3).astype(np.float32)
    scale = float(np.float32(scale))
    # p is held in fp16 (half a step: 2^-11) where the tensors are bfloat16
    want = ref.nll(x[listed], table, t[listed], scale, depth(typ), 2.0 ** 13 if typ == "bf16" else 1.0,
                   g[listed].astype(np.float64))
    loss, lse, eloss, elses, dx, dW, edx, edW = want
    xd, td, ln = put(np.where(listed[..., None], x, NAN), typ), dev(t), dev(lengths)
    wd = put(table, typ)
    got, glse = crf.token_nll(xd, wd, td, scale=scale, lengths=ln, want_lse=True, check_status=True)

    def spread(v, *shape):
        full = np.zeros((B, T) + shape)
        full[listed] = v
        return full

    near(got, spread(loss), spread(eloss), "f32", "loss")
    near(glse, spread(lse), spread(elses), "f32", "lse")
    gd = dev(np.where(listed, g, NAN).astype(np.float32))
    d = crf.token_nll_grad(gd, xd, wd, td, glse, scale=scale, lengths=ln, check_status=True)
    # rows of x and W far below the largest lose bits of fp16: 2^-25 of the largest a term
    floor = 2.0 ** -24 * abs(scale) if typ == "bf16" else 0.0
    ax, aw = (np.abs(x[listed]).max() if listed.any() else 0.0), np.abs(table).max()
    near(d["grad_x"], spread(dx, N), spread(edx + floor * 2 * aw * np.abs(g[listed])[:, None], N), typ, "grad_x")
    near(d["grad_table"], dW, edW + floor * ax * np.abs(g).sum() * 2, typ, "grad_table")
    for only in ("x", "table"):
        e = crf.token_nll_grad(gd, xd, wd, td, glse, scale=scale, lengths=ln, want_x=only == "x",
                               want_table=only == "table")
        assert list(e) == ["grad_" + only] and torch.equal(e["grad_" + only], d["grad_" + only])


def test_token_nll_in_pieces_of_the_vocabulary(crf):  # noqa: F811
    """More rows than leave room for p of all words at once: the pieces' sums."""
    import torch
    torch.manual_seed(4)
    M, N, V = 270_000, 16, 6001
    x = torch.randn(1, M, N, device="cuda").bfloat16()
    table = (0.5 * torch.randn(V, N, device="cuda")).bfloat16()
    t = torch.randint(0, V, (1, M), device="cuda", dtype=torch.int32)
    g = torch.rand(1, M, device="cuda")
    loss, lse = crf.token_nll(x, table, t, want_lse=True)
    d = crf.token_nll_grad(g, x, table, t, lse)
    z = x[0].double() @ table.double().t()
    want = torch.logsumexp(z, 1)
    assert float((lse[0] - want).abs().max()) < 1e-5          # sums of 6,001 terms, log sums below 16
    assert float((loss[0] - (want - z.gather(1, t[0].long()[:, None])[:, 0])).abs().max()) < 2e-5
    p = torch.exp(z - want[:, None])
    p[torch.arange(M, device="cuda"), t[0].long()] -= 1
    p *= g[0].double()[:, None]
    for name, exact in (("grad_x", p @ table.double()), ("grad_table", p.t().contiguous() @ x[0].double())):
        got = d[name].double().reshape(exact.shape)
        # half a step of bfloat16 of each value, 2^-8, and 2^-11 of its terms in fp16
        assert float((got - exact).norm() / exact.norm()) < 2.0 ** -8, name


def test_token_nll_targets_out_of_range(crf):  # noqa: F811
    import torch
    torch.manual_seed(6)
    x, table = torch.randn(1, 6, 20, device="cuda"), torch.randn(11, 20, device="cuda")
    t = torch.tensor([[3, 11, -1, 10, 2 ** 31 - 1, 0]], device="cuda")
    loss, lse = crf.token_nll(x, table, t, want_lse=True)
    assert loss.isnan().tolist() == [[False, True, False, False, True, False]] and float(loss[0, 2]) == 0.0
    with pytest.raises(crf.SemiCRFError):
        crf.token_nll(x, table, t, check_status=True)
    big = t.clone()
    big[0, 1] = 2 ** 40
    assert torch.equal(crf.token_nll(x, table, big).isnan(), loss.isnan())
    d = crf.token_nll_grad(torch.ones(1, 6, device="cuda"), x, table, t, lse)
    keep = torch.tensor([0, 3, 5], device="cuda")
    e = crf.token_nll_grad(torch.ones(1, 3, device="cuda"), x[:, keep].contiguous(), table, t[:, keep].contiguous(),
                           lse[:, keep].contiguous())
    assert torch.equal(d["grad_x"][:, keep], e["grad_x"]) and torch.equal(d["grad_table"], e["grad_table"])
    assert not d["grad_x"][0, [1, 2, 4]].any()


@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_token_nll_without_targets(crf, typ):  # noqa: F811
    import torch
    x = put(np.full((2, 9, 33), NAN), typ)
    table, t = put(np.ones((70, 33)), typ), torch.full((2, 9), -100, device="cuda")
    loss, lse = crf.token_nll(x, table, t, want_lse=True)
    d = crf.token_nll_grad(torch.ones(2, 9, device="cuda"), x, table, t, lse)
    assert not any(v.any() for v in (loss, lse, d["grad_x"], d["grad_table"]))


@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_token_nll_row_gradients_far_apart(crf, typ):  # noqa: F811
    """Rows whose gradients are 0, tiny, or 2^40 apart: each row's grad_x keeps its own accuracy."""
    rng = np.random.default_rng(12)
    N, V, M = 48, 200, 6
    x, table = values(rng, (1, M, N), typ), values(rng, (V, N), typ, 0.3)
    t = rng.integers(0, V, (1, M)).astype(np.int32)
    g = np.array([[1.0, 0.0, 2.0 ** -40, -(2.0 ** -20), 2.0 ** -30, 0.37]], np.float32)
    want = ref.nll(x[0], table, t[0], 1.0, depth(typ), 2.0 ** 13 if typ == "bf16" else 1.0, g[0].astype(float))
    args = put(x, typ), put(table, typ), dev(t)
    lse = crf.token_nll(*args, want_lse=True)[1]
    d = crf.token_nll_grad(dev(g), *args, lse)
    extra = 2.0 ** -23 * np.abs(table).max() * np.abs(g[0])[:, None] if typ == "bf16" else 0.0
    near(d["grad_x"][0], want[4], want[6] + extra, typ, "grad_x")
    near(d["grad_table"], want[5], want[7] + 2.0 ** -23 * np.abs(x).max(), typ, "grad_table")


def test_token_nll_scores_far_apart(crf):  # noqa: F811
    """Scores of hundreds: the largest is taken out before the exponential."""
    import torch
    N, V = 64, 500
    x = torch.ones(1, 3, N, device="cuda")
    table = torch.zeros(V, N, device="cuda")
    table[7], table[9] = 10.0, -10.0
    t = torch.tensor([[7, 9, 0]], device="cuda")
    loss = crf.token_nll(x, table, t)
    assert torch.allclose(loss, torch.tensor([[0.0, 1280.0, 640.0]], device="cuda"), atol=1e-3)
    big = crf.token_nll(x, table, t, scale=1e4)
    assert bool(torch.isfinite(big).all()) and float(big[0, 0]) == 0.0


def test_token_nll_gradients_against_differences(crf):  # noqa: F811
    rng = np.random.default_rng(31)
    N, V, B, T = 20, 50, 2, 12
    x, table = rng.standard_normal((B, T, N)).astype(np.float32), rng.standard_normal((V, N)).astype(np.float32)
    t, g = rng.integers(-3, V, (B, T)).astype(np.int32), rng.random((B, T)).astype(np.float32)
    lse = crf.token_nll(dev(x), dev(table), dev(t), scale=0.7, want_lse=True)[1]
    d = crf.token_nll_grad(dev(g), dev(x), dev(table), dev(t), lse, scale=0.7)
    for name, k in (("grad_x", 0), ("grad_table", 1)):
        D = rng.standard_normal((x, table)[k].shape).astype(np.float32)
        ends, step = [], 2.0 ** -7
        for s in (1, -1):
            a = [np.float32(v + s * step * D) if j == k else v for j, v in enumerate((x, table))]
            ends.append((host(crf.token_nll(dev(a[0]), dev(a[1]), dev(t), scale=0.7)) * g).sum())
        slope, want = (ends[0] - ends[1]) / (2 * step), (host(d[name]) * D).sum()
        size = np.abs(host(d[name]) * D).sum() + 1.0
        assert abs(slope - want) < 3e-3 * size, (name, slope, want)


# ---------------------------------------------------------------- together

def test_streams_and_graph_replays(crf):  # noqa: F811
    """A block and the loss, captured and replayed with eager work between: each replay equals the
    eager result bit by bit; also on a stream of its own."""
    import torch
    torch.manual_seed(9)
    B, T, N, V = 3, 300, 64, 500
    mk = lambda *s: torch.randn(*s, device="cuda").bfloat16()  # noqa: E731
    x, r, i, o = (mk(B, T, N) for _ in range(4))
    table, ld = mk(V, N), dev(decays(N, "spread"))
    t = torch.randint(-20, V, (B, T), device="cuda", dtype=torch.int32)
    lengths = torch.tensor([300, 17, 250], device="cuda", dtype=torch.int32)
    g = torch.rand(B, T, device="cuda")
    w = torch.ones(N, device="cuda", dtype=torch.bfloat16)

    def block():
        h, end, starts = crf.gated_recurrence(x, r, i, ld, lengths=lengths, want_state=True, want_starts=True)
        s, y, stats = crf.residual_norm(o, h, w, gate=r, lengths=lengths, want_stats=True)
        loss, lse = crf.token_nll(y, table, t, lengths=lengths, want_lse=True)
        d = crf.token_nll_grad(g, y, table, t, lse, lengths=lengths)
        e = crf.residual_norm_grad(None, d["grad_x"], o, h, w, stats, gate=r, lengths=lengths)
        f = crf.gated_recurrence_grad(e["grad_branch"], x, r, i, ld, starts, lengths=lengths)
        return [h, end, s, y, loss, *d.values(), *e.values(), *f.values()]

    eager = block()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = block()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(eager, again))
    with torch.cuda.graph(graph):
        out = block()
    for k in range(3):
        for v in (x, r, i, o):
            v.copy_(torch.randn_like(v, dtype=torch.float32))
        t.copy_(torch.randint(-20, V, (B, T), device="cuda", dtype=torch.int32))
        graph.replay()
        got = [v.clone() for v in out]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, block())), k


def test_two_calls_at_once(crf):  # noqa: F811
    """The same calls on two streams at a time."""
    import torch
    torch.manual_seed(10)
    sets = []
    for k in range(2):
        x, r, i = (torch.randn(4, 3000, 200, device="cuda") for _ in range(3))
        t = torch.randint(0, 900, (4, 3000), device="cuda", dtype=torch.int32)
        sets.append((x, r, i, dev(decays(200, "spread")), torch.randn(900, 200, device="cuda"), t))

    def work(s):
        h, starts = crf.gated_recurrence(*s[:4], want_starts=True)
        d = crf.gated_recurrence_grad(s[0], *s[:4], starts)
        loss, lse = crf.token_nll(s[0], s[4], s[5], want_lse=True)
        return [h, *d.values(), loss, *crf.token_nll_grad(loss, s[0], s[4], s[5], lse).values()]

    alone = [work(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = []
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(work(s))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_lengths_out_of_range(crf):  # noqa: F811
    import torch
    x = torch.randn(2, 5, 8, device="cuda")
    ld, bad = dev(decays(8, "spread")), torch.tensor([6, -1], device="cuda", dtype=torch.int32)
    ok = torch.tensor([5, 0], device="cuda", dtype=torch.int32)
    t = torch.zeros(2, 5, device="cuda", dtype=torch.int32)
    calls = [lambda **k: crf.gated_recurrence(x, x, x, ld, **k), lambda **k: crf.residual_norm(x, x, **k)[1],
             lambda **k: crf.token_nll(x, x[0].contiguous(), t, **k)]
    for f in calls:
        assert torch.equal(f(lengths=bad), f(lengths=ok))
        with pytest.raises(crf.SemiCRFError):
            f(lengths=bad, check_status=True)


def test_refusals(crf):  # noqa: F811
    import torch
    x, ld, w = torch.randn(2, 5, 8, device="cuda"), dev(decays(8, "spread")), torch.ones(8, device="cuda")
    t = torch.zeros(2, 5, device="cuda", dtype=torch.int32)
    small = torch.empty(1, dtype=torch.uint8, device="cuda")
    for f in (lambda: crf.gated_recurrence(x, x[:1], x, ld), lambda: crf.gated_recurrence(x, x, x, ld[:4]),
              lambda: crf.gated_recurrence(x, x.transpose(1, 2), x, ld), lambda: crf.gated_recurrence(x[0], x[0], x[0], ld),
              lambda: crf.gated_recurrence(x, x, x.cpu(), ld), lambda: crf.gated_recurrence(x, x, x, ld, state=x[0]),
              lambda: crf.gated_recurrence(x, x, x, ld, workspace=small),
              lambda: crf.gated_recurrence(*(v[..., ::2] for v in (x, x, x)), ld[:4].contiguous()),
              lambda: crf.gated_recurrence_grad(x, x, x, x, ld, x),
              lambda: crf.gated_recurrence_step(x[:, 0], x[:, 0], x[:, 0], ld, torch.zeros(1, 8, device="cuda")),
              lambda: crf.gated_recurrence_step(x[:, 0], x[:, 0], x[:, 0], ld, x),
              lambda: crf.residual_norm(x, x[:, :4]), lambda: crf.residual_norm(x.transpose(0, 1), x),
              lambda: crf.residual_norm(x, x, w[:4]), lambda: crf.residual_norm(x, x, gate=x[0]),
              lambda: crf.residual_norm(x, x, branch_weight=w), lambda: crf.residual_norm_grad(x, x, x, x, w, x),
              lambda: crf.token_nll(x, x[0, :, :4], t), lambda: crf.token_nll(x, x[0], t[:1]),
              lambda: crf.token_nll(x, x[0], t.t()), lambda: crf.token_nll(x, x[0], t, workspace=small),
              lambda: crf.token_nll_grad(x[..., 0].contiguous(), x, x[0], t, t.float(), want_x=False, want_table=False),
              lambda: crf.token_nll_grad(x, x, x[0], t, t.float())):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: crf.gated_recurrence(x, x.bfloat16(), x, ld), lambda: crf.gated_recurrence(x, x, x, ld.double()),
              lambda: crf.residual_norm(x, x, w.bfloat16()), lambda: crf.residual_norm(x, x.double()),
              lambda: crf.residual_norm(x.half(), x.half()), lambda: crf.token_nll(x, x[0].bfloat16(), t),
              lambda: crf.token_nll(x, x[0], t.float())):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(crf.SemiCRFError):
        crf.residual_norm(x, x, eps=-1.0)
    with pytest.raises(crf.SemiCRFError):
        crf.token_nll(x, x[0], t, scale=float("inf"))
    far = torch.zeros(2, device="cuda").as_strided((1, 1, 2), (2, 2, 1)).as_strided((1, 2, 1), (1, 1, 1))
    assert crf.gated_recurrence(far, far, far, ld[:1].contiguous()).shape == (1, 2, 1)
    wide = torch.zeros(1, 1, 16385, device="cuda")
    with pytest.raises(crf.SemiCRFError):
        crf.residual_norm(wide, wide)
