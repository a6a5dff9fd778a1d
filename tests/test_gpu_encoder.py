"""The encoder operators (embedding, layer norm, decayed linear attention) against their
definitions in 64 bits, through the package's entry points.

Tolerances, fixed from the arithmetic.  u = 2^-24 is half an ulp of float32 at 1 and w = 2^-8
that of bfloat16; `mag` is the sum of the absolute values of the terms a result adds up.
  * an fp32 sum of n terms is within n u mag of the exact one;
  * a result rounded to bfloat16 is within w |result| of the unrounded one;
  * attention in bfloat16 rounds the masked products once (w of each term) and takes the state
    as two bfloat16 numbers (w^2), so it is within 1.1 w mag before the final rounding;
  * a decay gamma^n is exp2 of an fp32 product: within (2 + |log2 gamma^n|) u, and terms with
    |log2 gamma^n| > 60 no longer matter: 64 u covers it.
"""

import numpy as np
import pytest

import encoder_ref as ref

pytestmark = pytest.mark.gpu

U, W = 2.0 ** -24, 2.0 ** -8
NAN = float("nan")


@pytest.fixture(scope="module")
def crf():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import semi_markov_crf_amd
    semi_markov_crf_amd._native.load()
    return semi_markov_crf_amd


def dev(a, typ="f32"):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    if a.dtype.kind == "f":
        t = t.to(torch.float32 if typ == "f32" else torch.bfloat16)
    return t


def host(t):
    return t.detach().double().cpu().numpy()


def close(got, want, tol, what):
    got = host(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    err = np.abs(got - want)
    bad = ~(err <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.where(np.isnan(err), np.inf, err), 0)), err.shape)
        t = np.broadcast_to(tol, err.shape)[i]
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, at {i} got {got[i]!r}, "
                             f"want {want[i]!r}, tolerance {t:.3e}")


def rounding(typ, want):
    return W * np.abs(want) if typ == "bf16" else U * np.abs(want)


def draw_lengths(rng, B, T, kind):
    if kind == "full":
        return np.full(B, T, np.int32)
    L = rng.integers(0, T + 1, B).astype(np.int32)
    L[0] = T
    if B > 1:
        L[1] = 0
    if B > 2:
        L[2] = min(1, T)
    return L


def poison(x, lengths):
    """NaN and infinities wherever a position is padding."""
    for b, L in enumerate(lengths):
        x[b, L:] = NAN
        if L < x.shape[1]:
            x[b, L] = np.inf
    return x


# ---------------------------------------------------------------- embedding

EMBED = [  # B, T, V, N, typ, token type, lengths
    (1, 1, 1, 1, "f32", np.int32, "full"),
    (2, 7, 5, 3, "bf16", np.int64, "full"),
    (3, 64, 11, 39, "f32", np.int64, "ragged"),
    (3, 65, 300, 64, "bf16", np.int32, "ragged"),
    (2, 500, 6, 333, "f32", np.int32, "ragged"),
    (4, 130, 70000, 257, "bf16", np.int32, "ragged"),
    (1, 9000, 300, 17, "f32", np.int32, "full"),      # several tiles of the sort, two digits
    (2, 20000, 6, 16, "bf16", np.int32, "ragged"),     # runs over hundreds of chunks
    (3, 4100, 2, 70, "f32", np.int32, "ragged"),
    (1, 40, 4, 1030, "bf16", np.int32, "full"),
    (2, 40000, 300, 9, "f32", np.int32, "ragged"),     # counts scanned by a launch of their own
]


@pytest.mark.parametrize("case", EMBED, ids=[f"B{c[0]}T{c[1]}V{c[2]}N{c[3]}{c[4]}" for c in EMBED])
def test_embed_and_its_gradient(crf, case):
    B, T, V, N, typ, tt, kind = case
    print(f"\n[embed {case}]", flush=True)
    rng = np.random.default_rng(B * T + N)
    lengths = draw_lengths(rng, B, T, kind)
    tok = rng.integers(0, V, (B, T)).astype(tt)
    for b, L in enumerate(lengths):
        tok[b, L:] = -7                                # padding is not looked at
    table = host(dev(rng.standard_normal((V, N)).astype(np.float32), typ))
    scale = float(np.float32(N ** 0.5))
    tk, ln = dev(tok), dev(lengths)
    y = crf.embed(tk, dev(table.astype(np.float32), typ), scale=scale, lengths=ln, check_status=True)
    want = ref.embed(tok, table, scale, lengths)
    close(y, want, U * np.abs(want) + rounding(typ, want), "y")

    g = rng.standard_normal((B, T, N)).astype(np.float32)
    g = host(dev(g, typ))
    gd = dev(poison(g.copy(), lengths).astype(np.float32), typ)
    d = crf.embed_grad(tk, gd, V, scale=scale, lengths=ln, check_status=True)
    want, mag, cnt = ref.embed_grad(tok, g, V, scale, lengths)
    close(d, want, (cnt[:, None] + 2) * U * mag + rounding(typ, want), "grad_table")
    again = crf.embed_grad(tk, gd, V, scale=scale, lengths=ln)
    assert (again == d).all()                          # fixed order: the same bits


def test_embed_gradient_against_differences(crf):
    """embed is linear in the table: (f(W + D) - f(W - D)) / 2 . g is D . grad exactly, up to
    rounding."""
    rng = np.random.default_rng(5)
    B, T, V, N = 2, 300, 40, 33
    tok, W0, D, g = (rng.integers(0, V, (B, T)).astype(np.int32), rng.standard_normal((V, N)),
                     rng.standard_normal((V, N)), rng.standard_normal((B, T, N)))
    W0, D, g = (x.astype(np.float32) for x in (W0, D, g))
    plus, minus = (host(crf.embed(dev(tok), dev(W0 + s * D), scale=1.5)) for s in (1, -1))
    slope = ((plus - minus) / 2 * g).sum()
    grad = host(crf.embed_grad(dev(tok), dev(g), V, scale=1.5))
    tol = 8 * U * (1.5 * (np.abs(W0) + np.abs(D))[tok] * np.abs(g)).sum()
    assert abs(slope - (grad * D).sum()) <= tol


def test_tokens_and_lengths_out_of_range(crf):
    rng = np.random.default_rng(6)
    B, T, V, N = 2, 20, 9, 12
    tok = rng.integers(0, V, (B, T)).astype(np.int64)
    tok[0, 3], tok[1, 5], tok[1, 6] = V, -1, 2 ** 40
    table, g = (rng.standard_normal(s).astype(np.float32) for s in ((V, N), (B, T, N)))
    y = host(crf.embed(dev(tok), dev(table)))
    want = ref.embed(tok, table, 1.0, [T, T])
    assert np.array_equal(np.isnan(y), np.isnan(want)) and np.isnan(y[1, 6]).all()
    d = crf.embed_grad(dev(tok), dev(g), V)
    want, mag, cnt = ref.embed_grad(tok, g, V, 1.0, [T, T])
    close(d, want, (cnt[:, None] + 2) * U * mag, "grad")
    for f in (lambda: crf.embed(dev(tok), dev(table), check_status=True),
              lambda: crf.embed_grad(dev(tok), dev(g), V, check_status=True)):
        with pytest.raises(crf.SemiCRFError):
            f()
    tok[:] = 1
    bad = dev(np.array([T + 5, -3], np.int32))         # taken as T and 0
    y = crf.embed(dev(tok), dev(table), lengths=bad)
    close(y, ref.embed(tok, table, 1.0, [T, 0]), 0.0, "clamped")
    with pytest.raises(crf.SemiCRFError):
        crf.embed(dev(tok), dev(table), lengths=bad, check_status=True)
    with pytest.raises(crf.SemiCRFError):
        crf.layer_norm(dev(g), lengths=bad, check_status=True)


def test_embed_offsets_past_32_bits(crf):
    """Outputs of more than 2^31 elements; the last rows are the ones that would go wrong."""
    import torch
    n, N, V = 530_000, 4100, 3
    print(f"\n[embed n={n} N={N}]", flush=True)
    tok = (torch.arange(n, device="cuda", dtype=torch.int32) % V).view(1, n)
    table = torch.randn(V, N, device="cuda").bfloat16()
    y = crf.embed(tok, table)
    assert torch.equal(y[0, -7:], table[tok[0, -7:].long()]) and torch.equal(y[0, 0], table[0])
    y.zero_()
    y[0, -5:] = 1.0
    d = crf.embed_grad(tok, y, V)
    want = torch.bincount(tok[0, -5:].long(), minlength=V).float()
    assert torch.equal(d.float(), want[:, None].expand(V, N))
    m = crf.layer_norm(y, eps=1.0)                     # rows of ones: zeros
    assert float(m[0, -6:].float().abs().max()) == 0.0


# ---------------------------------------------------------------- layer norm

NORM = [  # B, T, N, typ, weight type, lengths
    (1, 1, 1, "f32", "f32", "full"),
    (2, 5, 2, "bf16", "bf16", "full"),
    (3, 9, 6, "f32", "f32", "ragged"),
    (3, 40, 39, "bf16", "f32", "ragged"),
    (2, 64, 333, "f32", "f32", "full"),
    (4, 100, 64, "bf16", "bf16", "ragged"),
    (4, 700, 257, "f32", "f32", "ragged"),
    (3, 50, 512, "bf16", "bf16", "ragged"),
    (2, 33, 1023, "bf16", "f32", "ragged"),
    (3, 21, 2050, "f32", "f32", "ragged"),
    (3, 20, 4096, "bf16", "bf16", "ragged"),
    (3, 5, 8200, "f32", "f32", "ragged"),
    (2, 3, 32768, "bf16", "bf16", "full"),
    (1, 3, 32768, "f32", "f32", "full"),
]


def norm_inputs(case, affine=True):
    B, T, N, typ, wt, kind = case
    rng = np.random.default_rng(N + B)
    lengths = draw_lengths(rng, B, T, kind)
    x = rng.standard_normal((B, T, N)) * 2 + rng.standard_normal((B, T, 1)) * 3
    dy = rng.standard_normal((B, T, N))
    w, b = 1 + 0.2 * rng.standard_normal(N), 0.3 * rng.standard_normal(N)
    x, dy = (host(dev(a.astype(np.float32), typ)) for a in (x, dy))
    w, b = (host(dev(a.astype(np.float32), wt)) for a in (w, b))
    return lengths, x, dy, w, b


@pytest.mark.parametrize("case", NORM, ids=[f"B{c[0]}T{c[1]}N{c[2]}{c[3]}w{c[4]}" for c in NORM])
def test_layer_norm_and_its_gradient(crf, case):
    B, T, N, typ, wt, kind = case
    print(f"\n[layer_norm {case}]", flush=True)
    eps = 1e-5
    lengths, x, dy, w, b = norm_inputs(case)
    f = np.float32
    xd = dev(poison(x.copy(), lengths).astype(f), typ)
    wd, bd, ln = dev(w.astype(f), wt), dev(b.astype(f), wt), dev(lengths)
    y, mean, rstd = crf.layer_norm(xd, wd, bd, eps=eps, lengths=ln, want_stats=True, check_status=True)
    wy, wm, wr = ref.layer_norm(x, w, b, eps, lengths)
    # sums of a row run over log2 steps and the pieces of a lane: 64 terms in a chain at most.
    # An error dm of the mean moves the variance by dm^2, negligible beside its own 70 u.
    amax = np.abs(x).mean(-1)
    dm = 70 * U * amax
    close(mean, wm, dm, "mean")
    close(rstd, wr, 80 * U * wr + wr ** 3 * dm ** 2, "rstd")
    tol = np.abs(w) * wr[..., None] * dm[..., None] + 90 * U * (np.abs(wy - b) + np.abs(b))
    valid = (np.arange(T)[None] < lengths[:, None])[..., None]
    close(y, wy * valid, (tol + rounding(typ, wy)) * valid, "y")
    assert (crf.layer_norm(xd, wd, bd, eps=eps, lengths=ln) == y).all()

    gd = dev(poison(dy.copy(), lengths).astype(f), typ)
    m32, r32 = host(mean), host(rstd)                  # what the gradient is given
    d = crf.layer_norm_grad(gd, xd, wd, mean, rstd, lengths=ln, check_status=True)
    dx, dw, db, mx, mw, mb = ref.layer_norm_grad(dy, x, w, m32, r32, lengths)
    # x - mean is rounded once, at the size of |x| + |mean|, and enters h
    dh = U * (np.abs(x) + np.abs(m32)[..., None]) * r32[..., None] * valid
    ag = np.abs(dy * w) * valid
    extra = r32[..., None] * (dh * ag.mean(-1, keepdims=True) * 3
                              + np.abs((x - m32[..., None]) * r32[..., None]) * valid
                              * (ag * dh).mean(-1, keepdims=True))
    close(d["grad_x"], dx, 90 * U * mx + extra + rounding(typ, dx), "grad_x")
    n = 64 + int(lengths.sum()) // 64
    close(d["grad_weight"], dw, n * U * mw + (np.abs(dy) * valid * dh).sum((0, 1)) + rounding(wt, dw),
          "grad_weight")
    close(d["grad_bias"], db, n * U * mb + rounding(wt, db), "grad_bias")
    again = crf.layer_norm_grad(gd, xd, wd, mean, rstd, lengths=ln)
    assert all((again[q] == d[q]).all() for q in d)
    only = crf.layer_norm_grad(gd, xd, wd, mean, rstd, lengths=ln, want_params=False)
    assert set(only) == {"grad_x"} and (only["grad_x"] == d["grad_x"]).all()


def test_layer_norm_without_weights_and_constant_rows(crf):
    x = np.zeros((1, 3, 50), np.float32)
    x[0, 1], x[0, 2, 0] = 7.25, 50.0
    y = host(crf.layer_norm(dev(x), eps=1e-5))
    want, _, _ = ref.layer_norm(x.astype(np.float64), np.ones(50), np.zeros(50), 1e-5, [3])
    assert np.abs(y - want).max() <= 90 * U * np.abs(want).max()
    x[0, 1, 4] = NAN                                   # spoils its own row only
    y = host(crf.layer_norm(dev(x)))
    assert np.isnan(y[0, 1]).all() and np.isfinite(y[0, [0, 2]]).all()


def test_layer_norm_gradient_against_differences(crf):
    """Central differences of the 64-bit definition, h = 1e-5: error about h^2 times third
    derivatives of order rstd^2, and 1e-16 / h; 1e-7 covers both."""
    case = (2, 12, 39, "f32", "f32", "ragged")
    lengths, x, dy, w, b = norm_inputs(case)
    rng = np.random.default_rng(1)
    f = np.float32
    y, mean, rstd = crf.layer_norm(dev(x.astype(f)), dev(w.astype(f)), dev(b.astype(f)),
                                   lengths=dev(lengths), want_stats=True)
    d = crf.layer_norm_grad(dev(dy.astype(f)), dev(x.astype(f)), dev(w.astype(f)), mean, rstd,
                            lengths=dev(lengths))

    def loss(x, w, b):
        return (ref.layer_norm(x, w, b, 1e-5, lengths)[0] * dy).sum()

    h = 1e-5
    for i, what in enumerate(("grad_x", "grad_weight", "grad_bias")):
        args = [x, w, b]
        D = rng.standard_normal(args[i].shape)
        up, down = (loss(*[a + s * h * D if j == i else a for j, a in enumerate(args)]) for s in (1, -1))
        got, size = (host(d[what]) * D).sum(), np.abs(host(d[what]) * D).sum()
        assert abs((up - down) / (2 * h) - got) <= (200 * U + 1e-7) * size + 1e-6, what


# ---------------------------------------------------------------- attention

ATT = [  # B, T, Hq, Hk, Dk, Dv, typ, lengths, initial state
    (1, 1, 1, 1, 1, 1, "f32", "full", False),
    (1, 1, 2, 1, 16, 16, "bf16", "full", True),
    (3, 2, 2, 2, 32, 32, "f32", "ragged", True),
    (3, 63, 2, 1, 32, 32, "bf16", "ragged", True),
    (3, 64, 2, 2, 64, 64, "f32", "ragged", False),
    (2, 65, 4, 2, 64, 64, "bf16", "full", True),
    (4, 129, 3, 1, 39, 48, "f32", "ragged", True),
    (4, 200, 2, 2, 39, 17, "bf16", "ragged", False),
    (3, 150, 4, 1, 64, 100, "bf16", "ragged", True),
    (2, 97, 2, 2, 128, 128, "f32", "ragged", True),
    (3, 190, 2, 1, 128, 128, "bf16", "ragged", True),
    (2, 130, 1, 1, 128, 5, "f32", "full", True),
    (2, 1700, 2, 1, 16, 24, "f32", "ragged", True),      # several segments
    (3, 2300, 1, 1, 64, 32, "bf16", "ragged", True),
    (2, 1100, 2, 1, 80, 72, "bf16", "ragged", False),
]


def att_inputs(case, seed=0):
    B, T, Hq, Hk, Dk, Dv, typ, kind, with_state = case
    rng = np.random.default_rng(T * 7 + Dk + seed)
    lengths = draw_lengths(rng, B, T, kind)
    r = lambda *s: host(dev(rng.standard_normal(s).astype(np.float32), typ))  # noqa: E731
    q, k, v, do = r(B, T, Hq, Dk), r(B, T, Hk, Dk), r(B, T, Hk, Dv), r(B, T, Hq, Dv)
    g = -np.exp2(rng.uniform(-9, 1, Hq)).astype(np.float32)
    g[0] = 0.0 if Hq > 1 else g[0]                      # no decay at all
    st = rng.standard_normal((B, Hq, Dk, Dv)).astype(np.float32) if with_state else None
    gs = rng.standard_normal((B, Hq, Dk, Dv)).astype(np.float32) if with_state else None
    return lengths, q, k, v, do, g, st, gs


def att_tol(typ, T, D, want, mag):
    if typ == "bf16":
        return 1.1 * W * mag + W * np.abs(want)
    return (D + 2 * 64 + T // 32 + 64) * U * mag + U * np.abs(want)


def opt(x):
    return None if x is None else dev(x)


@pytest.mark.parametrize("case", ATT, ids=[f"B{c[0]}T{c[1]}H{c[2]}_{c[3]}D{c[4]}_{c[5]}{c[6]}" for c in ATT])
def test_attention_and_its_gradient(crf, case):
    B, T, Hq, Hk, Dk, Dv, typ, kind, _ = case
    print(f"\n[decay_attention {case}]", flush=True)
    lengths, q, k, v, do, g, st, gs = att_inputs(case)
    scale, f = 0.25, np.float32
    qd, kd, vd, dd = (dev(poison(a.copy(), lengths).astype(f), typ) for a in (q, k, v, do))
    ln, gd = dev(lengths), dev(g)
    o, end = crf.decay_attention(qd, kd, vd, gd, scale=scale, lengths=ln, state=opt(st),
                                 want_state=True, check_status=True)
    wo, ws = ref.attention(q, k, v, g, scale, lengths, st)
    ab = ref.absolute(q, k, v, st)
    mo, ms = ref.attention(ab[0], ab[1], ab[2], g, scale, lengths, ab[3])
    close(o, wo, att_tol(typ, T, Dk, wo, mo), "o")
    # the state is kept in fp32 whatever the type: three bfloat16 parts hold 24 bits
    close(end, ws, att_tol("f32", T, 1, ws, ms), "state")

    d = crf.decay_attention_grad(dd, qd, kd, vd, gd, scale=scale, lengths=ln, state=opt(st),
                                 grad_state=opt(gs), check_status=True)
    want = ref.attention_grad(do, q, k, v, g, scale, lengths, st, gs)
    a = ref.absolute(do, q, k, v, st, gs)
    mag = ref.attention_grad(a[0], a[1], a[2], a[3], g, scale, lengths, a[4], a[5])
    for n, x, m, D in zip(("grad_q", "grad_k", "grad_v"), want, mag, (Dv, Dv, Dk)):
        close(d[n], x, att_tol(typ, T, D + Hq // Hk, x, m), n)
    assert ("grad_state" in d) == (st is not None)
    if st is not None:
        close(d["grad_state"], want[3], att_tol("f32", T, 1, want[3], mag[3]), "grad_state")
    again = crf.decay_attention_grad(dd, qd, kd, vd, gd, scale=scale, lengths=ln, state=opt(st),
                                     grad_state=opt(gs))
    assert all((again[n] == d[n]).all() for n in d)


# rows narrower than a 16-byte piece, one element past whole pieces, and next to wide ones
NARROW_ATT = [
    (2, 150, 2, 1, 3, 7, "bf16", "ragged", True),
    (3, 70, 2, 2, 5, 100, "bf16", "ragged", False),
    (2, 140, 3, 3, 2, 3, "f32", "ragged", True),
    (2, 130, 2, 1, 9, 97, "bf16", "full", True),
    (2, 1500, 2, 1, 33, 65, "f32", "ragged", True),
    (2, 2000, 1, 1, 65, 33, "bf16", "ragged", True),
]


@pytest.mark.parametrize("case", NARROW_ATT, ids=[f"B{c[0]}T{c[1]}D{c[4]}_{c[5]}{c[6]}" for c in NARROW_ATT])
def test_attention_rows_of_odd_widths(crf, case):
    test_attention_and_its_gradient(crf, case)


def test_attention_gradient_against_differences(crf):
    """The output is linear in each of q, k, v and the state: half the difference of two calls
    is the slope exactly, up to the rounding of the calls."""
    case = (2, 150, 4, 2, 48, 40, "f32", "ragged", True)
    lengths, q, k, v, do, g, st, gs = att_inputs(case, 3)
    rng = np.random.default_rng(9)
    f, ln = np.float32, dev(lengths)
    x = {"q": q.astype(f), "k": k.astype(f), "v": v.astype(f), "state": st}
    d = crf.decay_attention_grad(dev(do.astype(f)), dev(x["q"]), dev(x["k"]), dev(x["v"]), dev(g),
                                 scale=0.3, lengths=ln, state=dev(st), grad_state=dev(gs))

    def loss(y):
        o, s = crf.decay_attention(dev(y["q"]), dev(y["k"]), dev(y["v"]), dev(g), scale=0.3,
                                   lengths=ln, state=dev(y["state"]), want_state=True)
        return (host(o) * do).sum() + (host(s) * gs).sum()

    for n in x:
        D = rng.standard_normal(x[n].shape).astype(f)
        up, down = ({**x, n: x[n] + s * D} for s in (1, -1))
        slope = (loss(up) - loss(down)) / 2
        got = (host(d["grad_" + n]) * D).sum()
        a = ref.absolute(*(up[m] if m != n else np.abs(x[n]) + np.abs(D) for m in ("q", "k", "v", "state")))
        mo, ms = ref.attention(a[0], a[1], a[2], g, 0.3, lengths, a[3])
        tol = 500 * U * ((mo * np.abs(do)).sum() + (ms * np.abs(gs)).sum())
        assert abs(slope - got) <= tol, (n, slope, got, tol)


def test_attention_views_and_alignment(crf):
    """q, k, v as views of one projection, heads before positions, an odd element offset."""
    import torch
    torch.manual_seed(0)
    B, T, H, D = 2, 140, 3, 40
    g = dev(np.array([-0.5, -0.01, 0.0], np.float32))
    for typ in (torch.float32, torch.bfloat16):
        qkv = torch.randn(B, T, 3 * H * D + 1, device="cuda").to(typ)[..., 1:]
        q, k, v = (qkv[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in range(3))
        want, ws = crf.decay_attention(q.contiguous(), k.contiguous(), v.contiguous(), g, want_state=True)
        o, s = crf.decay_attention(q, k, v, g, want_state=True)
        assert torch.equal(o, want) and torch.equal(s, ws)
        t = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, v)]
        assert torch.equal(crf.decay_attention(*t, g), want)
        do = torch.randn(B, T, H, D, device="cuda").to(typ)
        a, b = (crf.decay_attention_grad(do, *z, g) for z in ((q, k, v), [x.contiguous() for x in (q, k, v)]))
        assert all(torch.equal(a[n], b[n]) for n in a)


def test_attention_decays_at_the_ends(crf):
    """gamma 0 (log decay -inf) keeps the position alone; very strong and very weak decays."""
    case = (2, 200, 4, 4, 32, 32, "f32", "full", True)
    lengths, q, k, v, do, g, st, gs = att_inputs(case, 1)
    g = np.array([-np.inf, -80.0, -1e-6, 0.0], np.float32)
    f = np.float32
    args = [dev(a.astype(f)) for a in (q, k, v)]
    o, s = crf.decay_attention(*args, dev(g), scale=1.0, state=dev(st), want_state=True)
    wo, ws = ref.attention(q, k, v, g, 1.0, lengths, st)
    a = ref.absolute(q, k, v, st)
    mo, ms = ref.attention(a[0], a[1], a[2], g, 1.0, lengths, a[3])
    close(o, wo, att_tol("f32", 200, 32, wo, mo), "o")
    close(s, ws, att_tol("f32", 200, 1, ws, ms), "state")
    d = crf.decay_attention_grad(dev(do.astype(f)), *args, dev(g), scale=1.0, state=dev(st),
                                 grad_state=dev(gs))
    want = ref.attention_grad(do, q, k, v, g, 1.0, lengths, st, gs)
    a = ref.absolute(do, q, k, v, st, gs)
    mag = ref.attention_grad(a[0], a[1], a[2], a[3], g, 1.0, lengths, a[4], a[5])
    for n, x, m in zip(("grad_q", "grad_k", "grad_v", "grad_state"), want, mag):
        close(d[n], x, att_tol("f32", 200, 34, x, m), n)


def test_attention_offsets_past_32_bits(crf):
    """A batch whose arrays hold more than 2^31 elements: each sequence equals itself alone."""
    import torch
    torch.manual_seed(1)
    B, T, H, D = 4, 70_000, 64, 128
    print(f"\n[decay_attention B={B} T={T} H={H} D={D}]", flush=True)
    q, k, v = (torch.randn(B, T, H, D, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    g = -torch.exp2(torch.linspace(-8, -1, H, device="cuda"))
    o, s = crf.decay_attention(q, k, v, g, want_state=True)
    # the last positions by hand, from the state 256 positions before (head 63 forgets at once)
    t0 = T - 512
    o1 = crf.decay_attention(q[3:, t0:], k[3:, t0:], v[3:, t0:], g)
    h = 63
    a, b = o[3, -200:, h].float(), o1[0, -200:, h].float()
    assert float((a - b).norm() / b.norm()) < 4 * W
    del o, o1
    d = crf.decay_attention_grad(v, q, k, v, g)
    d1 = crf.decay_attention_grad(v[3:, t0:].contiguous(), q[3:, t0:], k[3:, t0:], v[3:, t0:], g)
    for n in ("grad_q", "grad_k", "grad_v"):
        a, b = d[n][3, -200:, h].float(), d1[n][0, -200:, h].float()
        assert float((a - b).norm() / b.norm()) < 4 * W, n


STEP = [  # B, pool, Hq, Hk, Dk, Dv, typ
    (1, 1, 1, 1, 1, 1, "f32"), (1, 4, 8, 8, 64, 64, "bf16"), (5, 9, 4, 2, 39, 50, "f32"),
    (7, 7, 2, 1, 128, 128, "bf16"), (33, 40, 3, 3, 16, 100, "bf16"), (3, 3, 1, 1, 80, 3, "f32"),
]


@pytest.mark.parametrize("case", STEP, ids=[f"B{c[0]}H{c[2]}D{c[4]}_{c[5]}{c[6]}" for c in STEP])
def test_step_is_one_position_of_the_sequence_form(crf, case):
    B, pool, Hq, Hk, Dk, Dv, typ = case
    rng = np.random.default_rng(B + Dk)
    r = lambda *s: host(dev(rng.standard_normal(s).astype(np.float32), typ))  # noqa: E731
    q, k, v = r(B, Hq, Dk), r(B, Hk, Dk), r(B, Hk, Dv)
    st = rng.standard_normal((pool, Hq, Dk, Dv)).astype(np.float32)
    g = -np.exp2(rng.uniform(-9, 1, Hq)).astype(np.float32)
    slots = rng.permutation(pool)[:B].astype(np.int32)
    if B > 2:
        slots[1], slots[2] = -1, pool                   # idle rows
    f = np.float32
    args = [dev(a.astype(f), typ) for a in (q, k, v)] + [dev(g)]
    state = dev(st)
    out = dev(st) * 0 + 5
    o = crf.decay_attention_step(*args, state, scale=0.5, slots=dev(slots), state_out=out)
    assert np.array_equal(host(state), st)
    o2 = crf.decay_attention_step(*args, state, scale=0.5, slots=dev(slots))
    assert (o2 == o).all()
    live = (slots >= 0) & (slots < pool)
    wo, ws, mo, ms = np.zeros((B, Hq, Dv)), st.astype(np.float64), np.zeros((B, Hq, Dv)), np.abs(st)
    for b in np.nonzero(live)[0]:
        p = slots[b]
        x, s = ref.attention(q[b][None, None], k[b][None, None], v[b][None, None], g, 0.5, [1], st[p][None])
        a = ref.absolute(q[b][None, None], k[b][None, None], v[b][None, None], st[p][None])
        xm, sm = ref.attention(a[0], a[1], a[2], g, 0.5, [1], a[3])
        wo[b], ws[p], mo[b], ms[p] = x[0, 0], s[0], xm[0, 0], sm[0]
    close(o, wo, (Dk + 8) * U * mo + rounding(typ, wo), "o")
    close(state, ws, 8 * U * ms, "state")
    kept = np.setdiff1d(np.arange(pool), slots[live])
    assert np.array_equal(host(state)[kept], st[kept]) and (host(out)[kept] == 5).all()
    assert np.array_equal(host(out)[slots[live]], host(state)[slots[live]])


def test_steps_continue_a_sequence(crf):
    """A prefix in the sequence form, then tokens one by one, against the whole at once."""
    import torch
    torch.manual_seed(2)
    B, T, cut, H, D = 2, 90, 70, 2, 32
    q, k, v = (torch.randn(B, T, H, D, device="cuda") for _ in range(3))
    g = torch.tensor([-0.2, -0.003], device="cuda")
    want, end = crf.decay_attention(q, k, v, g, want_state=True)
    _, s = crf.decay_attention(q[:, :cut], k[:, :cut], v[:, :cut], g, want_state=True)
    for t in range(cut, T):
        o = crf.decay_attention_step(q[:, t], k[:, t], v[:, t], g, s)
        assert float((o - want[:, t]).abs().max() / want.abs().max()) < 400 * U
    assert float((s - end).abs().max() / end.abs().max()) < 400 * U


# ---------------------------------------------------------------- autograd, streams, graphs

def test_autograd_matches_the_gradients(crf):
    import torch
    torch.manual_seed(3)
    B, T, H, D, V = 2, 75, 2, 24, 30
    tok = torch.randint(0, V, (B, T), device="cuda")
    ln = torch.tensor([T, 31], device="cuda", dtype=torch.int32)
    table = torch.randn(V, H * D, device="cuda", requires_grad=True)
    w = torch.ones(H * D, device="cuda", requires_grad=True)
    s0 = torch.randn(B, H, D, D, device="cuda", requires_grad=True)
    g = torch.tensor([-0.2, -0.003], device="cuda")
    x = crf.embed(tok, table, lengths=ln)
    y = crf.layer_norm(x, w, None, lengths=ln).unflatten(-1, (H, D))
    o, s = crf.decay_attention(y, y, y, g, state=s0, lengths=ln, want_state=True)
    do, ds = torch.randn_like(o), torch.randn_like(s)
    (o * do).sum().add((s * ds).sum()).backward()
    with torch.no_grad():
        d = crf.decay_attention_grad(do, y, y, y, g, lengths=ln, state=s0, grad_state=ds)
        dy = (d["grad_q"] + d["grad_k"] + d["grad_v"]).flatten(-2)
        xs = x.detach()
        _, mean, rstd = crf.layer_norm(xs, w, None, lengths=ln, want_stats=True)
        n = crf.layer_norm_grad(dy, xs, w, mean, rstd, lengths=ln)
        e = crf.embed_grad(tok, n["grad_x"], V, lengths=ln)
    assert torch.equal(s0.grad, d["grad_state"])
    for a, b in ((table.grad, e), (w.grad, n["grad_weight"])):
        assert float((a - b).norm() / b.norm()) < 1e-5      # q + k + v may be added in another order


def test_other_streams_and_graph_replays(crf):
    """The calls run on torch's current stream and can be captured: every replay of a graph,
    with eager work between, gives the eager result."""
    import torch
    torch.manual_seed(4)
    B, T, H, D, V = 2, 1200, 2, 32, 500
    tok = torch.randint(0, V, (B, T), device="cuda", dtype=torch.int32)
    table = torch.randn(V, H * D, device="cuda")
    w = torch.randn(H * D, device="cuda")
    g = torch.tensor([-0.2, -0.003], device="cuda")

    def work():
        x = crf.embed(tok, table)
        y, m, r = crf.layer_norm(x, w, w, want_stats=True)
        z = y.unflatten(-1, (H, D))
        o, s = crf.decay_attention(z, z, z, g, want_state=True)
        d = crf.decay_attention_grad(o, z, z, z, g)
        n = crf.layer_norm_grad(d["grad_q"].flatten(-2), x, w, m, r)
        return [o, s, n["grad_x"], n["grad_weight"], crf.embed_grad(tok, n["grad_x"], V)]

    want = work()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = work()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for i in range(4):
        table.mul_(-1.5 if i % 2 else 0.5)
        graph.replay()
        torch.cuda.synchronize()
        eager = work()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager)), i


def test_refusals(crf):
    import torch
    x = torch.zeros(2, 3, 8, device="cuda")
    tok = torch.zeros(2, 3, device="cuda", dtype=torch.int32)
    q = torch.zeros(2, 3, 2, 8, device="cuda")
    g = torch.zeros(2, device="cuda")
    st = torch.zeros(2, 2, 8, 8, device="cuda")
    m = torch.zeros(2, 3, device="cuda")
    bad = [
        (TypeError, lambda: crf.embed(tok, x[0].half())),
        (TypeError, lambda: crf.embed(tok.float(), x[0])),
        (ValueError, lambda: crf.embed(tok.cpu(), x[0])),
        (ValueError, lambda: crf.embed(tok[0], x[0])),
        (ValueError, lambda: crf.embed(tok, x[0].t())),
        (TypeError, lambda: crf.embed(tok, x[0], lengths=torch.zeros(2, device="cuda"))),
        (ValueError, lambda: crf.embed(tok, x[0], lengths=tok[0])),
        (ValueError, lambda: crf.embed_grad(tok, x[:1], 4)),
        (crf.SemiCRFError, lambda: crf.embed_grad(tok, x, 0)),
        (ValueError, lambda: crf.embed_grad(tok, x, 4, workspace=torch.zeros(8, device="cuda"))),
        (ValueError, lambda: crf.layer_norm(x, torch.ones(7, device="cuda"))),
        (TypeError, lambda: crf.layer_norm(x, torch.ones(8, device="cuda").bfloat16())),
        (ValueError, lambda: crf.layer_norm(x[0])),
        (crf.SemiCRFError, lambda: crf.layer_norm(x, eps=-1.0)),
        (crf.SemiCRFError, lambda: crf.layer_norm(torch.zeros(1, 1, 32769, device="cuda"))),
        (TypeError, lambda: crf.layer_norm_grad(x.bfloat16(), x, None, m, m)),
        (ValueError, lambda: crf.layer_norm_grad(x, x, None, m[:1], m)),
        (ValueError, lambda: crf.decay_attention(q, q[..., :4], q, g)),
        (ValueError, lambda: crf.decay_attention(q[:, :, :1], q, q, g[:1])),
        (TypeError, lambda: crf.decay_attention(q, q, q.bfloat16(), g)),
        (ValueError, lambda: crf.decay_attention(q.transpose(2, 3), q, q, g)),
        (ValueError, lambda: crf.decay_attention(q, q, q, g[:1])),
        (ValueError, lambda: crf.decay_attention(q, q, q, g.requires_grad_())),
        (ValueError, lambda: crf.decay_attention(q, q, q, g.detach(), state=st[:1])),
        (crf.SemiCRFError, lambda: crf.decay_attention(*[torch.zeros(1, 1, 1, 129, device="cuda")] * 3,
                                                       g.detach()[:1])),
        (ValueError, lambda: crf.decay_attention_grad(q[:1], q, q, q, g.detach())),
        (ValueError, lambda: crf.decay_attention_step(q[:, 0], q[:, 0], q[:, 0], g.detach(), st[:1])),
        (TypeError, lambda: crf.decay_attention_step(q[:, 0], q[:, 0], q[:, 0], g.detach(), st,
                                                     slots=torch.zeros(2, device="cuda"))),
        (TypeError, lambda: crf.decay_attention_step(q[:, 0], q[:, 0], q[:, 0], g.detach(), st.bfloat16())),
    ]
    for i, (err, f) in enumerate(bad):
        with pytest.raises(err):
            f()
            pytest.fail(f"call {i} was not refused")
    torch.cuda.synchronize()
