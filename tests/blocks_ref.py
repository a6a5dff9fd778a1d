"""The operators of a block and the token loss by their definitions, in 64 bits (numpy), with
first-order bounds of the rounding errors of a computation in float32.

A bound is in units of U = 2^-24, half an ulp of float32 at 1.  What enters it:
  * one operation rounds by 1 U of its result; the hardware's exponential, reciprocal, square root and
    reciprocal square root are within 1 ulp, 2 U;
  * sig(z) = 1 / (1 + exp2(-z log2 e)): the product rounds by U |z|, so it is within (|z| + 5) U, and
    1 - sig(z) = exp2(..) sig(z) within (2 |z| + 8) U.  G(z) below, with room for one product more;
  * m = expm1(s) is within 12 U of itself where s is exact, and moves by at most the relative error
    of s; 1 - a^2 = -m (m + 2) adds 3 U, its root halves that and adds 2;
  * a = exp(s) moves by |s| times the relative error of s, and its own exponent rounds by U |s|; the
    hardware's exponential is 0 below 2^-126, which is an absolute error of that size: FLUSHED.
"""

import numpy as np

U = 2.0 ** -24
FLUSHED = 2.0 ** -126 / U


def sig(z):
    return 1.0 / (1.0 + np.exp(-z))


def G(z):
    return 2 * np.abs(z) + 9


def gates(x, r, i, lam):
    """sig(r), sig(i), s, a, m = a - 1, b, and relative bounds [U] of a, m, b and of b sig(i) x."""
    sr, si = sig(r), sig(i)
    s = lam * sr
    a, m = np.exp(s), np.expm1(s)
    b = np.sqrt(-np.expm1(2 * s))
    em = G(r) + 14
    eb = em / 2 + 4
    return sr, si, s, a, m, b, np.abs(s) * (G(r) + 3) + 4, em, eb, eb + G(i) + 3


def recurrence(x, r, i, lam, lengths, state=None):
    """h, final state, their bounds, and the states before every 16th position."""
    B, T, N = x.shape
    h, eh = np.zeros((B, T, N)), np.zeros((B, T, N))
    end, eend = np.zeros((B, N)), np.zeros((B, N))
    starts = np.zeros((B, -(-T // 16), N))
    for b in range(B):
        v = np.zeros(N) if state is None else np.array(state[b], np.float64)
        e, w = np.zeros(N), np.abs(v)
        for t in range(int(lengths[b])):
            if t % 16 == 0:
                starts[b, t // 16] = v
            _, si, _, a, m, bb, _, em, _, ebu = gates(x[b, t], r[b, t], i[b, t], lam)
            u = bb * si * x[b, t]
            e = a * e + em * np.abs(m) * w + ebu * np.abs(u)
            v, w = a * v + u, a * w + np.abs(u)
            e = e + 2 * w
            h[b, t], eh[b, t] = v, e
        end[b], eend[b] = v, e
    return h, end, U * eh, U * eend, starts


def recurrence_grad(g, x, r, i, lam, lengths, state=None, grad_state=None):
    """dict of gradients and dict of bounds."""
    B, T, N = x.shape
    h, _, eh, _, _ = recurrence(x, r, i, lam, lengths, state)
    out = {k: np.zeros((B, T, N)) for k in ("x", "decay_gate", "input_gate")}
    err = {k: np.zeros((B, T, N)) for k in out}
    out["log_decay"], err["log_decay"] = np.zeros(N), np.zeros(N)
    out["state"], err["state"] = np.zeros((B, N)), np.zeros((B, N))
    mag, count = np.zeros(N), 0
    for b in range(B):
        first = np.zeros(N) if state is None else np.array(state[b], np.float64)
        E = np.zeros(N) if grad_state is None else np.array(grad_state[b], np.float64)
        e, w = np.zeros(N), np.abs(E)
        for t in range(int(lengths[b]) - 1, -1, -1):
            sr, si, s, a, m, bb, ea, em, eb, _ = gates(x[b, t], r[b, t], i[b, t], lam)
            E, w = E + g[b, t], w + np.abs(g[b, t])
            e = e + w
            u = si * x[b, t]
            prev, eprev = (h[b, t - 1], eh[b, t - 1] / U) if t else (first, 0.0)
            q = a * a / bb * u
            ds = E * (a * prev - q)
            eds = e * np.abs(a * prev - q) + w * (a * eprev + ((ea + 4) * a + FLUSHED) * np.abs(prev)
                                                  + (2 * ea + eb + G(i[b, t]) + 8) * np.abs(q))
            du = E * bb
            out["x"][b, t] = du * si
            err["x"][b, t] = e * bb * si + w * bb * si * (eb + G(i[b, t]) + 3)
            out["input_gate"][b, t] = du * u * (1 - si)
            err["input_gate"][b, t] = np.abs(u) * (1 - si) * (e * bb + w * bb * (eb + 2 * G(i[b, t]) + 5))
            out["decay_gate"][b, t] = ds * s * (1 - sr)
            err["decay_gate"][b, t] = np.abs(s) * (1 - sr) * (eds + np.abs(ds) * (2 * G(r[b, t]) + 4))
            out["log_decay"] += ds * sr
            err["log_decay"] += eds * sr + np.abs(ds) * sr * (G(r[b, t]) + 2)
            mag += np.abs(ds) * sr
            count += 1
            e = a * e + em * np.abs(m) * w
            E, w = a * E, a * w
            e = e + 2 * w
        out["state"][b], err["state"][b] = E, e
    err["log_decay"] += count * mag                # a sum in any order
    return out, {k: U * v for k, v in err.items()}


def norm(z, center, eps):
    mean = z.mean(-1, keepdims=True) if center else np.zeros(z.shape[:-1] + (1,))
    rstd = 1.0 / np.sqrt(((z - mean) ** 2).mean(-1, keepdims=True) + eps)
    return (z - mean) * rstd, mean, rstd


# A row's sum in float32: at most 46 additions in a row for widths up to 16,384 (a lane's 32 elements, the
# wavefront's lanes by halves, 8 wavefronts in order), so that a mean is within 48 U of the mean of
# absolute values.
D = 48


def normed(z, ez, center, eps):
    """norm(z), rstd and the bound [U] of the first where z has the bound ez."""
    h, mean, rstd = norm(z, center, eps)
    a = np.abs(z - mean)
    em = D * np.abs(z).mean(-1, keepdims=True) + ez.mean(-1, keepdims=True) if center else 0.0
    ea = ez + em + a
    # the variance: its terms' errors and the sum's; rstd takes half of it and 3 operations
    var = 1.0 / rstd ** 2
    ev = ((2 * a * ea).mean(-1, keepdims=True) + (D + 1) * (a * a).mean(-1, keepdims=True)) / var
    return h, rstd, rstd * ea + np.abs(h) * (ev / 2 + 5)


def norm_back(g, eg, h, eh, rstd, center):
    """The gradient through norm from that of its rows, and its bound [U] (rstd within 64 U)."""
    gh = (g * h).mean(-1, keepdims=True)
    egh = (eg * np.abs(h) + np.abs(g) * eh).mean(-1, keepdims=True) + (D + 2) * np.abs(g * h).mean(-1, keepdims=True)
    t = g - h * gh
    et = eg + np.abs(h) * egh + eh * np.abs(gh) + 3 * (np.abs(g) + np.abs(h * gh))
    if center:
        t = t - g.mean(-1, keepdims=True)
        et = et + eg.mean(-1, keepdims=True) + (D + 2) * np.abs(g).mean(-1, keepdims=True)
    return rstd * t, rstd * et + 66 * np.abs(rstd * t)


def residual(x, o, w, b, gate, scale, norm_branch, bw, bb, center, eps, grad_r=None, grad_y=None):
    """Rows of any leading shape (no padding).  dict of values and dict of bounds; gradients where
    grad_r and grad_y are given, those of the weights summed over the leading axes."""
    N = x.shape[-1]
    one, zero = np.ones(N), np.zeros(N)
    w, b, c = (one if w is None else w), (zero if b is None else b), (one if scale is None else scale)
    f, ef, k, ek = o, np.zeros_like(o), None, None
    if norm_branch:
        p, q = (one if bw is None else bw), (zero if bb is None else bb)
        k, rstd_o, ek = normed(o, np.zeros_like(o), center, eps)
        f, ef = k * p + q, ek * np.abs(p) + 2 * (np.abs(k * p) + np.abs(q))
    sg, es = (np.ones_like(x), np.zeros_like(x)) if gate is None else (sig(gate), G(gate) * sig(gate))
    cs, ecs = c * sg, np.abs(c) * (es + sg)
    r = x + cs * f
    er = np.abs(cs) * ef + ecs * np.abs(f) + np.abs(cs * f) + np.abs(r)
    h, rstd, eh = normed(r, er, center, eps)
    y, ey = h * w + b, eh * np.abs(w) + 2 * (np.abs(h * w) + np.abs(b))
    out, err = {"r": r, "y": y}, {"r": er, "y": ey}
    if grad_y is not None:
        lead = tuple(range(x.ndim - 1))
        n = int(np.prod(x.shape[:-1])) + 8
        g = grad_y * w
        e, ee = norm_back(g, np.abs(g), h, eh, rstd, center)
        e, ee = e + grad_r, ee + np.abs(e) + np.abs(grad_r)

        def add(name, term, bound):
            out[name] = term.sum(lead)
            err[name] = bound.sum(lead) + n * np.abs(term).sum(lead)

        out["grad_x"], err["grad_x"] = e, ee
        add("grad_weight", grad_y * h, np.abs(grad_y) * (eh + np.abs(h)))
        add("grad_bias", grad_y, np.zeros_like(g))
        add("grad_scale", e * sg * f, np.abs(f) * (ee * sg + np.abs(e) * (es + 2 * sg)) + np.abs(e * sg) * ef)
        qg = 1 - sg
        d, ed = e * cs, ee * np.abs(cs) + np.abs(e) * (ecs + np.abs(cs))
        if gate is not None:
            out["grad_gate"] = d * f * qg
            err["grad_gate"] = qg * (ed * np.abs(f) + np.abs(d) * ef + (G(gate) + 3) * np.abs(d * f))
        if norm_branch:
            add("grad_branch_weight", d * k, ed * np.abs(k) + np.abs(d) * (ek + np.abs(k)))
            add("grad_branch_bias", d, ed)
            d, ed = norm_back(d * p, (ed + np.abs(d)) * np.abs(p), k, ek, rstd_o, center)
        out["grad_branch"], err["grad_branch"] = d, ed
    return out, {k: U * v for k, v in err.items()}


def nll(x, table, target, scale, depth, held, grad=None):
    """Listed rows x [M, N].  loss, lse, bounds; with the rows' gradients also dx, dW and bounds.
    depth: additions in a row of a product's sum over n terms, as a function of n; held: relative
    rounding of the second products' first operand, in units of U."""
    V, N = table.shape
    z = scale * (x @ table.T)
    ez = (depth(N) + 3) * abs(scale) * (np.abs(x) @ np.abs(table).T)
    top = z.max(1, keepdims=True)
    lse = top[:, 0] + np.log(np.exp(z - top).sum(1))
    at = np.arange(len(x)), target
    # exponents in units of log2: a product and a difference of values up to |z|, |lse|
    p = np.exp(z - lse[:, None])
    arg = 4 * (np.abs(z) + np.abs(lse[:, None])) + 4
    elog = (p * (ez + arg)).sum(1) + V / 8 + 40
    else_ = elog + 4 * np.abs(lse) + 4
    loss = lse - z[at]
    eloss = elog + ez[at] + 6 * (np.abs(lse) + np.abs(z[at])) + 4
    if grad is None:
        return loss, lse, U * eloss, U * else_
    ep = p * (ez + else_[:, None] + arg)
    p[at] -= 1.0
    ep += np.abs(p) * (held + 3)
    g = (scale * grad)[:, None]
    dx, dW = g * (p @ table), (g * p).T @ x
    edx = np.abs(g) * (ep @ np.abs(table) + (depth(V) + 8) * (np.abs(p) @ np.abs(table)))
    edW = (np.abs(g) * ep).T @ np.abs(x) + (depth(len(x)) + 8) * ((np.abs(g * p)).T @ np.abs(x))
    return loss, lse, U * eloss, U * else_, dx, dW, U * edx, U * edW
