"""The encoder operators by their definitions, in 64 bits, position by position (numpy).

Beside each result stands the sum of the absolute values of the terms it adds up: rounding
errors are bounded by it, so the tests' tolerances are fractions of it.
"""

import numpy as np


def embed(tokens, table, scale, lengths):
    B, T = tokens.shape
    V, N = table.shape
    y = np.zeros((B, T, N))
    for b in range(B):
        for t in range(int(lengths[b])):
            v = int(tokens[b, t])
            y[b, t] = scale * table[v] if 0 <= v < V else np.nan
    return y


def embed_grad(tokens, grad_out, V, scale, lengths):
    """(gradient, sum of absolute terms, terms per row)."""
    B, T, N = grad_out.shape
    g, mag, cnt = np.zeros((V, N)), np.zeros((V, N)), np.zeros(V, int)
    for b in range(B):
        L = int(lengths[b])
        tok, x = tokens[b, :L].astype(np.int64), scale * grad_out[b, :L]
        ok = (tok >= 0) & (tok < V)
        np.add.at(g, tok[ok], x[ok])
        np.add.at(mag, tok[ok], np.abs(x[ok]))
        np.add.at(cnt, tok[ok], 1)
    return g, mag, cnt


def layer_norm(x, w, b, eps, lengths):
    y, mean, rstd = np.zeros_like(x), np.zeros(x.shape[:2]), np.zeros(x.shape[:2])
    for i in range(x.shape[0]):
        L = int(lengths[i])
        m = x[i, :L].mean(-1)
        r = 1.0 / np.sqrt(((x[i, :L] - m[:, None]) ** 2).mean(-1) + eps)
        y[i, :L] = (x[i, :L] - m[:, None]) * r[:, None] * w + b
        mean[i, :L], rstd[i, :L] = m, r
    return y, mean, rstd


def layer_norm_grad(dy, x, w, mean, rstd, lengths):
    """grad_x, grad_weight, grad_bias and the absolute sums of the three."""
    N = x.shape[-1]
    dx, mx = np.zeros_like(x), np.zeros_like(x)
    dw, db, mw, mb = (np.zeros(N) for _ in range(4))
    for i in range(x.shape[0]):
        L = int(lengths[i])
        h = (x[i, :L] - mean[i, :L, None]) * rstd[i, :L, None]
        d = dy[i, :L]
        g = d * w
        r = rstd[i, :L, None]
        dx[i, :L] = r * (g - g.mean(-1, keepdims=True) - h * (g * h).mean(-1, keepdims=True))
        mx[i, :L] = r * (np.abs(g) + np.abs(g).mean(-1, keepdims=True)
                         + np.abs(h) * np.abs(g * h).mean(-1, keepdims=True))
        dw += (d * h).sum(0)
        mw += np.abs(d * h).sum(0)
        db += d.sum(0)
        mb += np.abs(d).sum(0)
    return dx, dw, db, mx, mw, mb


def attention(q, k, v, log_decay, scale, lengths, state=None):
    """o, final state (the recurrence, a position at a time)."""
    B, T, Hq, Dk = q.shape
    rep = Hq // k.shape[2]
    o = np.zeros((B, T, Hq, v.shape[-1]))
    S = np.zeros((B, Hq, Dk, v.shape[-1])) if state is None else np.array(state, np.float64)
    gamma = np.exp(np.asarray(log_decay, np.float64))
    for b in range(B):
        for h in range(Hq):
            s = S[b, h]
            for t in range(int(lengths[b])):
                s = gamma[h] * s + np.outer(k[b, t, h // rep], v[b, t, h // rep])
                o[b, t, h] = scale * (q[b, t, h] @ s)
            S[b, h] = s
    return o, S


def attention_grad(do, q, k, v, log_decay, scale, lengths, state=None, grad_state=None):
    """dq, dk, dv, grad of the initial state: the recurrence backward, a position at a time."""
    B, T, Hq, Dk = q.shape
    rep, Dv = Hq // k.shape[2], v.shape[-1]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    ds = np.zeros((B, Hq, Dk, Dv))
    gamma = np.exp(np.asarray(log_decay, np.float64))
    for b in range(B):
        L = int(lengths[b])
        for h in range(Hq):
            kk, vv = k[b, :, h // rep], v[b, :, h // rep]
            s = np.zeros((Dk, Dv)) if state is None else np.array(state[b, h], np.float64)
            for t in range(L):
                s = gamma[h] * s + np.outer(kk[t], vv[t])
                dq[b, t, h] = scale * (s @ do[b, t, h])
            r = np.zeros((Dk, Dv)) if grad_state is None else np.array(grad_state[b, h], np.float64)
            for t in range(L - 1, -1, -1):
                r = r + scale * np.outer(q[b, t, h], do[b, t, h])
                dk[b, t, h // rep] += r @ vv[t]
                dv[b, t, h // rep] += r.T @ kk[t]
                r = gamma[h] * r
            ds[b, h] = r
    return dq, dk, dv, ds


def absolute(*arrays):
    return [None if a is None else np.abs(a) for a in arrays]
