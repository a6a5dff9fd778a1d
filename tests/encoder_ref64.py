"""Decayed linear attention by its definition in 64 bits, a position at a time over all sequences and
heads at once (torch), for lengths where encoder_ref.py takes too long.  The same arguments and
results, as numpy arrays."""

import numpy as np
import torch


def attention(q, k, v, log_decay, scale, lengths, state=None, device="cpu"):
    q, k, v, gamma, live, _ = _arrays(q, k, v, log_decay, lengths, device)
    s = torch.zeros(*q.shape[::2], q.shape[3], v.shape[3], dtype=torch.float64, device=device) if state is None \
        else torch.tensor(np.asarray(state), dtype=torch.float64, device=device)
    o = torch.zeros(*q.shape[:3], v.shape[3], dtype=torch.float64, device=device)
    for t in range(q.shape[1]):
        s = torch.where(live[t], gamma * s + k[:, t, :, :, None] * v[:, t, :, None, :], s)
        o[:, t] = torch.where(live[t][..., 0], scale * (q[:, t, :, :, None] * s).sum(2), 0.0)
    return o.cpu().numpy(), s.cpu().numpy()


def attention_grad(do, q, k, v, log_decay, scale, lengths, state=None, grad_state=None, device="cpu"):
    Hk = k.shape[2]
    q, k, v, gamma, live, make = _arrays(q, k, v, log_decay, lengths, device)
    do = make(do)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    zero = torch.zeros(*q.shape[::2], q.shape[3], v.shape[3], dtype=torch.float64, device=device)
    s = zero if state is None else make(state)
    for t in range(q.shape[1]):
        s = torch.where(live[t], gamma * s + k[:, t, :, :, None] * v[:, t, :, None, :], s)
        dq[:, t] = torch.where(live[t][..., 0], scale * (s * do[:, t, :, None, :]).sum(3), 0.0)
    r = zero if grad_state is None else make(grad_state)
    for t in range(q.shape[1] - 1, -1, -1):
        x = r + scale * q[:, t, :, :, None] * do[:, t, :, None, :]
        dk[:, t] = torch.where(live[t][..., 0], (x * v[:, t, :, None, :]).sum(3), 0.0)
        dv[:, t] = torch.where(live[t][..., 0], (x * k[:, t, :, :, None]).sum(2), 0.0)
        r = torch.where(live[t], gamma * x, r)
    shared = lambda x: x.unflatten(2, (Hk, -1)).sum(3)  # noqa: E731
    return tuple(x.cpu().numpy() for x in (dq, shared(dk), shared(dv), r))


def _arrays(q, k, v, log_decay, lengths, device):
    def make(x):
        return torch.tensor(np.asarray(x), dtype=torch.float64, device=device)

    rep = q.shape[2] // k.shape[2]
    q, k, v = make(q), make(k).repeat_interleave(rep, 2), make(v).repeat_interleave(rep, 2)
    gamma = torch.exp(make(log_decay))[:, None, None]
    t = torch.arange(q.shape[1], device=device)[:, None]
    live = (t < make(lengths)[None])[..., None, None, None]
    return q, k, v, gamma, live, make
