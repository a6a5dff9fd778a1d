"""The encoder operators that feed the semi-CRF head, as they are timed: the cases, their
inputs, the operators' plain forms and their definitions in 64 bits.

A tagger embeds its tokens, normalises, mixes positions with decayed linear attention and
projects to emissions; the sizes below are the library's own workloads (B, T and lengths of
the tiny, speech, genomic and long configurations) with generic widths and head counts.

Operators ("op" of a case):
  embed           y[b,t] = scale * W[tok[b,t]], 0 at padding
  embed_grad      dW[v] = scale * sum of dy[b,t] over tok[b,t] = v
  norm            layer norm over the last axis, 0 at padding
  norm_grad       its gradients: x, weight, bias
  attention       S_t = g S_{t-1} + k_t v_t^T, o_t = scale q_t S_t for every position
  attention_grad  gradients of q, k, v (and of the initial state)
  step            one token of the recurrence for every sequence, on states in a pool
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5
CHUNK = 128       # positions per chunk of the plain attention


def listed():
    return [
        # one token of one stream through one layer: a call whose latency counts
        {"name": "step_one", "op": "step", "B": 1, "pool": 1, "Hq": 8, "Hk": 8, "Dk": 64, "Dv": 64, "type": "bf16"},
        # a serving batch: 256 streams in a pool of states, some slots idle
        {"name": "step_batch", "op": "step", "B": 256, "pool": 320, "Hq": 16, "Hk": 16, "Dk": 128, "Dv": 128, "type": "bf16"},
        # a training step of the speech workload: ragged lengths, shared key/value heads
        {"name": "attention_speech", "op": "attention", "B": 32, "T": 800, "Hq": 8, "Hk": 2, "Dk": 64, "Dv": 64, "type": "bf16", "ragged": True, "state": False},
        # the genomic workload: four sequences of 100,000 positions
        {"name": "attention_genomic", "op": "attention", "B": 4, "T": 100000, "Hq": 8, "Hk": 8, "Dk": 64, "Dv": 64, "type": "bf16", "ragged": False, "state": True},
        # the speech workload's backward pass
        {"name": "attention_grad_speech", "op": "attention_grad", "B": 32, "T": 800, "Hq": 8, "Hk": 2, "Dk": 64, "Dv": 64, "type": "bf16", "ragged": True, "state": False},
        # one long sequence backward in full precision: few heads, the long axis has to be split
        {"name": "attention_grad_long", "op": "attention_grad", "B": 1, "T": 100001, "Hq": 6, "Hk": 6, "Dk": 64, "Dv": 64, "type": "f32", "ragged": False, "state": True},
        # 6-mers of the genomic workload looked up in a table of 4,096
        {"name": "embed_kmers", "op": "embed", "B": 4, "T": 100000, "V": 4096, "N": 512, "type": "bf16", "ragged": False, "zipf": False},
        # single letters: six rows that each gather tens of thousands of positions
        {"name": "embed_grad_letters", "op": "embed_grad", "B": 4, "T": 100000, "V": 6, "N": 256, "type": "f32", "ragged": False, "zipf": True},
        # a word vocabulary: most rows absent, a few frequent ones
        {"name": "embed_grad_words", "op": "embed_grad", "B": 16, "T": 1000, "V": 50001, "N": 1024, "type": "bf16", "ragged": True, "zipf": True},
        # the tiny workload at an odd width: a call whose latency counts
        {"name": "norm_tiny", "op": "norm", "B": 2, "T": 64, "N": 333, "type": "f32", "ragged": False},
        # the speech workload, ragged, a common width
        {"name": "norm_speech", "op": "norm", "B": 32, "T": 800, "N": 1024, "type": "bf16", "ragged": True},
        # the genomic workload's backward pass with the reduction over 400,000 rows
        {"name": "norm_grad_genomic", "op": "norm_grad", "B": 4, "T": 100000, "N": 512, "type": "bf16", "ragged": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "attention", "attention",
                     "attention_grad", "attention_grad", "step"])
    case = {"op": op, "type": rng.choice(["f32", "bf16"])}
    if op == "step":
        B = _log(rng, 1, 256)
        Hk = rng.choice([1, 2, 4, 8])
        case.update(B=B, pool=B + rng.choice([0, 1, 64]), Hq=Hk * rng.choice([1, 1, 2]), Hk=Hk,
                    Dk=rng.choice([16, 32, 39, 64, 80, 128]), Dv=rng.choice([32, 48, 64, 100, 128]))
        return case
    if op.startswith("attention"):
        Hk = rng.choice([1, 2, 3, 4, 8])
        Hq = Hk * rng.choice([1, 1, 1, 2, 4])
        D = rng.choice([(16, 16), (32, 32), (39, 48), (64, 64), (64, 64), (64, 100), (80, 80),
                        (128, 64), (128, 128)])
        T = _log(rng, 1, 100000)
        # at most a sixth of the largest listed case's elements, fewer for gradients
        room = 4 * 100000 * 8 * 64 // (6 if op == "attention" else 12)
        B = _log(rng, 1, max(1, min(64, room // (T * Hq * max(D)))))
        while B * T * Hq * max(D) > room:
            T = max(1, T // 2)
        case.update(B=B, T=T, Hq=Hq, Hk=Hk, Dk=D[0], Dv=D[1], ragged=rng.random() < 0.5,
                    state=rng.random() < 0.4)
        return case
    N = rng.choice([_log(rng, 6, 4096), rng.choice([64, 128, 256, 512, 768, 1024, 2048])])
    N = 3073 if N == 3072 else N
    n = min(_log(rng, 64, 400000), 100_000_000 // N)
    B = rng.choice([1, 2, 8, 32])
    case.update(B=B, T=max(1, n // B), N=N, ragged=rng.random() < 0.5)
    if op.startswith("embed"):
        case.update(V=min(_log(rng, 4, 131072), 100_000_000 // N), zipf=rng.random() < 0.5)
    return case


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")
    typ = DTYPES[case["type"]]
    op, B = case["op"], case["B"]

    def normal(*shape, sd=1.0, dtype=typ):
        return (sd * torch.randn(*shape, generator=gen, device=dev)).to(dtype)

    s = {"case": case}
    if op == "step":
        pool, Hq, Hk, Dk, Dv = (case[k] for k in ("pool", "Hq", "Hk", "Dk", "Dv"))
        s.update(q=normal(B, Hq, Dk), k=normal(B, Hk, Dk, sd=Dk ** -0.5), v=normal(B, Hk, Dv),
                 log_decay=_log_decay(Hq, dev), scale=1.0,
                 state=normal(pool, Hq, Dk, Dv, dtype=torch.float32))
        s["state_out"] = torch.empty_like(s["state"])
        slots = torch.randperm(pool, generator=gen, device=dev)[:B].to(torch.int32)
        if B > 8:
            slots[::7] = -1          # idle rows of the batch
        s["slots"] = slots
        # the rows that no slot names keep what they have: the new pool starts as a copy
        s["state_out"].copy_(s["state"])
        return s
    T = case["T"]
    if case["ragged"]:
        low = T // 2
        lengths = torch.randint(low, T + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
    else:
        lengths = torch.full((B,), T, device=dev, dtype=torch.int32)
    s["lengths"] = lengths
    if op.startswith("attention"):
        Hq, Hk, Dk, Dv = (case[k] for k in ("Hq", "Hk", "Dk", "Dv"))
        s.update(q=normal(B, T, Hq, Dk), k=normal(B, T, Hk, Dk, sd=Dk ** -0.5),
                 v=normal(B, T, Hk, Dv), log_decay=_log_decay(Hq, dev), scale=1.0)
        s["state"] = normal(B, Hq, Dk, Dv, dtype=torch.float32) if case["state"] else None
        if op == "attention_grad":
            s["grad_out"] = normal(B, T, Hq, Dv)
            s["grad_state"] = normal(B, Hq, Dk, Dv, dtype=torch.float32) if case["state"] else None
        return s
    N = case["N"]
    if op.startswith("embed"):
        V = case["V"]
        u = torch.rand(B, T, generator=gen, device=dev, dtype=torch.float64)
        if case["zipf"]:             # ranks with probability about 1 / rank
            ids = (torch.exp(u * math.log(V + 1.0)) - 1.0).long()
            ids = torch.randperm(V, generator=gen, device=dev)[ids.clamp_(0, V - 1)]
        else:
            ids = (u * V).long().clamp_(0, V - 1)
        s.update(tokens=ids.to(torch.int32), V=V, scale=math.sqrt(N))
        if op == "embed":
            s["table"] = normal(V, N, sd=N ** -0.5)
        else:
            s["grad_out"] = normal(B, T, N)
        return s
    s["x"] = normal(B, T, N, sd=2.0) + 0.5
    s["weight"] = 1.0 + normal(N, sd=0.1)
    s["bias"] = normal(N, sd=0.1)
    if op == "norm_grad":
        s["grad_out"] = normal(B, T, N)
        x = s["x"].float()           # what the forward pass left
        s["mean"] = x.mean(-1)
        s["rstd"] = torch.rsqrt((x - s["mean"][..., None]).square().mean(-1) + EPS)
    return s


def _log_decay(H, dev):
    """Time constants from 8 to 8,192 positions, spread over the heads."""
    h = torch.arange(H, device=dev, dtype=torch.float32) / max(1, H - 1)
    return -torch.exp2(-3.0 - 10.0 * h)


def run(s):
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    return {"embed": _embed, "embed_grad": _embed_grad, "norm": _norm, "norm_grad": _norm_grad,
            "attention": _attention, "attention_grad": _attention_grad, "step": _step}[op](s)


def _run_own(s):
    import semi_markov_crf_amd as crf
    op = s["case"]["op"]
    if op == "embed":
        return {"y": crf.embed(s["tokens"], s["table"], scale=s["scale"], lengths=s["lengths"])}
    if op == "embed_grad":
        return {"grad_table": crf.embed_grad(s["tokens"], s["grad_out"], s["V"], scale=s["scale"],
                                             lengths=s["lengths"])}
    if op == "norm":
        return {"y": crf.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS,
                                    lengths=s["lengths"])}
    if op == "norm_grad":
        return crf.layer_norm_grad(s["grad_out"], s["x"], s["weight"], s["mean"], s["rstd"],
                                   lengths=s["lengths"])
    if op == "attention":
        o, state = crf.decay_attention(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"],
                                       lengths=s["lengths"], state=s["state"], want_state=True)
        return {"out": o, "state": state}
    if op == "attention_grad":
        return crf.decay_attention_grad(s["grad_out"], s["q"], s["k"], s["v"], s["log_decay"],
                                        scale=s["scale"], lengths=s["lengths"], state=s["state"],
                                        grad_state=s["grad_state"])
    o = crf.decay_attention_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"],
                                 scale=s["scale"], slots=s["slots"], state_out=s["state_out"])
    return {"out": o, "state": s["state_out"]}


# ---------------------------------------------------------------- plain forms (32 bits)

def _valid(s, T, dev):
    """[B, T]: the positions before each sequence's length."""
    return torch.arange(T, device=dev)[None, :] < s["lengths"][:, None]


def _embed(s):
    tok = s["tokens"].long()
    y = s["table"].float()[tok] * s["scale"]
    y = torch.where(_valid(s, tok.shape[1], tok.device)[..., None], y, 0.0)
    return {"y": y.to(s["table"].dtype)}


def _embed_grad(s):
    g, tok = s["grad_out"], s["tokens"].long()
    x = torch.where(_valid(s, tok.shape[1], tok.device)[..., None], g.float() * s["scale"], 0.0)
    out = torch.zeros(s["V"], g.shape[-1], device=g.device)
    out.index_add_(0, tok.reshape(-1), x.reshape(-1, g.shape[-1]))
    return {"grad_table": out.to(g.dtype)}


def _norm(s):
    x = s["x"].float()
    c = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS)
    y = c * r * s["weight"].float() + s["bias"].float()
    y = torch.where(_valid(s, x.shape[1], x.device)[..., None], y, 0.0)
    return {"y": y.to(s["x"].dtype)}


def _norm_grad(s):
    typ = s["x"].dtype
    m = _valid(s, s["x"].shape[1], s["x"].device)[..., None]
    xh = (s["x"].float() - s["mean"][..., None]) * s["rstd"][..., None]
    dy = torch.where(m, s["grad_out"].float(), 0.0)
    xh = torch.where(m, xh, 0.0)
    g = dy * s["weight"].float()
    dx = s["rstd"][..., None] * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    dx = torch.where(m, dx, 0.0)
    return {"grad_x": dx.to(typ), "grad_weight": (dy * xh).sum((0, 1)).to(typ),
            "grad_bias": dy.sum((0, 1)).to(typ)}


def _chunked(x, m, rep):
    """[B, T, H, D] -> float32 [B, H * rep, n, CHUNK, D], zero at padding."""
    B, T, H, D = x.shape
    x = torch.where(m[..., None, None], x.float(), 0.0)
    x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, -T % CHUNK))
    x = x.permute(0, 2, 1, 3).repeat_interleave(rep, 1)
    return x.reshape(B, H * rep, -1, CHUNK, D).contiguous()


def _whole(x, T):
    """[B, H, n, CHUNK, D] -> [B, T, H, D]."""
    B, H, _, _, D = x.shape
    return x.reshape(B, H, -1, D)[:, :, :T].permute(0, 2, 1, 3)


def _powers(g, n):
    """exp(g * n), 0 where n < 0: the decay over n positions."""
    return torch.where(n >= 0, torch.exp(g * n.clamp(min=0)), 0.0)


def _decays(s, n, dev):
    g = s["log_decay"].float()[:, None, None]
    i = torch.arange(CHUNK, device=dev, dtype=torch.float32)
    c = torch.arange(n, device=dev, dtype=torch.float32)
    inside = _powers(g, i[:, None] - i[None, :])                       # [H, CHUNK, CHUNK]
    across = _powers(g, CHUNK * (c[:, None] - c[None, :] - 1.0))       # [H, n, n]: c' < c
    before = torch.exp(g * (i[:, None] + 1.0))                         # [H, CHUNK, 1]
    after = torch.exp(g * (CHUNK - 1.0 - i[:, None]))
    return inside, across, before[:, None], after[:, None], torch.exp(g * CHUNK * c[:, None])


def _starts(k, v, across, after, first, state):
    """State before each chunk [B, H, n, Dk, Dv]."""
    kv = (k * after).transpose(-1, -2).contiguous() @ v
    B, H, n, Dk, Dv = kv.shape
    out = (across @ kv.reshape(B, H, n, -1)).reshape(B, H, n, Dk, Dv)
    return out if state is None else out + first[..., None] * state[:, :, None]


def _attention(s):
    q, T, dev = s["q"], s["q"].shape[1], s["q"].device
    m, rep = _valid(s, T, dev), s["q"].shape[2] // s["k"].shape[2]
    Q, K, V = _chunked(q, m, 1), _chunked(s["k"], m, rep), _chunked(s["v"], m, rep)
    inside, across, before, after, first = _decays(s, Q.shape[2], dev)
    S = _starts(K, V, across, after, first, s["state"])
    A = (Q @ K.transpose(-1, -2).contiguous()) * inside[:, None]
    o = s["scale"] * (A @ V + (Q * before) @ S)
    # the state after each sequence's last position
    L = s["lengths"].float()[:, None, None]
    t = torch.arange(T, device=dev, dtype=torch.float32)
    w = _powers(s["log_decay"].float()[None, :, None], L - 1.0 - t)[..., None]     # [B, H, T, 1]
    flat = [x.reshape(*x.shape[:2], -1, x.shape[-1])[:, :, :T] for x in (K, V)]
    end = (flat[0] * w).transpose(-1, -2).contiguous() @ flat[1]
    if s["state"] is not None:
        end = end + torch.exp(s["log_decay"].float()[None, :, None] * L)[..., None] * s["state"]
    return {"out": torch.where(m[..., None, None], _whole(o, T), 0.0).to(q.dtype), "state": end}


def _attention_grad(s):
    q, T, dev, scale = s["q"], s["q"].shape[1], s["q"].device, s["scale"]
    Hk = s["k"].shape[2]
    m, rep = _valid(s, T, dev), q.shape[2] // Hk
    Q, K, V = _chunked(q, m, 1), _chunked(s["k"], m, rep), _chunked(s["v"], m, rep)
    G = _chunked(s["grad_out"], m, 1) * scale
    inside, across, before, after, first = _decays(s, Q.shape[2], dev)
    S = _starts(K, V, across, after, first, s["state"])
    P = (Q @ K.transpose(-1, -2).contiguous()) * inside[:, None]
    dP = (G @ V.transpose(-1, -2).contiguous()) * inside[:, None]
    dq = dP @ K + (G * before) @ S.transpose(-1, -2).contiguous()
    # what later chunks send back, at the end of each chunk
    u = (Q * before).transpose(-1, -2).contiguous() @ G
    B, H, n, Dk, Dv = u.shape
    R = (across.transpose(-1, -2).contiguous() @ u.reshape(B, H, n, -1)).reshape(B, H, n, Dk, Dv)
    dk = dP.transpose(-1, -2).contiguous() @ Q + (V * after) @ R.transpose(-1, -2).contiguous()
    dv = P.transpose(-1, -2).contiguous() @ G + (K * after) @ R
    dq, dk, dv = _whole(dq, T), _whole(dk, T), _whole(dv, T)
    out = {}
    if s["state"] is not None:
        L = s["lengths"].float()[:, None, None]
        g = s["log_decay"].float()[None, :, None]
        t = torch.arange(T, device=dev, dtype=torch.float32)
        w = _powers(g, L - 1.0 - t)[..., None]                         # [B, H, T, 1]
        k, v, Qf, Gf = (x.reshape(*x.shape[:2], -1, x.shape[-1])[:, :, :T] for x in (K, V, Q, G))
        dS = s["grad_state"]
        dk = dk + ((v * w) @ dS.transpose(-1, -2).contiguous()).permute(0, 2, 1, 3)
        dv = dv + ((k * w) @ dS).permute(0, 2, 1, 3)
        w0 = torch.exp(g * (t + 1.0))[..., None]
        out["grad_state"] = torch.exp(g * L)[..., None] * dS + (Qf * w0).transpose(-1, -2).contiguous() @ Gf
    dk = dk.reshape(B, T, Hk, rep, Dk).sum(3)
    dv = dv.reshape(B, T, Hk, rep, Dv).sum(3)
    mm = m[..., None, None]
    out.update(grad_q=torch.where(mm, dq, 0.0).to(q.dtype),
               grad_k=torch.where(mm, dk, 0.0).to(q.dtype),
               grad_v=torch.where(mm, dv, 0.0).to(q.dtype))
    return out


def _step(s):
    rep = s["q"].shape[1] // s["k"].shape[1]
    k = s["k"].float().repeat_interleave(rep, 1)
    v = s["v"].float().repeat_interleave(rep, 1)
    live = s["slots"] >= 0
    at = s["slots"].clamp(min=0).long()
    S = torch.exp(s["log_decay"].float())[None, :, None, None] * s["state"][at]
    S = S + k[..., :, None] * v[..., None, :]
    o = s["scale"] * (s["q"].float()[..., None, :] @ S)[..., 0, :]
    s["state_out"][at[live]] = S[live]
    return {"out": torch.where(live[:, None, None], o, 0.0).to(s["q"].dtype),
            "state": s["state_out"]}


# ---------------------------------------------------------------- definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "step":
        return _exact_step(s)
    B, T = case["B"], case["T"]
    L = s["lengths"].tolist()
    if op.startswith("attention"):
        return _exact_attention(s, L)
    if op == "embed":
        y = torch.zeros(B, T, case["N"], dtype=torch.float64, device="cuda")
        for b in range(B):
            y[b, :L[b]] = s["table"].double().index_select(0, s["tokens"][b, :L[b]]) * s["scale"]
        return {"y": y}
    if op == "embed_grad":
        tok = torch.cat([s["tokens"][b, :L[b]] for b in range(B)]).long()
        g = torch.cat([s["grad_out"][b, :L[b]] for b in range(B)])
        order = torch.argsort(tok, stable=True)
        ends = torch.cumsum(torch.bincount(tok, minlength=case["V"]), 0)
        part = max(1, 100_000_000 // max(1, tok.numel()))
        cols = []
        for c in range(0, case["N"], part):
            run_sum = torch.cumsum(g[order, c:c + part].double(), 0)
            run_sum = torch.cat([torch.zeros_like(run_sum[:1]), run_sum])
            upto = run_sum[ends]
            cols.append(torch.diff(upto, dim=0, prepend=torch.zeros_like(upto[:1])))
        return {"grad_table": torch.cat(cols, 1) * s["scale"]}
    outs = {"y": []} if op == "norm" else {"grad_x": []}
    N = case["N"]
    w, bias = s["weight"].double(), s["bias"].double()
    dw, db = torch.zeros_like(w), torch.zeros_like(w)
    for b in range(B):
        x = s["x"][b, :L[b]].double()
        pad = torch.zeros(T - L[b], N, dtype=torch.float64, device="cuda")
        if op == "norm":
            var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
            outs["y"].append(torch.cat([(x - mean) / torch.sqrt(var + EPS) * w + bias, pad]))
            continue
        r = s["rstd"][b, :L[b], None].double()
        xh = (x - s["mean"][b, :L[b], None].double()) * r
        dy = s["grad_out"][b, :L[b]].double()
        dw += (dy * xh).sum(0)
        db += dy.sum(0)
        t = dy * w
        t = N * t - t.sum(-1, keepdim=True) - xh * (t * xh).sum(-1, keepdim=True)
        outs["grad_x"].append(torch.cat([r / N * t, pad]))
    outs = {k: torch.stack(v) for k, v in outs.items()}
    return outs if op == "norm" else {**outs, "grad_weight": dw, "grad_bias": db}


def _exact_step(s):
    c = s["case"]
    rep = c["Hq"] // c["Hk"]
    out = torch.zeros(c["B"], c["Hq"], c["Dv"], dtype=torch.float64, device="cuda")
    state = s["state"].double()
    live = [(b, p) for b, p in enumerate(s["slots"].tolist()) if p >= 0]
    if live:
        rows = torch.tensor([b for b, _ in live], device="cuda")
        pool = torch.tensor([p for _, p in live], device="cuda")
        head = torch.arange(c["Hq"], device="cuda") // rep
        k, v = s["k"].double()[rows][:, head], s["v"].double()[rows][:, head]
        gamma = torch.exp(s["log_decay"].double()).reshape(1, -1, 1, 1)
        new = state[pool] * gamma + k.unsqueeze(-1) * v.unsqueeze(-2)
        state[pool] = new
        out[rows] = (s["q"].double()[rows].unsqueeze(-1) * new).sum(-2) * s["scale"]
    return {"out": out, "state": state}


def _exact_attention(s, L):
    """Blocks of 256 positions in order (and in reverse for the gradients), each sequence by
    itself, every sum in float64."""
    c, step, scale = s["case"], 256, s["scale"]
    B, T, Hq, rep = c["B"], c["T"], c["Hq"], c["Hq"] // c["Hk"]
    head = torch.arange(Hq, device="cuda") // rep
    g = s["log_decay"].double()
    # sequences sorted into one loop: the block loop runs over all of them at once, with the
    # positions past a length given no weight
    pos = torch.arange(step, device="cuda", dtype=torch.float64)
    Lt = torch.tensor(L, device="cuda", dtype=torch.float64)
    zero = torch.zeros(B, Hq, c["Dk"], c["Dv"], dtype=torch.float64, device="cuda")
    grad = c["op"] == "attention_grad"

    def take(x, t0, t1, heads=None):
        x = x[:, t0:t1]
        x = x if heads is None else x[:, :, heads]
        keep = (torch.arange(t0, t1, device="cuda")[None] < Lt[:, None])[..., None, None]
        return torch.where(keep, x.double(), 0.0).transpose(1, 2)           # [B, Hq, n, D]

    def pairs(n):
        d = pos[:n, None] - pos[None, :n]
        return torch.where(d >= 0, torch.exp(g[:, None, None] * d.clamp(min=0)), 0.0)

    S = zero.clone() if s["state"] is None else s["state"].double()
    out = torch.zeros(B, T, Hq, c["Dv"], dtype=torch.float64, device="cuda")
    dq = torch.zeros(B, T, Hq, c["Dk"], dtype=torch.float64, device="cuda") if grad else None
    for t0 in range(0, T, step):
        t1 = min(T, t0 + step)
        n = t1 - t0
        k, v = take(s["k"], t0, t1, head), take(s["v"], t0, t1, head)
        D, w = pairs(n), torch.exp(g[:, None] * (pos[:n] + 1))[..., None]
        if grad:
            do = take(s["grad_out"], t0, t1)
            x = ((do @ v.mT) * D) @ k + (do * w) @ S.mT
            dq[:, t0:t1] = scale * x.transpose(1, 2)
        else:
            q = take(s["q"], t0, t1)
            x = ((q @ k.mT) * D) @ v + (q * w) @ S
            out[:, t0:t1] = scale * x.transpose(1, 2)
        # each sequence's own number of positions in this block
        m = (Lt - t0).clamp(0, n)
        e = m[:, None, None] - 1 - pos[None, None, :n]
        w = torch.where(e >= 0, torch.exp(g[None, :, None] * e.clamp(min=0)), 0.0)
        S = S * torch.exp(g[None, :] * m[:, None])[..., None, None] + (k * w[..., None]).mT @ v
    if not grad:
        return {"out": out, "state": S}
    R = zero.clone() if s["grad_state"] is None else s["grad_state"].double()
    dk = torch.zeros(B, T, c["Hk"], c["Dk"], dtype=torch.float64, device="cuda")
    dv = torch.zeros(B, T, c["Hk"], c["Dv"], dtype=torch.float64, device="cuda")
    for t0 in range((T - 1) // step * step, -1, -step):
        t1 = min(T, t0 + step)
        n = t1 - t0
        q, do = take(s["q"], t0, t1), take(s["grad_out"], t0, t1) * scale
        k, v = take(s["k"], t0, t1, head), take(s["v"], t0, t1, head)
        D = pairs(n)
        m = (Lt - t0).clamp(0, n)
        e = m[:, None, None] - 1 - pos[None, None, :n]
        w = torch.where(e >= 0, torch.exp(g[None, :, None] * e.clamp(min=0)), 0.0)[..., None]
        a = ((do @ v.mT) * D).mT @ q + (v * w) @ R.mT
        b = ((q @ k.mT) * D).mT @ do + (k * w) @ R
        dk[:, t0:t1] = a.transpose(1, 2).reshape(B, n, c["Hk"], rep, -1).sum(3)
        dv[:, t0:t1] = b.transpose(1, 2).reshape(B, n, c["Hk"], rep, -1).sum(3)
        w = torch.exp(g[:, None] * (pos[:n] + 1))[..., None]
        R = R * torch.exp(g[None, :] * m[:, None])[..., None, None] + (q * w).mT @ do
    res = {"grad_q": dq, "grad_k": dk, "grad_v": dv}
    if s["state"] is not None:
        res["grad_state"] = R
    return res


def work(case):
    """Bytes and operations a pass cannot do without, with the mean length of ragged cases."""
    op, e = case["op"], 4 if case["type"] == "f32" else 2
    B = case["B"]
    if op == "step":
        Hq, Hk, Dk, Dv = (case[k] for k in ("Hq", "Hk", "Dk", "Dv"))
        live = B if B <= 8 else B - -(-B // 7)
        io = e * B * (Hq * (Dk + Dv) + Hk * (Dk + Dv)) + 4 * B
        return {"bytes": io + live * Hq * Dk * Dv * 8, "flops": live * Hq * Dk * Dv * 5}
    T = case["T"]
    used = B * T * (0.75 if case["ragged"] else 1.0)     # rows that hold data
    if op.startswith("attention"):
        Hq, Hk, Dk, Dv = (case[k] for k in ("Hq", "Hk", "Dk", "Dv"))
        kv, st = Hk * (Dk + Dv), 4 * B * Hq * Dk * Dv
        if op == "attention":
            return {"bytes": e * (used * (Hq * Dk + kv) + B * T * Hq * Dv) + st * (2 if case["state"] else 1),
                    "flops": used * Hq * Dk * Dv * 4}
        return {"bytes": e * (used * (Hq * (Dk + Dv) + kv) + B * T * (Hq * Dk + kv)) + (3 * st if case["state"] else 0),
                "flops": used * Hq * Dk * Dv * 10}
    N = case["N"]
    if op == "embed":
        return {"bytes": 4 * used + e * N * (min(case["V"], used) + B * T), "flops": used * N}
    if op == "embed_grad":
        return {"bytes": 4 * used + e * N * (used + case["V"]), "flops": used * N}
    if op == "norm":
        return {"bytes": e * N * (used + B * T + 2), "flops": used * N * 8}
    return {"bytes": e * N * (2 * used + B * T + 3) + 8 * used, "flops": used * N * 14}
