"""The operators of an encoder block and of its pretraining, as they are timed: the cases, their
inputs, the operators' plain forms and their definitions in 64 bits.

A block mixes positions with a gated recurrence, adds what it made to the residual stream and
normalises it for the next block; before there are segments to train on, the encoder learns to
predict tokens over the vocabulary of its embedding.  Sizes are the library's own workloads (B, T
and lengths of the tiny, speech and genomic configurations) with generic widths.

Operators ("op" of a case; "train": the forward pass and all gradients):
  step        one token of the recurrence for every stream, on states in a pool
  recurrence  a = exp(log_decay sig(r)), h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sig(i_t) x_t
  residual    r = x + scale sig(gate) norm(branch), y = norm(r)
  nll         -log softmax(scale x W^T)[target] at the positions that have a target
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


def listed():
    return [
        # one token of one stream through one layer: a call whose latency counts
        {"name": "step_one", "op": "step", "B": 1, "pool": 1, "N": 1024, "type": "bf16"},
        # the speech workload, ragged, as it is tagged
        {"name": "recurrence_speech", "op": "recurrence", "train": False, "B": 32, "T": 800, "N": 1024, "type": "bf16", "ragged": True, "state": False},
        # a training step of the genomic workload: four sequences of 100,000 positions
        {"name": "recurrence_train_genomic", "op": "recurrence", "train": True, "B": 4, "T": 100000, "N": 512, "type": "bf16", "ragged": False, "state": False},
        # one long sequence in full precision, carried on from a state: the long axis has to be split
        {"name": "recurrence_train_long", "op": "recurrence", "train": True, "B": 1, "T": 250001, "N": 256, "type": "f32", "ragged": False, "state": True},
        # one token of 64 streams through the end of a block: a call whose latency counts
        {"name": "residual_stream", "op": "residual", "train": False, "B": 64, "T": 1, "N": 1024, "type": "bf16", "ragged": False, "gate": True, "post": True, "scale": True, "center": True},
        # an odd width in full precision, a plain residual with the root-mean-square norm
        {"name": "residual_odd", "op": "residual", "train": False, "B": 16, "T": 1000, "N": 777, "type": "f32", "ragged": True, "gate": False, "post": False, "scale": False, "center": False},
        # a training step of the speech workload with everything a block may have
        {"name": "residual_train_speech", "op": "residual", "train": True, "B": 32, "T": 800, "N": 1024, "type": "bf16", "ragged": True, "gate": True, "post": True, "scale": True, "center": True},
        # the genomic workload: sums for the weights over 400,000 rows
        {"name": "residual_train_genomic", "op": "residual", "train": True, "B": 4, "T": 100000, "N": 512, "type": "bf16", "ragged": False, "gate": True, "post": False, "scale": True, "center": False},
        # the tiny workload: a call whose latency counts
        {"name": "nll_tiny", "op": "nll", "train": True, "B": 2, "T": 64, "N": 65, "V": 300, "type": "f32", "ragged": False, "share": 1.0},
        # scores of ragged sentences over a word vocabulary
        {"name": "nll_speech", "op": "nll", "train": False, "B": 32, "T": 800, "N": 1024, "V": 50001, "type": "bf16", "ragged": True, "share": 1.0},
        # a pretraining step over a word vocabulary, every position predicted
        {"name": "nll_train_words", "op": "nll", "train": True, "B": 16, "T": 1000, "N": 1024, "V": 50001, "type": "bf16", "ragged": False, "share": 1.0},
        # a pretraining step on 6-mers of the genome, 15 of 100 positions masked and predicted
        {"name": "nll_train_kmers", "op": "nll", "train": True, "B": 4, "T": 25000, "N": 512, "V": 4096, "type": "bf16", "ragged": False, "share": 0.15},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "recurrence", "recurrence", "recurrence", "residual", "residual",
                     "nll", "nll", "nll"])
    case = {"op": op, "type": rng.choice(["f32", "bf16", "bf16"])}
    N = rng.choice([_log(rng, 8, 2048), rng.choice([64, 128, 256, 512, 768, 1024, 2048])])
    if op == "step":
        B = _log(rng, 1, 512)
        case.update(B=B, pool=B + rng.choice([0, 1, 64]), N=N)
        return case
    case.update(train=rng.random() < 0.6, ragged=rng.random() < 0.5)
    if op == "nll":
        V = _log(rng, 40, 100000)
        # at most a third of the largest listed case's products, an eighth in full precision
        room = 16000 * 1024 * 50001 // (3 if case["type"] == "bf16" else 8)
        n = min(_log(rng, 32, 100000), max(1, room // (N * V)), 400_000_000 // V)
        B = rng.choice([1, 2, 8, 32])
        case.update(B=B, T=max(1, n // B), N=N, V=V, share=rng.choice([1.0, 1.0, 0.15, 0.5]))
        return case
    # at most a quarter of the largest listed case's elements
    n = min(_log(rng, 16, 200000), 50_000_000 // N)
    B = rng.choice([1, 2, 4, 8, 32]) if op == "residual" else min(n, _log(rng, 1, 64))
    case.update(B=B, T=max(1, n // B), N=N)
    if op == "recurrence":
        case["state"] = rng.random() < 0.4
    else:
        case.update(gate=rng.random() < 0.5, post=rng.random() < 0.5, scale=rng.random() < 0.5,
                    center=rng.random() < 0.5)
    return case


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")
    typ = DTYPES[case["type"]]
    op, B, N = case["op"], case["B"], case["N"]

    def normal(*shape, sd=1.0, mean=0.0, dtype=typ):
        return (mean + sd * torch.randn(*shape, generator=gen, device=dev)).to(dtype)

    def leaf(x):
        return x.requires_grad_(case["train"])

    s = {"case": case}
    if op == "step":
        pool = case["pool"]
        s.update(x=normal(B, N), decay_gate=normal(B, N), input_gate=normal(B, N),
                 log_decay=_log_decay(N, dev), state=normal(pool, N, dtype=torch.float32))
        slots = torch.randperm(pool, generator=gen, device=dev)[:B].to(torch.int32)
        if B > 8:
            slots[::7] = -1          # idle rows of the batch
        s["slots"] = slots
        s["state_out"] = s["state"].clone()     # the rows that no slot names keep what they have
        return s
    T = case["T"]
    if case["ragged"]:
        lengths = torch.randint(T // 2, T + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
    else:
        lengths = torch.full((B,), T, device=dev, dtype=torch.int32)
    s["lengths"] = lengths
    if op == "recurrence":
        s.update(x=leaf(normal(B, T, N)), decay_gate=leaf(normal(B, T, N)),
                 input_gate=leaf(normal(B, T, N)), log_decay=leaf(_log_decay(N, dev)))
        s["state"] = leaf(normal(B, N, dtype=torch.float32)) if case["state"] else None
        if case["train"]:
            s["grad_out"] = normal(B, T, N)
            s["grad_state"] = normal(B, N, dtype=torch.float32) if case["state"] else None
        return s
    if op == "residual":
        s.update(x=leaf(normal(B, T, N, sd=2.0)), branch=leaf(normal(B, T, N, sd=1.5, mean=0.3)),
                 weight=leaf(normal(N, sd=0.1, mean=1.0)), bias=leaf(normal(N, sd=0.1)))
        s["gate"] = leaf(normal(B, T, N)) if case["gate"] else None
        s["scale"] = leaf(normal(N, sd=0.1, mean=0.5)) if case["scale"] else None
        s["branch_weight"] = leaf(normal(N, sd=0.1, mean=1.0)) if case["post"] else None
        s["branch_bias"] = leaf(normal(N, sd=0.1)) if case["post"] else None
        if case["train"]:
            s.update(grad_r=normal(B, T, N), grad_y=normal(B, T, N))
        return s
    V = case["V"]
    table = normal(V, N, sd=N ** -0.5)
    u = torch.rand(B, T, generator=gen, device=dev, dtype=torch.float64)
    t = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1)   # about 1 / rank
    t = torch.randperm(V, generator=gen, device=dev)[t]
    # some targets are foreseen almost surely, some not at all
    sure = 14.0 * torch.rand(B, T, 1, generator=gen, device=dev)
    s["x"] = leaf((normal(B, T, N, dtype=torch.float32) + sure * table[t].float()).to(typ))
    s["table"] = leaf(table)
    has = torch.rand(B, T, generator=gen, device=dev) < case["share"]
    s["targets"] = torch.where(has, t, -1).to(torch.int32)
    s["scale"] = 1.0
    if case["train"]:
        n = (has & _valid(s, T)).sum().clamp(min=1)
        s["grad_loss"] = (torch.ones(B, T, device=dev) / n).contiguous()
    return s


def _log_decay(N, dev):
    """Time constants from 2 to 2,048 positions where the gate is open, spread over the channels."""
    n = torch.arange(N, device=dev, dtype=torch.float32) / max(1, N - 1)
    return -torch.exp2(-1.0 - 10.0 * n)


def run(s):
    if own:
        return _run_own(s)
    with torch.no_grad():
        return {"step": _step, "recurrence": _recurrence, "residual": _residual,
                "nll": _nll}[s["case"]["op"]](s)


def _run_own(s):
    import semi_markov_crf_amd as crf
    c = s["case"]
    op = c["op"]
    if op == "step":
        out = crf.gated_recurrence_step(s["x"], s["decay_gate"], s["input_gate"], s["log_decay"],
                                        s["state"], slots=s["slots"], state_out=s["state_out"])
        return {"out": out, "state": s["state_out"]}
    if op == "recurrence":
        out, state = crf.gated_recurrence(s["x"], s["decay_gate"], s["input_gate"], s["log_decay"],
                                          lengths=s["lengths"], state=s["state"], want_state=True)
        res = {"out": out, "state": state}
        if c["train"]:
            names = ["x", "decay_gate", "input_gate", "log_decay"]
            outs, grads = [out], [s["grad_out"]]
            if c["state"]:
                names, outs, grads = names + ["state"], [out, state], [s["grad_out"], s["grad_state"]]
            d = torch.autograd.grad(outs, [s[n] for n in names], grads)
            res.update({"grad_" + n: g for n, g in zip(names, d)})
        return res
    if op == "residual":
        r, y = crf.residual_norm(s["x"], s["branch"], s["weight"], s["bias"], gate=s["gate"],
                                 scale=s["scale"], norm_branch=c["post"],
                                 branch_weight=s["branch_weight"], branch_bias=s["branch_bias"],
                                 center=c["center"], eps=EPS, lengths=s["lengths"])
        res = {"r": r, "y": y}
        if c["train"]:
            names = [n for n in ("x", "branch", "gate", "weight", "bias", "scale", "branch_weight",
                                 "branch_bias") if s[n] is not None]
            d = torch.autograd.grad([r, y], [s[n] for n in names], [s["grad_r"], s["grad_y"]])
            res.update({"grad_" + n: g for n, g in zip(names, d)})
        return res
    loss = crf.token_nll(s["x"], s["table"], s["targets"], scale=s["scale"], lengths=s["lengths"])
    res = {"loss": loss}
    if c["train"]:
        d = torch.autograd.grad(loss, [s["x"], s["table"]], s["grad_loss"])
        res.update(grad_x=d[0], grad_table=d[1])
    return res


# ---------------------------------------------------------------- plain forms (32 bits)

def _valid(s, T):
    """[B, T]: the positions before each sequence's length."""
    return torch.arange(T, device=s["lengths"].device)[None, :] < s["lengths"][:, None]


def _gates(s, x, decay_gate, input_gate):
    """sig(r), s, 1 - a^2 and sig(i) in 32 bits; expm1 keeps decays next to 1 apart from 1."""
    sr, si = torch.sigmoid(decay_gate.float()), torch.sigmoid(input_gate.float())
    ls = s["log_decay"] * sr
    return sr, ls, -torch.expm1(2.0 * ls), si


def _step(s):
    live = s["slots"] >= 0
    at = s["slots"].clamp(min=0).long()
    _, ls, bb, si = _gates(s, s["x"], s["decay_gate"], s["input_gate"])
    h = torch.exp(ls) * s["state"][at] + torch.sqrt(bb) * si * s["x"].float()
    s["state_out"][at[live]] = h[live]
    return {"out": torch.where(live[:, None], h, 0.0).to(s["x"].dtype), "state": s["state_out"]}


def _doubling(ls, v):
    """h_t = exp(ls_t) h_{t-1} + v_t along axis 1, and the running sum of ls: spans of 1, 2, 4, ...
    positions joined."""
    d = 1
    while d < v.shape[1]:
        v = torch.cat([v[:, :d], torch.exp(ls[:, d:]) * v[:, :-d] + v[:, d:]], 1)
        ls = torch.cat([ls[:, :d], ls[:, :-d] + ls[:, d:]], 1)
        d *= 2
    return v, ls


def _recurrence(s):
    x, typ = s["x"].float(), s["x"].dtype
    T = x.shape[1]
    m = _valid(s, T)[..., None]
    sr, ls, bb, si = _gates(s, x, s["decay_gate"], s["input_gate"])
    b = torch.sqrt(bb)
    ls = torch.where(m, ls, 0.0)                 # padding keeps the state
    h, upto = _doubling(ls, torch.where(m, b * si * x, 0.0))
    if s["state"] is not None:
        h = h + torch.exp(upto) * s["state"][:, None]
    res = {"out": torch.where(m, h, 0.0).to(typ), "state": h[:, -1]}
    if not s["case"]["train"]:
        return res
    g = torch.where(m, s["grad_out"].float(), 0.0)
    if s["state"] is not None:
        g[:, -1] += s["grad_state"]
    back = torch.cat([torch.zeros_like(ls[:, :1]), ls.flip(1)[:, :-1]], 1)
    e = _doubling(back, g.flip(1))[0].flip(1)
    del back, g, upto
    a = torch.exp(ls)
    first = torch.zeros_like(h[:, :1]) if s["state"] is None else s["state"][:, None]
    before = torch.cat([first, h[:, :-1]], 1)
    dls = torch.where(m, e * (a * before - a * a / b * (si * x)), 0.0)
    du = torch.where(m, e * b, 0.0)
    if s["state"] is not None:
        res["grad_state"] = a[:, 0] * e[:, 0]
    res.update(grad_x=(du * si).to(typ), grad_input_gate=(du * x * si * (1.0 - si)).to(typ),
               grad_decay_gate=(dls * s["log_decay"] * sr * (1.0 - sr)).to(typ),
               grad_log_decay=(dls * sr).sum((0, 1)))
    return res


def _normed(x, center):
    """The normalised rows and 1 / their size."""
    x = x - x.mean(-1, keepdim=True) if center else x
    rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * rstd, rstd


def _norm_back(g, h, rstd, center):
    """The gradient through _normed from that of its rows."""
    t = g - h * (g * h).mean(-1, keepdim=True)
    return rstd * (t - g.mean(-1, keepdim=True) if center else t)


def _residual(s):
    center, typ = s["case"]["center"], s["x"].dtype
    x, o = s["x"].float(), s["branch"].float()
    m = _valid(s, x.shape[1])[..., None]
    n = o
    if s["branch_weight"] is not None:
        oh, orstd = _normed(o, center)
        n = oh * s["branch_weight"].float() + s["branch_bias"].float()
    sg = 1.0 if s["gate"] is None else torch.sigmoid(s["gate"].float())
    sc = 1.0 if s["scale"] is None else s["scale"].float()
    r = x + sc * sg * n
    h, rstd = _normed(r, center)
    w = s["weight"].float()
    y = h * w + s["bias"].float()
    res = {"r": torch.where(m, r, 0.0).to(typ), "y": torch.where(m, y, 0.0).to(typ)}
    if not s["case"]["train"]:
        return res
    dy = torch.where(m, s["grad_y"].float(), 0.0)
    e = torch.where(m, s["grad_r"].float() + _norm_back(dy * w, h, rstd, center), 0.0)
    res.update(grad_x=e.to(typ), grad_weight=(dy * h).sum((0, 1)).to(typ),
               grad_bias=dy.sum((0, 1)).to(typ))
    if s["scale"] is not None:
        res["grad_scale"] = (e * sg * n).sum((0, 1)).to(typ)
    if s["gate"] is not None:
        res["grad_gate"] = (e * sc * n * sg * (1.0 - sg)).to(typ)
    dn = e * sc * sg
    if s["branch_weight"] is not None:
        res["grad_branch_weight"] = (dn * oh).sum((0, 1)).to(typ)
        res["grad_branch_bias"] = dn.sum((0, 1)).to(typ)
        dn = _norm_back(dn * s["branch_weight"].float(), oh, orstd, center)
    res["grad_branch"] = dn.to(typ)
    return res


def _nll(s):
    typ = s["x"].dtype
    B, T, N = s["x"].shape
    x, w = s["x"].float().reshape(-1, N), s["table"].float()
    t = s["targets"].long()
    has = (_valid(s, T) & (t >= 0)).reshape(-1)
    t = t.clamp(min=0).reshape(-1, 1)
    z = s["scale"] * (x @ w.t())
    top = z.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
    loss = torch.where(has, (lse - z.gather(1, t))[:, 0], 0.0)
    res = {"loss": loss.reshape(B, T)}
    if not s["case"]["train"]:
        return res
    p = torch.exp(z - lse)
    p.scatter_add_(1, t, torch.full_like(lse, -1.0))
    p = p * torch.where(has, s["scale"] * s["grad_loss"].reshape(-1), 0.0)[:, None]
    res.update(grad_x=(p @ w).reshape(B, T, N).to(typ), grad_table=(p.t() @ x).to(typ))
    return res


# ---------------------------------------------------------------- definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"step": _exact_step, "recurrence": _exact_recurrence, "residual": _exact_residual,
                "nll": _exact_nll}[case["op"]](s)


def _sig(x):
    return 1.0 / (1.0 + torch.exp(-x.double()))


def _exact_step(s):
    out = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    state = s["state"].double()
    live = [(b, p) for b, p in enumerate(s["slots"].tolist()) if p >= 0]
    if live:
        rows, at = (torch.tensor(v, device="cuda") for v in zip(*live))
        a = torch.exp(s["log_decay"].double() * _sig(s["decay_gate"][rows]))
        b = torch.sqrt((1.0 - a) * (1.0 + a))
        new = a * state[at] + b * _sig(s["input_gate"][rows]) * s["x"][rows].double()
        state[at] = new
        out[rows] = new
    return {"out": out, "state": state}


def _in_blocks(a, v, first):
    """h_t = a_t h_{t-1} + v_t from h = first, a position of every block at a time, then a block at
    a time; the last axis is any, axis 1 the positions."""
    B, T, N = v.shape
    S = max(1, int(math.sqrt(T)))
    pad = -T % S
    a = torch.nn.functional.pad(a, (0, 0, 0, pad), value=1.0).reshape(B, -1, S, N)
    v = torch.nn.functional.pad(v, (0, 0, 0, pad)).reshape(B, -1, S, N).clone()
    keep = torch.ones_like(a)
    keep[:, :, 0] = a[:, :, 0]
    for i in range(1, S):
        v[:, :, i] += a[:, :, i] * v[:, :, i - 1]
        keep[:, :, i] = keep[:, :, i - 1] * a[:, :, i]
    h = first
    for j in range(v.shape[1]):
        v[:, j] += keep[:, j] * h[:, None]
        h = v[:, j, -1]
    return v.reshape(B, -1, N)[:, :T]


def _exact_recurrence(s):
    x, lam = s["x"].double(), s["log_decay"].double()
    B, T, N = x.shape
    pos = torch.arange(T, device="cuda")
    live = (pos[None] < s["lengths"][:, None])[..., None]
    R, I = _sig(s["decay_gate"]), _sig(s["input_gate"])
    A = torch.where(live, torch.exp(lam * R), 1.0)
    root = torch.sqrt((1.0 - torch.exp(lam * R)) * (1.0 + torch.exp(lam * R)))
    U = torch.where(live, I * x, 0.0)
    zero = torch.zeros(B, N, dtype=torch.float64, device="cuda")
    h0 = zero if s["state"] is None else s["state"].double()
    H = _in_blocks(A, root * U, h0)
    res = {"out": H * live, "state": H[:, -1].clone()}
    if not s["case"]["train"]:
        return res
    G = s["grad_out"].double() * live
    # later positions' share of the gradient of h_t, seen from the end
    last = zero if s["state"] is None else s["grad_state"].double()
    mirrored = _in_blocks(A.flip(1), (G.flip(1) * A.flip(1)), last)     # a_t E_t
    after = torch.cat([mirrored.flip(1)[:, 1:], last[:, None]], 1)      # a_{t+1} E_{t+1}
    if s["state"] is not None:
        res["grad_state"] = mirrored[:, -1].clone()
    del mirrored
    E = (G + after) * live
    del after, G
    prev = torch.cat([h0[:, None], H[:, :-1]], 1)
    del H
    res["grad_x"] = E * root * I
    res["grad_input_gate"] = E * root * U * (1.0 - I)
    # d a = E h, d b = E u with b = sqrt(1 - a^2): db/da = -a / b
    dA = E * (prev - A / root * U)
    dlam = dA * A
    res["grad_log_decay"] = (dlam * R).sum((0, 1))
    res["grad_decay_gate"] = dlam * lam * R * (1.0 - R)
    return res


def _exact_residual(s):
    """A sequence at a time."""
    c = s["case"]
    T, L = c["T"], s["lengths"].tolist()
    par = {n: None if s[n] is None else s[n].double() for n in ("weight", "bias", "scale",
                                                                "branch_weight", "branch_bias")}
    rows, sums = {}, {}

    def put(name, x):
        pad = torch.zeros(T - x.shape[0], c["N"], dtype=torch.float64, device="cuda")
        rows.setdefault(name, []).append(torch.cat([x, pad]))

    def add(name, x):
        sums[name] = sums.get(name, 0.0) + x.sum(0)

    def stats(x):
        mean = x.mean(-1, keepdim=True) if c["center"] else torch.zeros_like(x[:, :1])
        return mean, 1.0 / torch.sqrt((x - mean).pow(2).mean(-1, keepdim=True) + EPS)

    def back(d, h, q):
        """d loss / d row of h = (row - mean) q, written out over the row's Jacobian."""
        N = c["N"]
        t = N * d - h * (d * h).sum(-1, keepdim=True)
        return q / N * (t - d.sum(-1, keepdim=True) if c["center"] else t)

    for b, n in enumerate(L):
        x, o = s["x"][b, :n].double(), s["branch"][b, :n].double()
        f = o
        if c["post"]:
            mu, q = stats(o)
            hat = (o - mu) * q
            f = par["branch_weight"] * hat + par["branch_bias"]
        k = torch.ones_like(o) if s["gate"] is None else _sig(s["gate"][b, :n])
        z = k if par["scale"] is None else k * par["scale"]
        r = x + z * f
        mean, rs = stats(r)
        h = (r - mean) * rs
        put("r", r)
        put("y", h * par["weight"] + par["bias"])
        if not c["train"]:
            continue
        dy = s["grad_y"][b, :n].double()
        e = s["grad_r"][b, :n].double() + back(dy * par["weight"], h, rs)
        put("grad_x", e)
        add("grad_weight", dy * h)
        add("grad_bias", dy)
        if c["scale"]:
            add("grad_scale", e * k * f)
        if c["gate"]:
            put("grad_gate", e * f * z * (1.0 - k))
        d = e * z
        if c["post"]:
            add("grad_branch_weight", d * hat)
            add("grad_branch_bias", d)
            d = back(d * par["branch_weight"], hat, q)
        put("grad_branch", d)
    return {**{k: torch.stack(v) for k, v in rows.items()}, **sums}


def _exact_nll(s):
    """The positions that have a target, a few thousand words of the vocabulary at a time."""
    c = s["case"]
    B, T, N, V = c["B"], c["T"], c["N"], c["V"]
    live = torch.arange(T, device="cuda")[None] < s["lengths"][:, None]
    at = torch.nonzero((live & (s["targets"] >= 0)).reshape(-1))[:, 0]
    t = s["targets"].reshape(-1)[at].long()
    x = s["x"].reshape(-1, N)[at].double()
    W = s["table"].double()
    lse = torch.full((len(at),), -math.inf, dtype=torch.float64, device="cuda")
    step = max(1, 200_000_000 // max(1, len(at)))
    for v in range(0, V, step):
        lse = torch.logaddexp(lse, torch.logsumexp(s["scale"] * (x @ W[v:v + step].mT), 1))
    loss = torch.zeros(B * T, dtype=torch.float64, device="cuda")
    loss[at] = lse - s["scale"] * (x * W[t]).sum(1)
    res = {"loss": loss.reshape(B, T)}
    if not c["train"]:
        return res
    k = s["scale"] * s["grad_loss"].reshape(-1)[at].double()
    dx, dW = torch.zeros_like(x), torch.zeros_like(W)
    for v in range(0, V, step):
        p = torch.exp(s["scale"] * (x @ W[v:v + step].mT) - lse[:, None])
        hit = torch.nonzero((t >= v) & (t < v + step))[:, 0]
        p[hit, t[hit] - v] -= 1.0
        p *= k[:, None]
        dx += p @ W[v:v + step]
        dW[v:v + step] = p.mT @ x
    grad = torch.zeros(B * T, N, dtype=torch.float64, device="cuda")
    grad[at] = dx
    res.update(grad_x=grad.reshape(B, T, N), grad_table=dW)
    return res


# ---------------------------------------------------------------- work

def work(case):
    """Bytes and operations a pass cannot do without, with the mean length of ragged cases."""
    op, B, N, e = case["op"], case["B"], case["N"], 4 if case["type"] == "f32" else 2
    if op == "step":
        live = B if B <= 8 else B - -(-B // 7)
        return {"bytes": 4 * e * B * N + 8 * live * N + 4 * N + 4 * B, "flops": 12 * live * N}
    T, train = case["T"], case["train"]
    used = B * T * (0.75 if case["ragged"] else 1.0)     # rows that hold data
    if op == "recurrence":
        state = 4 * B * N * (2 if case["state"] else 1)
        if not train:
            return {"bytes": e * N * (3 * used + B * T) + state + 4 * N, "flops": 12 * used * N}
        return {"bytes": e * N * (7 * used + 4 * B * T) + state + (8 * B * N if case["state"] else 0) + 12 * N,
                "flops": 40 * used * N}
    if op == "residual":
        n = 2 + case["gate"]                             # arrays read, and their gradients
        w = N * e * (2 + case["scale"] + 2 * case["post"])
        flops = 8 + 4 * case["gate"] + case["scale"] + 6 * case["post"]
        if not train:
            return {"bytes": e * N * (n * used + 2 * B * T) + w, "flops": flops * used * N}
        return {"bytes": e * N * (2 * (n + 1) * used + (n + 2) * B * T) + 3 * w, "flops": 3 * flops * used * N}
    used *= case["share"]
    V = case["V"]
    if not train:
        return {"bytes": e * N * (used + V) + 8 * B * T, "flops": 2 * used * N * V}
    return {"bytes": e * N * (2 * used + B * T + 3 * V) + 16 * B * T, "flops": 6 * used * N * V}
