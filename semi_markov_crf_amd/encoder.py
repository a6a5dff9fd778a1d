"""What makes the emissions: embedding, layer norm and decayed linear attention.

Like the calls of the CRF itself these functions only check and marshal arguments; the work
runs in the library's HIP kernels, on torch's current stream.

    embed(tokens, table)                       -> scale * table[tokens]  [B, T, N]
    layer_norm(x, weight, bias)                -> y  [B, T, N]
    decay_attention(q, k, v, log_decay)        -> o  [B, T, Hq, Dv] (and the final state)
    decay_attention_step(q, k, v, ..., state)  -> o  [B, Hq, Dv], one token a stream

embed, layer_norm and decay_attention are differentiable; embed_grad, layer_norm_grad and
decay_attention_grad are the gradients by themselves.  Tensors are float32 or bfloat16 on one
GPU.  lengths [B] int32 (0 <= lengths[b] <= T, None = T everywhere): what lies at t >= lengths[b]
is not read and outputs are 0 there.  check_status=True waits for the call and raises when a
length or a token was out of range.
"""

from __future__ import annotations

import ctypes

import torch

from . import _native

__all__ = ["embed", "embed_grad", "layer_norm", "layer_norm_grad", "decay_attention",
           "decay_attention_grad", "decay_attention_step"]

_TYPES = {torch.float32: _native.F32, torch.bfloat16: _native.BF16}


def _stream(device):
    return torch.cuda.current_stream(device).cuda_stream


def _ptr(x):
    return None if x is None else x.data_ptr()


def _need(name, x, dtype=None, shape=None, device=None, dense=True):
    if not isinstance(x, torch.Tensor) or x.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and x.device != device:
        raise ValueError(f"{name} is on {x.device}, expected {device}")
    if dtype is None:
        if x.dtype not in _TYPES:
            raise TypeError(f"{name} must be float32 or bfloat16, got {x.dtype}")
    elif x.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {x.dtype}")
    if shape is not None and tuple(x.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(x.shape)}")
    if dense and not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _lengths(lengths, B, device):
    if lengths is not None:
        _need("lengths", lengths, torch.int32, (B,), device)


def _workspace(fn, n, device, workspace):
    if n == 0:
        raise _native.SemiCRFError(fn, 3)
    if workspace is None:
        workspace = torch.empty(n, dtype=torch.uint8, device=device)
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {device}")
    if workspace.numel() * workspace.element_size() < n or workspace.data_ptr() % 256:
        raise ValueError(f"workspace must hold {n} bytes, 256-byte aligned")
    return workspace


class _Status:
    """The status word of one call, present only where it is asked for."""

    def __init__(self, fn, want, device):
        self.fn = fn
        self.word = torch.zeros(1, dtype=torch.int32, device=device) if want else None

    def check(self, rc):
        _native.check(self.fn, rc)
        if self.word is not None and int(self.word.item()):
            raise _native.SemiCRFError(self.fn, 1)


def _tracked(*tensors):
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


# ---------------------------------------------------------------- embedding

def _tokens(tokens, device):
    if not isinstance(tokens, torch.Tensor) or tokens.device != device:
        raise ValueError(f"tokens must be on {device}")
    if tokens.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"tokens must be int32 or int64, got {tokens.dtype}")
    if tokens.dim() != 2 or not tokens.is_contiguous():
        raise ValueError("tokens must be contiguous [B, T]")
    return int(tokens.shape[0]), int(tokens.shape[1]), tokens.element_size() * 8


def embed(tokens, table, *, scale=1.0, lengths=None, check_status=False) -> torch.Tensor:
    """scale * table[tokens]: tokens [B, T] int32 or int64, table [V, N], out [B, T, N].  A
    token outside [0, V) gives a row of NaN."""
    if _tracked(table):
        return _Embed.apply(tokens, table, float(scale), lengths, check_status)
    _need("table", table)
    if table.dim() != 2:
        raise ValueError("table must be [V, N]")
    B, T, bits = _tokens(tokens, table.device)
    _lengths(lengths, B, table.device)
    V, N = table.shape
    out = torch.empty((B, T, N), dtype=table.dtype, device=table.device)
    st = _Status("semicrf_embed", check_status, table.device)
    st.check(_native.load().semicrf_embed(
        tokens.data_ptr(), bits, _ptr(lengths), table.data_ptr(), _TYPES[table.dtype], B, T, V, N,
        scale, _stream(table.device), out.data_ptr(), _ptr(st.word)))
    return out


def embed_grad(tokens, grad_out, V, *, scale=1.0, lengths=None, workspace=None,
               check_status=False) -> torch.Tensor:
    """Gradient [V, N] of the table: row v is scale times the sum of grad_out [B, T, N] over
    the positions that hold token v, in the order of the positions."""
    _need("grad_out", grad_out)
    dev = grad_out.device
    B, T, bits = _tokens(tokens, dev)
    _lengths(lengths, B, dev)
    if grad_out.dim() != 3 or grad_out.shape[:2] != tokens.shape:
        raise ValueError(f"grad_out must be [{B}, {T}, N], got {list(grad_out.shape)}")
    N, V, lib, typ = int(grad_out.shape[2]), int(V), _native.load(), _TYPES[grad_out.dtype]
    n = lib.semicrf_embed_grad_bytes(typ, B, T, V, N)
    ws = _workspace("semicrf_embed_grad", n, dev, workspace)
    out = torch.empty((V, N), dtype=grad_out.dtype, device=dev)
    st = _Status("semicrf_embed_grad", check_status, dev)
    st.check(lib.semicrf_embed_grad(
        tokens.data_ptr(), bits, _ptr(lengths), grad_out.data_ptr(), typ, B, T, V, N, scale,
        _stream(dev), ws.data_ptr(), n, out.data_ptr(), _ptr(st.word)))
    return out


class _Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, table, scale, lengths, check_status):
        ctx.save_for_backward(tokens, lengths)
        ctx.scale, ctx.V = scale, table.shape[0]
        return embed(tokens, table.detach(), scale=scale, lengths=lengths,
                     check_status=check_status)

    @staticmethod
    def backward(ctx, g):
        tokens, lengths = ctx.saved_tensors
        return (None, embed_grad(tokens, g.contiguous(), ctx.V, scale=ctx.scale, lengths=lengths),
                None, None, None)


# ---------------------------------------------------------------- layer norm

def _norm_shape(x, weight, bias):
    _need("x", x)
    if x.dim() != 3:
        raise ValueError("x must be [B, T, N]")
    B, T, N = (int(n) for n in x.shape)
    wtype = x.dtype if weight is None else weight.dtype
    if wtype not in (x.dtype, torch.float32):
        raise TypeError(f"weight must be {x.dtype} or float32, got {wtype}")
    if weight is not None:
        _need("weight", weight, wtype, (N,), x.device)
    if bias is not None:
        wtype = wtype if weight is not None else bias.dtype
        if wtype not in (x.dtype, torch.float32):
            raise TypeError(f"bias must be {x.dtype} or float32, got {wtype}")
        _need("bias", bias, wtype, (N,), x.device)
    return B, T, N, wtype


def layer_norm(x, weight=None, bias=None, *, eps=1e-5, lengths=None, want_stats=False,
               check_status=False):
    """Layer norm over the last axis of x [B, T, N].  weight, bias [N] in x's type or float32
    (None: ones, zeros).  With want_stats, (y, mean [B, T], rstd [B, T]), which
    layer_norm_grad takes; those two carry no gradient."""
    if _tracked(x, weight, bias):
        y, mean, rstd = _LayerNorm.apply(x, weight, bias, float(eps), lengths, check_status)
        return (y, mean, rstd) if want_stats else y
    B, T, N, wtype = _norm_shape(x, weight, bias)
    _lengths(lengths, B, x.device)
    y = torch.empty_like(x)
    mean = torch.empty((B, T), dtype=torch.float32, device=x.device) if want_stats else None
    rstd = torch.empty_like(mean) if want_stats else None
    st = _Status("semicrf_layer_norm", check_status, x.device)
    st.check(_native.load().semicrf_layer_norm(
        x.data_ptr(), _TYPES[x.dtype], _ptr(weight), _ptr(bias), _TYPES[wtype], _ptr(lengths), B, T,
        N, eps, _stream(x.device), y.data_ptr(), _ptr(mean), _ptr(rstd), _ptr(st.word)))
    return (y, mean, rstd) if want_stats else y


def layer_norm_grad(grad_out, x, weight, mean, rstd, *, lengths=None, want_params=True,
                    workspace=None, check_status=False) -> dict:
    """Gradients of layer_norm from the mean and rstd it left: a dict with grad_x [B, T, N] and,
    unless want_params is False, grad_weight and grad_bias [N] in the weight's type (x's where
    weight is None)."""
    B, T, N, wtype = _norm_shape(x, weight, None)
    return _norm_grad(grad_out, x, weight, wtype, mean, rstd, lengths, want_params, workspace,
                      check_status, B, T, N)


def _norm_grad(grad_out, x, weight, wtype, mean, rstd, lengths, want_params, workspace,
               check_status, B, T, N):
    dev = x.device
    _need("grad_out", grad_out, x.dtype, x.shape, dev)
    _need("mean", mean, torch.float32, (B, T), dev)
    _need("rstd", rstd, torch.float32, (B, T), dev)
    _lengths(lengths, B, dev)
    lib = _native.load()
    n = lib.semicrf_layer_norm_grad_bytes(_TYPES[x.dtype], B, T, N)
    ws = _workspace("semicrf_layer_norm_grad", n, dev, workspace)
    gx = torch.empty_like(x)
    gw = torch.empty(N, dtype=wtype, device=dev) if want_params else None
    gb = torch.empty(N, dtype=wtype, device=dev) if want_params else None
    st = _Status("semicrf_layer_norm_grad", check_status, dev)
    st.check(lib.semicrf_layer_norm_grad(
        grad_out.data_ptr(), x.data_ptr(), _TYPES[x.dtype], _ptr(weight), _TYPES[wtype],
        mean.data_ptr(), rstd.data_ptr(), _ptr(lengths), B, T, N, _stream(dev), ws.data_ptr(), n,
        gx.data_ptr(), _ptr(gw), _ptr(gb), _ptr(st.word)))
    out = {"grad_x": gx}
    if want_params:
        out.update(grad_weight=gw, grad_bias=gb)
    return out


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, lengths, check_status):
        ctx.wtype = _norm_shape(x, weight, bias)[3]
        y, mean, rstd = layer_norm(x, weight, bias, eps=eps, lengths=lengths, want_stats=True,
                                   check_status=check_status)
        ctx.save_for_backward(x, weight, mean, rstd, lengths)
        ctx.mark_non_differentiable(mean, rstd)
        return y, mean, rstd

    @staticmethod
    def backward(ctx, g, _mean, _rstd):
        x, weight, mean, rstd, lengths = ctx.saved_tensors
        need_w, need_b = ctx.needs_input_grad[1:3]
        B, T, N = x.shape
        d = _norm_grad(g.contiguous(), x, weight, ctx.wtype, mean, rstd, lengths,
                       need_w or need_b, None, False, B, T, N)
        return (d["grad_x"], d.get("grad_weight") if need_w else None,
                d.get("grad_bias") if need_b else None, None, None, None)


# ---------------------------------------------------------------- attention

def _attention(q, k, v, log_decay, scale, lengths, state, state_shape, T):
    """The checked argument struct; q, k, v [B, T, H, D] (or [B, H, D] for one token)."""
    dims = 3 if T is None else 4
    for name, x in (("q", q), ("k", k), ("v", v)):
        _need(name, x, None if name == "q" else q.dtype, device=q.device, dense=False)
        if x.dim() != dims:
            raise ValueError(f"{name} must have {dims} dimensions, got {list(x.shape)}")
        if x.shape[-1] != 1 and x.stride(-1) != 1:
            raise ValueError(f"the last axis of {name} must be dense")
    B, (Hq, Dk), (Hk, Dv) = q.shape[0], q.shape[-2:], v.shape[-2:]
    if k.shape[:-1] != v.shape[:-1] or k.shape[-1] != Dk or q.shape[:-2] != k.shape[:-2] or \
            Hk < 1 or Hq % Hk:
        raise ValueError(f"shape mismatch: q {list(q.shape)}, k {list(k.shape)}, v "
                         f"{list(v.shape)}; query heads must be a multiple of key heads")
    _need("log_decay", log_decay, torch.float32, (Hq,), q.device)
    _lengths(lengths, B, q.device)
    if state is not None:
        _need("state", state, torch.float32, state_shape or (B, Hq, Dk, Dv), q.device)
    a = _native.Attention()
    a.q, a.k, a.v = q.data_ptr(), k.data_ptr(), v.data_ptr()
    for s, x in ((a.q_stride, q), (a.k_stride, k), (a.v_stride, v)):
        s[0], s[1], s[2] = x.stride(0), x.stride(1) if dims == 4 else 0, x.stride(-2)
    a.lengths, a.log_decay, a.state = _ptr(lengths), log_decay.data_ptr(), _ptr(state)
    a.scale = float(Dk) ** -0.5 if scale is None else float(scale)
    a.dtype = _TYPES[q.dtype]
    a.B, a.T, a.Hq, a.Hk, a.Dk, a.Dv = B, 1 if T is None else q.shape[1], Hq, Hk, Dk, Dv
    return a


def decay_attention(q, k, v, log_decay, *, scale=None, lengths=None, state=None,
                    want_state=False, workspace=None, check_status=False):
    """S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T and o_t = scale q_t^T S_t for every position:
    q [B, T, Hq, Dk], k [B, T, Hk, Dk], v [B, T, Hk, Dv] (views with a dense last axis), Hq a
    multiple of Hk, Dk and Dv up to 128; log_decay [Hq] float32, a constant; scale Dk**-0.5 by
    default; state [B, Hq, Dk, Dv] float32 before the first position (None: 0).  Returns o
    [B, T, Hq, Dv], and with want_state also the state after each sequence's last position."""
    if log_decay.requires_grad and torch.is_grad_enabled():
        raise ValueError("log_decay is a constant of the head: it has no gradient")
    if _tracked(q, k, v, state):
        o, end = _DecayAttention.apply(q, k, v, log_decay, scale, lengths, state, want_state,
                                       check_status)
        return (o, end) if want_state else o
    a = _attention(q, k, v, log_decay, scale, lengths, state, None, 0)
    dev, lib = q.device, _native.load()
    n = lib.semicrf_decay_attention_bytes(a, 0)
    ws = _workspace("semicrf_decay_attention", n, dev, workspace)
    out = torch.empty((a.B, a.T, a.Hq, a.Dv), dtype=q.dtype, device=dev)
    end = torch.empty((a.B, a.Hq, a.Dk, a.Dv), dtype=torch.float32, device=dev) if want_state else None
    st = _Status("semicrf_decay_attention", check_status, dev)
    st.check(lib.semicrf_decay_attention(a, _stream(dev), ws.data_ptr(), n, out.data_ptr(),
                                         _ptr(end), _ptr(st.word)))
    return (out, end) if want_state else out


def decay_attention_grad(grad_out, q, k, v, log_decay, *, scale=None, lengths=None, state=None,
                         grad_state=None, workspace=None, check_status=False) -> dict:
    """Gradients of decay_attention from those of its output, grad_out [B, T, Hq, Dv], and of its
    final state, grad_state [B, Hq, Dk, Dv] (None: 0): a dict with grad_q, grad_k, grad_v and,
    where an initial state is given, grad_state."""
    a = _attention(q, k, v, log_decay, scale, lengths, state, None, 0)
    dev, lib = q.device, _native.load()
    _need("grad_out", grad_out, q.dtype, (a.B, a.T, a.Hq, a.Dv), dev)
    if grad_state is not None:
        _need("grad_state", grad_state, torch.float32, (a.B, a.Hq, a.Dk, a.Dv), dev)
    n = lib.semicrf_decay_attention_bytes(a, 1)
    ws = _workspace("semicrf_decay_attention_grad", n, dev, workspace)
    gq, gk, gv = (torch.empty(x.shape, dtype=x.dtype, device=dev) for x in (q, k, v))
    gs = torch.empty_like(state) if state is not None else None
    st = _Status("semicrf_decay_attention_grad", check_status, dev)
    st.check(lib.semicrf_decay_attention_grad(
        a, grad_out.data_ptr(), _ptr(grad_state), _stream(dev), ws.data_ptr(), n, gq.data_ptr(),
        gk.data_ptr(), gv.data_ptr(), _ptr(gs), _ptr(st.word)))
    out = {"grad_q": gq, "grad_k": gk, "grad_v": gv}
    if gs is not None:
        out["grad_state"] = gs
    return out


class _DecayAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_decay, scale, lengths, state, want_state, check_status):
        ctx.save_for_backward(q, k, v, log_decay, lengths, state)
        ctx.scale = scale
        out = decay_attention(q, k, v, log_decay, scale=scale, lengths=lengths, state=state,
                              want_state=want_state, check_status=check_status)
        return out if want_state else (out, None)

    @staticmethod
    def backward(ctx, g, g_state):
        q, k, v, log_decay, lengths, state = ctx.saved_tensors
        d = decay_attention_grad(g.contiguous(), q, k, v, log_decay, scale=ctx.scale,
                                 lengths=lengths, state=state,
                                 grad_state=None if g_state is None else g_state.contiguous())
        return (d["grad_q"], d["grad_k"], d["grad_v"], None, None, None, d.get("grad_state"), None,
                None)


def decay_attention_step(q, k, v, log_decay, state, *, scale=None, slots=None,
                         state_out=None) -> torch.Tensor:
    """One token of B streams: q [B, Hq, Dk], k [B, Hk, Dk], v [B, Hk, Dv] and a pool of states
    [pool, Hq, Dk, Dv] float32, updated in place (or written to state_out, whose other rows are
    left alone).  Stream b uses row slots[b] (int32; None: row b).  A slot outside [0, pool) is
    idle: its output is 0.  Slots in use must be distinct.  Returns o [B, Hq, Dv]; carries no
    gradient."""
    if state.dim() != 4:
        raise ValueError("state must be [pool, Hq, Dk, Dv]")
    pool = state.shape[0]
    a = _attention(q, k, v, log_decay, scale, None, state,
                   (pool, q.shape[-2], q.shape[-1], v.shape[-1]), None)
    if slots is None:
        if pool < a.B:
            raise ValueError(f"a pool of {pool} states for {a.B} streams needs slots")
    else:
        _need("slots", slots, torch.int32, (a.B,), q.device)
    if state_out is None:
        state_out = state
    else:
        _need("state_out", state_out, torch.float32, state.shape, q.device)
    out = torch.empty((a.B, a.Hq, a.Dv), dtype=q.dtype, device=q.device)
    _native.check("semicrf_decay_attention_step", _native.load().semicrf_decay_attention_step(
        a, _ptr(slots), pool, _stream(q.device), out.data_ptr(), state_out.data_ptr()))
    return out
