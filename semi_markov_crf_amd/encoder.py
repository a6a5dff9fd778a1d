"""What makes the emissions: embedding, layer norm and decayed linear attention.

Like the calls of the CRF itself these functions only check and marshal arguments; the work
runs in the library's HIP kernels, on torch's current stream.

    embed(tokens, table)                       -> scale * table[tokens]  [B, T, N]
    layer_norm(x, weight, bias)                -> y  [B, T, N]
    decay_attention(q, k, v, log_decay)        -> o  [B, T, Hq, Dv] (and the final state)
    decay_attention_step(q, k, v, ..., state)  -> o  [B, Hq, Dv], one token a stream

embed, layer_norm and decay_attention are differentiable, once and backward: a derivative of their
gradients and a forward-mode tangent raise.  embed_grad, layer_norm_grad and decay_attention_grad are the
gradients by themselves; they and decay_attention_step carry none.  Tensors are float32 or bfloat16 on one
GPU.  lengths [B] int32 (0 <= lengths[b] <= T, None = T everywhere): what lies at t >= lengths[b]
is not read and outputs are 0 there.  check_status=True waits for the call and raises when a
length or a token was out of range.
"""

from __future__ import annotations

import torch
from torch.autograd import forward_ad
from torch.autograd.graph import increment_version

from . import _native
from ._autograd import first_order

__all__ = ["embed", "embed_grad", "layer_norm", "layer_norm_grad", "decay_attention",
           "decay_attention_grad", "decay_attention_step"]

_TYPES = {torch.float32: _native.F32, torch.bfloat16: _native.BF16}


# the current stream of a device, as an address; single-token calls are host-bound, and the public
# way builds a Stream object for it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _ptr(x):
    return None if x is None else x.data_ptr()


def _index(name, x):
    """Device index of the tensor that says where a call runs."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if x.dtype not in _TYPES:
        raise TypeError(f"{name} must be float32 or bfloat16, got {x.dtype}")
    return x.get_device()


def _need(name, x, dtype, shape, dev):
    """Refuses what is not a dense tensor of this type and shape on GPU `dev`."""
    try:
        if x.dtype is dtype and x.shape == shape and x.get_device() == dev and x.is_contiguous():
            return
    except AttributeError:
        pass
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if x.get_device() != dev:
        raise ValueError(f"{name} is on {x.device}, expected cuda:{dev}")
    if x.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {x.dtype}")
    if tuple(x.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(x.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _lengths(lengths, B, dev):
    if lengths is not None:
        _need("lengths", lengths, torch.int32, (B,), dev)


def _workspace(fn, n, device, workspace):
    if n == 0:
        raise _native.SemiCRFError(fn, 3)
    if workspace is None:
        return torch.empty(n, dtype=torch.uint8, device=device)
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {device}")
    if workspace.numel() * workspace.element_size() < n or workspace.data_ptr() % 256:
        raise ValueError(f"workspace must hold {n} bytes, 256-byte aligned")
    return workspace


def _status(want, device):
    """The status word of a call, where it is asked for."""
    return torch.zeros(1, dtype=torch.int32, device=device) if want else None


def _run(fn, dev, word, *args):
    """A call of the library on GPU `dev`, whose status word (or None) is `word`."""
    rc = _native.call(dev, fn, *args)
    if rc:
        raise _native.SemiCRFError(fn, rc)
    if word is not None and int(word.item()):
        raise _native.SemiCRFError(fn, 1)


def _tracked(*tensors):
    """Whether a call goes through its autograd function: one of its inputs wants a gradient, or
    carries a forward-mode tangent, which the function refuses."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    return getattr(forward_ad, "_current_level", 0) >= 0 and any(
        t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors)


# ---------------------------------------------------------------- embedding

def _tokens(tokens, dev):
    if not isinstance(tokens, torch.Tensor) or tokens.get_device() != dev:
        raise ValueError(f"tokens must be on cuda:{dev}")
    if tokens.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"tokens must be int32 or int64, got {tokens.dtype}")
    if tokens.dim() != 2 or not tokens.is_contiguous():
        raise ValueError("tokens must be contiguous [B, T]")
    B, T = tokens.shape
    return B, T, tokens.element_size() * 8


def embed(tokens, table, *, scale=1.0, lengths=None, check_status=False) -> torch.Tensor:
    """scale * table[tokens]: tokens [B, T] int32 or int64, table [V, N], out [B, T, N].  A
    token outside [0, V) gives a row of NaN."""
    dev = _index("table", table)
    if _tracked(table):
        return _Embed.apply(tokens, table, float(scale), lengths, check_status)
    if table.dim() != 2 or not table.is_contiguous():
        raise ValueError("table must be contiguous [V, N]")
    B, T, bits = _tokens(tokens, dev)
    _lengths(lengths, B, dev)
    V, N = table.shape
    out = table.new_empty((B, T, N))
    word = _status(check_status, table.device)
    _run("semicrf_embed", dev, word, tokens.data_ptr(), bits, _ptr(lengths), table.data_ptr(),
         _TYPES[table.dtype], B, T, V, N, scale, _raw_stream(dev), out.data_ptr(), _ptr(word))
    return out


def embed_grad(tokens, grad_out, V, *, scale=1.0, lengths=None, workspace=None,
               check_status=False) -> torch.Tensor:
    """Gradient [V, N] of the table: row v is scale times the sum of grad_out [B, T, N] over
    the positions that hold token v, in the order of the positions."""
    dev = _index("grad_out", grad_out)
    B, T, bits = _tokens(tokens, dev)
    _lengths(lengths, B, dev)
    if grad_out.dim() != 3 or grad_out.shape[:2] != tokens.shape or not grad_out.is_contiguous():
        raise ValueError(f"grad_out must be contiguous [{B}, {T}, N], got {list(grad_out.shape)}")
    N, V, lib, typ = grad_out.shape[2], int(V), _native.load(), _TYPES[grad_out.dtype]
    n = lib.semicrf_embed_grad_bytes(typ, B, T, V, N)
    ws = _workspace("semicrf_embed_grad", n, grad_out.device, workspace)
    out = grad_out.new_empty((V, N))
    word = _status(check_status, grad_out.device)
    _run("semicrf_embed_grad", dev, word, tokens.data_ptr(), bits, _ptr(lengths),
         grad_out.data_ptr(), typ, B, T, V, N, scale, _raw_stream(dev), ws.data_ptr(), n,
         out.data_ptr(), _ptr(word))
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
        grad = first_order("embed", lambda: embed_grad(tokens, g.contiguous(), ctx.V, scale=ctx.scale,
                                                       lengths=lengths), g)
        return None, grad, None, None, None


# ---------------------------------------------------------------- layer norm

def _norm_shape(x, weight, bias):
    """Device index, B, T, N and the type of the weights."""
    dev = _index("x", x)
    if x.dim() != 3 or not x.is_contiguous():
        raise ValueError("x must be contiguous [B, T, N]")
    B, T, N = x.shape
    first = weight if weight is not None else bias
    wtype = x.dtype if first is None else first.dtype
    if wtype is not x.dtype and wtype is not torch.float32:
        raise TypeError(f"weight and bias must be {x.dtype} or float32, got {wtype}")
    if weight is not None:
        _need("weight", weight, wtype, (N,), dev)
    if bias is not None:
        _need("bias", bias, wtype, (N,), dev)
    return dev, B, T, N, wtype


def layer_norm(x, weight=None, bias=None, *, eps=1e-5, lengths=None, want_stats=False,
               check_status=False):
    """Layer norm over the last axis of x [B, T, N].  weight, bias [N] in x's type or float32
    (None: ones, zeros).  With want_stats, (y, mean [B, T], rstd [B, T]), which
    layer_norm_grad takes; those two carry no gradient."""
    dev, B, T, N, wtype = _norm_shape(x, weight, bias)
    if _tracked(x, weight, bias):
        y, mean, rstd = _LayerNorm.apply(x, weight, bias, float(eps), lengths, wtype, check_status)
        return (y, mean, rstd) if want_stats else y
    _lengths(lengths, B, dev)
    y = torch.empty_like(x)
    mean = rstd = None
    if want_stats:
        mean, rstd = (torch.empty((B, T), dtype=torch.float32, device=x.device) for _ in range(2))
    word = _status(check_status, x.device)
    _run("semicrf_layer_norm", dev, word, x.data_ptr(), _TYPES[x.dtype], _ptr(weight),
         _ptr(bias), _TYPES[wtype], _ptr(lengths), B, T, N, eps, _raw_stream(dev), y.data_ptr(),
         _ptr(mean), _ptr(rstd), _ptr(word))
    return (y, mean, rstd) if want_stats else y


def layer_norm_grad(grad_out, x, weight, mean, rstd, *, lengths=None, want_params=True,
                    workspace=None, check_status=False) -> dict:
    """Gradients of layer_norm from the mean and rstd it left: a dict with grad_x [B, T, N] and,
    unless want_params is False, grad_weight and grad_bias [N] in the weight's type (x's where
    weight is None)."""
    dev, B, T, N, wtype = _norm_shape(x, weight, None)
    return _norm_grad(grad_out, x, weight, wtype, mean, rstd, lengths, want_params, workspace,
                      check_status, dev, B, T, N)


def _norm_grad(grad_out, x, weight, wtype, mean, rstd, lengths, want_params, workspace,
               check_status, dev, B, T, N):
    _need("grad_out", grad_out, x.dtype, x.shape, dev)
    _need("mean", mean, torch.float32, (B, T), dev)
    _need("rstd", rstd, torch.float32, (B, T), dev)
    _lengths(lengths, B, dev)
    lib = _native.load()
    n = lib.semicrf_layer_norm_grad_bytes(_TYPES[x.dtype], B, T, N)
    ws = _workspace("semicrf_layer_norm_grad", n, x.device, workspace)
    gx = torch.empty_like(x)
    gw = gb = None
    if want_params:
        gw, gb = (torch.empty(N, dtype=wtype, device=x.device) for _ in range(2))
    word = _status(check_status, x.device)
    _run("semicrf_layer_norm_grad", dev, word, grad_out.data_ptr(), x.data_ptr(),
         _TYPES[x.dtype], _ptr(weight), _TYPES[wtype], mean.data_ptr(), rstd.data_ptr(),
         _ptr(lengths), B, T, N, _raw_stream(dev), ws.data_ptr(), n, gx.data_ptr(), _ptr(gw),
         _ptr(gb), _ptr(word))
    out = {"grad_x": gx}
    if want_params:
        out.update(grad_weight=gw, grad_bias=gb)
    return out


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, lengths, wtype, check_status):
        ctx.wtype = wtype
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

        def grads():
            d = _norm_grad(g.contiguous(), x, weight, ctx.wtype, mean, rstd, lengths,
                           need_w or need_b, None, False, x.get_device(), B, T, N)
            return (d["grad_x"], d["grad_weight"] if need_w else None,
                    d["grad_bias"] if need_b else None)

        return *first_order("layer_norm", grads, g, x, weight), None, None, None, None


# ---------------------------------------------------------------- attention

def _attention(q, k, v, log_decay, scale, lengths, state, pool, dims):
    """Device index and the checked argument struct; q, k, v [B, T, H, D] (dims 4), or [B, H, D] for
    one token (dims 3) with states in a pool of `pool` rows."""
    dev = _index("q", q)
    try:
        (B, *qt, Hq, Dk), (Bk, *kt, Hk, Dkk), (Bv, *vt, Hv, Dv) = q.shape, k.shape, v.shape
    except (AttributeError, ValueError):
        raise ValueError(f"q, k and v must be tensors of {dims} dimensions") from None
    if len(qt) != dims - 3 or qt != kt or qt != vt or not B == Bk == Bv or Hk != Hv or Dk != Dkk or \
            Hk < 1 or Hq % Hk:
        raise ValueError(f"shape mismatch: q {list(q.shape)}, k {list(k.shape)}, v "
                         f"{list(v.shape)}; query heads must be a multiple of key heads")
    if k.dtype is not q.dtype or v.dtype is not q.dtype:
        raise TypeError(f"q, k and v must be of one type, got {q.dtype}, {k.dtype}, {v.dtype}")
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError(f"k and v must be on cuda:{dev}")
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    if qs[-1] != 1 and Dk != 1 or ks[-1] != 1 and Dk != 1 or vs[-1] != 1 and Dv != 1:
        raise ValueError("the last axis of q, k and v must be dense")
    _need("log_decay", log_decay, torch.float32, (Hq,), dev)
    _lengths(lengths, B, dev)
    if state is not None:
        _need("state", state, torch.float32, (B if pool is None else pool, Hq, Dk, Dv), dev)
    S = _native.Strides
    return dev, _native.Attention(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), S(qs[0], qs[-3], qs[-2]), S(ks[0], ks[-3], ks[-2]),
        S(vs[0], vs[-3], vs[-2]), _ptr(lengths), log_decay.data_ptr(), _ptr(state),
        Dk ** -0.5 if scale is None else scale, _TYPES[q.dtype], B, qt[0] if qt else 1, Hq, Hk, Dk, Dv)


def decay_attention(q, k, v, log_decay, *, scale=None, lengths=None, state=None,
                    want_state=False, workspace=None, check_status=False):
    """S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T and o_t = scale q_t^T S_t for every position:
    q [B, T, Hq, Dk], k [B, T, Hk, Dk], v [B, T, Hk, Dv] (views with a dense last axis), Hq a
    multiple of Hk, Dk and Dv up to 128; log_decay [Hq] float32, a constant; scale Dk**-0.5 by
    default; state [B, Hq, Dk, Dv] float32 before the first position (None: 0).  Returns o
    [B, T, Hq, Dv], and with want_state also the state after each sequence's last position."""
    if _tracked(log_decay):
        raise ValueError("log_decay is a constant of the head: it has no gradient")
    if _tracked(q, k, v, state):
        o, end = _DecayAttention.apply(q, k, v, log_decay, scale, lengths, state, want_state,
                                       check_status)
        return (o, end) if want_state else o
    dev, a = _attention(q, k, v, log_decay, scale, lengths, state, None, 4)
    lib = _native.load()
    n = lib.semicrf_decay_attention_bytes(a, 0)
    ws = _workspace("semicrf_decay_attention", n, q.device, workspace)
    out = q.new_empty((a.B, a.T, a.Hq, a.Dv))
    end = q.new_empty((a.B, a.Hq, a.Dk, a.Dv), dtype=torch.float32) if want_state else None
    word = _status(check_status, q.device)
    _run("semicrf_decay_attention", dev, word, a, _raw_stream(dev), ws.data_ptr(), n,
         out.data_ptr(), _ptr(end), _ptr(word))
    return (out, end) if want_state else out


def decay_attention_grad(grad_out, q, k, v, log_decay, *, scale=None, lengths=None, state=None,
                         grad_state=None, workspace=None, check_status=False) -> dict:
    """Gradients of decay_attention from those of its output, grad_out [B, T, Hq, Dv], and of its
    final state, grad_state [B, Hq, Dk, Dv] (None: 0): a dict with grad_q, grad_k, grad_v and,
    where an initial state is given, grad_state."""
    dev, a = _attention(q, k, v, log_decay, scale, lengths, state, None, 4)
    lib = _native.load()
    _need("grad_out", grad_out, q.dtype, (a.B, a.T, a.Hq, a.Dv), dev)
    if grad_state is not None:
        _need("grad_state", grad_state, torch.float32, (a.B, a.Hq, a.Dk, a.Dv), dev)
    n = lib.semicrf_decay_attention_bytes(a, 1)
    ws = _workspace("semicrf_decay_attention_grad", n, q.device, workspace)
    gq, gk, gv = (x.new_empty(x.shape) for x in (q, k, v))
    gs = torch.empty_like(state) if state is not None else None
    word = _status(check_status, q.device)
    _run("semicrf_decay_attention_grad", dev, word, a, grad_out.data_ptr(), _ptr(grad_state),
         _raw_stream(dev), ws.data_ptr(), n, gq.data_ptr(), gk.data_ptr(), gv.data_ptr(),
         _ptr(gs), _ptr(word))
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

        def grads():
            d = decay_attention_grad(g.contiguous(), q, k, v, log_decay, scale=ctx.scale,
                                     lengths=lengths, state=state,
                                     grad_state=None if g_state is None else g_state.contiguous())
            return d["grad_q"], d["grad_k"], d["grad_v"], d.get("grad_state")

        gq, gk, gv, gs = first_order("decay_attention", grads, g, g_state, q, k, v, state)
        return gq, gk, gv, None, None, None, gs, None, None


def decay_attention_step(q, k, v, log_decay, state, *, scale=None, slots=None,
                         state_out=None) -> torch.Tensor:
    """One token of B streams: q [B, Hq, Dk], k [B, Hk, Dk], v [B, Hk, Dv] and a pool of states
    [pool, Hq, Dk, Dv] float32, updated in place (or written to state_out, whose other rows are
    left alone).  Stream b uses row slots[b] (int32; None: row b).  A slot outside [0, pool) is
    idle: its output is 0.  Slots in use must be distinct.  Returns o [B, Hq, Dv]; carries no
    gradient, and refuses to overwrite a state that wants one.  Autograd sees the write as that of
    any in-place operation."""
    try:
        pool = state.shape[0]
    except (AttributeError, IndexError):
        raise ValueError("state must be [pool, Hq, Dk, Dv]") from None
    dev, a = _attention(q, k, v, log_decay, scale, None, state, pool, 3)
    if slots is not None:
        _need("slots", slots, torch.int32, (a.B,), dev)
    elif pool < a.B:
        raise ValueError(f"a pool of {pool} states for {a.B} streams needs slots")
    if state_out is None:
        state_out = state
    else:
        _need("state_out", state_out, torch.float32, state.shape, dev)
    if state_out.requires_grad and torch.is_grad_enabled():
        raise ValueError("the state that is written requires a gradient, which a step does not carry")
    out = q.new_empty((a.B, a.Hq, a.Dv))
    _run("semicrf_decay_attention_step", dev, None, a, _ptr(slots), pool, _raw_stream(dev),
         out.data_ptr(), state_out.data_ptr())
    increment_version(state_out)
    return out
