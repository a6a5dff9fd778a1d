"""A block around its mixer, and what an encoder learns before there are segments: gated
recurrence, residual norm and the token loss.

Like the encoder operators these functions check and marshal arguments; the work runs in the
library's HIP kernels, on torch's current stream.

    gated_recurrence(x, decay_gate, input_gate, log_decay)  -> h  [B, T, N] (and the final state)
    gated_recurrence_step(x, ..., state)                    -> h  [B, N], one token a stream
    residual_norm(x, branch, weight, bias, gate=, scale=)   -> r, y  [B, T, N]
    token_nll(x, table, targets)                            -> loss  [B, T] float32

gated_recurrence, residual_norm and token_nll are differentiable, once and backward: a derivative of
their gradients and a forward-mode tangent raise.  The functions named _grad are the gradients by
themselves; they and gated_recurrence_step carry none.  Types, lengths, padding and check_status are
those of the encoder operators.
"""

from __future__ import annotations

import torch
from torch.autograd.graph import increment_version

from . import _native, encoder
from ._autograd import first_order
from .encoder import _TYPES, _index, _lengths, _need, _ptr, _run, _status, _tokens, _tracked, _workspace

__all__ = ["gated_recurrence", "gated_recurrence_grad", "gated_recurrence_step", "residual_norm",
           "residual_norm_grad", "token_nll", "token_nll_grad"]


def _view(name, x, like, dev):
    """Refuses what is not a tensor like another with a dense last axis; its strides but the last."""
    try:
        if x.dtype is like.dtype and x.shape == like.shape and x.get_device() == dev:
            s = x.stride()
            if s[-1] == 1 or x.shape[-1] == 1:
                return _native.Strides2(s[0], s[1] if len(s) == 3 else 0)
    except AttributeError:
        pass
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if x.get_device() != dev:
        raise ValueError(f"{name} is on {x.device}, expected cuda:{dev}")
    if x.dtype is not like.dtype:
        raise TypeError(f"{name} must be {like.dtype}, got {x.dtype}")
    if x.shape != like.shape:
        raise ValueError(f"{name} must be {list(like.shape)}, got {list(x.shape)}")
    raise ValueError(f"the last axis of {name} must be dense")


# ---------------------------------------------------------------- gated recurrence

def _recurrence(x, decay_gate, input_gate, log_decay, lengths, state, pool, dims):
    """Device index and the checked argument struct; x and the gates [B, T, N] (dims 3), or [B, N]
    for one token (dims 2) with states in a pool of `pool` rows."""
    dev = _index("x", x)
    if x.dim() != dims:
        raise ValueError(f"x must be {'[B, T, N]' if dims == 3 else '[B, N]'}, got {list(x.shape)}")
    B, N = x.shape[0], x.shape[-1]
    sx, sr, si = (_view("x", x, x, dev), _view("decay_gate", decay_gate, x, dev),
                  _view("input_gate", input_gate, x, dev))
    _need("log_decay", log_decay, torch.float32, (N,), dev)
    _lengths(lengths, B, dev)
    if state is not None:
        _need("state", state, torch.float32, (B if pool is None else pool, N), dev)
    return dev, _native.Recurrence(
        x.data_ptr(), decay_gate.data_ptr(), input_gate.data_ptr(), sx, sr, si, _ptr(lengths),
        log_decay.data_ptr(), _ptr(state), _TYPES[x.dtype], B, x.shape[1] if dims == 3 else 1, N)


def gated_recurrence(x, decay_gate, input_gate, log_decay, *, lengths=None, state=None,
                     want_state=False, want_starts=False, workspace=None, check_status=False):
    """h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sig(input_gate_t) x_t with a_t = exp(log_decay
    sig(decay_gate_t)), for every position and channel: x and the gates [B, T, N] (views with a dense
    last axis, the gates before their sigmoid), log_decay [N] float32, at most 0; state [B, N] float32
    before the first position (None: 0).  Returns h [B, T, N]; with want_state also the state after
    each sequence's last position; with want_starts also the states [B, ceil(T / 16), N] float32
    before every 16th position, which gated_recurrence_grad takes and which carry no gradient."""
    if _tracked(x, decay_gate, input_gate, log_decay, state):
        h, end, starts = _GatedRecurrence.apply(x, decay_gate, input_gate, log_decay, lengths, state,
                                                want_state, want_starts, check_status)
    else:
        h, end, starts = _run_recurrence(x, decay_gate, input_gate, log_decay, lengths, state,
                                         want_state, want_starts, workspace, check_status)
    out = (h,) + ((end,) if want_state else ()) + ((starts,) if want_starts else ())
    return out if len(out) > 1 else h


def _run_recurrence(x, decay_gate, input_gate, log_decay, lengths, state, want_state, want_starts,
                    workspace, check_status):
    dev, a = _recurrence(x, decay_gate, input_gate, log_decay, lengths, state, None, 3)
    n = _native.load().semicrf_gated_recurrence_bytes(a, 0)
    ws = _workspace("semicrf_gated_recurrence", n, x.device, workspace)
    h = x.new_empty((a.B, a.T, a.N))
    end = x.new_empty((a.B, a.N), dtype=torch.float32) if want_state else None
    starts = None
    if want_starts:
        spans = -(-a.T // _native.RECURRENCE_SPAN)
        starts = x.new_empty((a.B, spans, a.N), dtype=torch.float32)
    word = _status(check_status, x.device)
    _run("semicrf_gated_recurrence", dev, word, a, encoder._raw_stream(dev), ws.data_ptr(), n,
         h.data_ptr(), _ptr(end), _ptr(starts), _ptr(word))
    return h, end, starts


def gated_recurrence_grad(grad_out, x, decay_gate, input_gate, log_decay, starts, *, lengths=None,
                          state=None, grad_state=None, workspace=None, check_status=False) -> dict:
    """Gradients of gated_recurrence from those of its output, grad_out [B, T, N], and of its final
    state, grad_state [B, N] (None: 0), and the starts it left: a dict with grad_x,
    grad_decay_gate, grad_input_gate, grad_log_decay [N] float32 and, where an initial state is given,
    grad_state."""
    dev, a = _recurrence(x, decay_gate, input_gate, log_decay, lengths, state, None, 3)
    _need("grad_out", grad_out, x.dtype, (a.B, a.T, a.N), dev)
    _need("starts", starts, torch.float32, (a.B, -(-a.T // _native.RECURRENCE_SPAN), a.N), dev)
    if grad_state is not None:
        _need("grad_state", grad_state, torch.float32, (a.B, a.N), dev)
    n = _native.load().semicrf_gated_recurrence_bytes(a, 1)
    ws = _workspace("semicrf_gated_recurrence_grad", n, x.device, workspace)
    gx, gr, gi = (x.new_empty((a.B, a.T, a.N)) for _ in range(3))
    gl = torch.empty_like(log_decay)
    gs = torch.empty_like(state) if state is not None else None
    word = _status(check_status, x.device)
    _run("semicrf_gated_recurrence_grad", dev, word, a, starts.data_ptr(), grad_out.data_ptr(),
         _ptr(grad_state), encoder._raw_stream(dev), ws.data_ptr(), n, gx.data_ptr(), gr.data_ptr(),
         gi.data_ptr(), gl.data_ptr(), _ptr(gs), _ptr(word))
    out = {"grad_x": gx, "grad_decay_gate": gr, "grad_input_gate": gi, "grad_log_decay": gl}
    if gs is not None:
        out["grad_state"] = gs
    return out


class _GatedRecurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, decay_gate, input_gate, log_decay, lengths, state, want_state, want_starts,
                check_status):
        h, end, starts = _run_recurrence(x, decay_gate, input_gate, log_decay, lengths, state,
                                         want_state, True, None, check_status)
        ctx.save_for_backward(x, decay_gate, input_gate, log_decay, lengths, state, starts)
        ctx.set_materialize_grads(False)
        if not want_starts:
            return h, end, None
        ctx.mark_non_differentiable(starts)
        return h, end, starts

    @staticmethod
    def backward(ctx, g, g_state, _starts):
        if g is None and g_state is None:
            return (None,) * 9
        x, decay_gate, input_gate, log_decay, lengths, state, starts = ctx.saved_tensors
        if g is None:
            g = torch.zeros(x.shape, dtype=x.dtype, device=x.device)

        def grads():
            d = gated_recurrence_grad(g.contiguous(), x, decay_gate, input_gate, log_decay, starts,
                                      lengths=lengths, state=state,
                                      grad_state=None if g_state is None else g_state.contiguous())
            return (d["grad_x"], d["grad_decay_gate"], d["grad_input_gate"], d["grad_log_decay"],
                    d.get("grad_state"))

        gx, gr, gi, gl, gs = first_order("gated_recurrence", grads, g, g_state, x, decay_gate,
                                         input_gate, log_decay, state)
        return gx, gr, gi, gl, None, gs, None, None, None


def gated_recurrence_step(x, decay_gate, input_gate, log_decay, state, *, slots=None,
                          state_out=None) -> torch.Tensor:
    """One token of B streams: x and the gates [B, N] and a pool of states [pool, N] float32, updated
    in place (or written to state_out, whose other rows are left alone).  slots, idle rows and
    autograd as in decay_attention_step.  Returns h [B, N]."""
    try:
        pool = state.shape[0]
    except (AttributeError, IndexError):
        raise ValueError("state must be [pool, N]") from None
    dev, a = _recurrence(x, decay_gate, input_gate, log_decay, None, state, pool, 2)
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
    out = x.new_empty((a.B, a.N))
    _run("semicrf_gated_recurrence_step", dev, None, a, _ptr(slots), pool, encoder._raw_stream(dev),
         out.data_ptr(), state_out.data_ptr())
    increment_version(state_out)
    return out


# ---------------------------------------------------------------- residual norm

def _residual(x, branch, weight, bias, gate, scale, norm_branch, branch_weight, branch_bias, center,
              eps, lengths):
    """Device index, the checked argument struct and the type of the weights."""
    dev = _index("x", x)
    if x.dim() != 3 or not x.is_contiguous():
        raise ValueError("x must be contiguous [B, T, N]")
    if not norm_branch and (branch_weight is not None or branch_bias is not None):
        raise ValueError("branch_weight and branch_bias need norm_branch")
    B, T, N = x.shape
    sb = _view("branch", branch, x, dev)
    sg = _native.Strides2(0, 0) if gate is None else _view("gate", gate, x, dev)
    wtype, size = None, (N,)
    for name, p in (("scale", scale), ("weight", weight), ("bias", bias),
                    ("branch_weight", branch_weight), ("branch_bias", branch_bias)):
        if p is None:
            continue
        if wtype is None:
            wtype = getattr(p, "dtype", None)
            if wtype is not x.dtype and wtype is not torch.float32:
                raise TypeError(f"weights must be {x.dtype} or float32, got {wtype}")
        _need(name, p, wtype, size, dev)
    wtype = wtype or x.dtype
    _lengths(lengths, B, dev)
    return dev, _native.Residual(
        x.data_ptr(), branch.data_ptr(), _ptr(gate), sb, sg, _ptr(scale), _ptr(weight), _ptr(bias),
        _ptr(branch_weight), _ptr(branch_bias), _ptr(lengths), eps, _TYPES[x.dtype], _TYPES[wtype],
        bool(norm_branch), bool(center), B, T, N), wtype


def residual_norm(x, branch, weight=None, bias=None, *, gate=None, scale=None, norm_branch=False,
                  branch_weight=None, branch_bias=None, center=True, eps=1e-5, lengths=None,
                  want_stats=False, check_status=False):
    """r = x + scale sig(gate) f(branch) and y = norm(r) weight + bias, where f is the identity or, with
    norm_branch, norm(branch) branch_weight + branch_bias.  x [B, T, N] contiguous, branch and gate
    shaped like it (views with a dense last axis; no gate: 1); scale, weights and biases [N] in
    x's type or float32, all in one (None: ones, zeros).  norm is layer norm, or with center=False the
    root-mean-square norm.  Returns (r, y); with want_stats, (r, y, stats [B, T, 4] float32), which
    residual_norm_grad takes and which carry no gradient."""
    if _tracked(x, branch, gate, scale, weight, bias, branch_weight, branch_bias):
        r, y, stats = _ResidualNorm.apply(x, branch, weight, bias, gate, scale, branch_weight,
                                          branch_bias, norm_branch, center, float(eps), lengths,
                                          check_status)
    else:
        r, y, stats = _run_residual(x, branch, weight, bias, gate, scale, branch_weight, branch_bias,
                                    norm_branch, center, eps, lengths, want_stats, check_status)
    return (r, y, stats) if want_stats else (r, y)


def _run_residual(x, branch, weight, bias, gate, scale, branch_weight, branch_bias, norm_branch,
                  center, eps, lengths, want_stats, check_status):
    dev, a, _ = _residual(x, branch, weight, bias, gate, scale, norm_branch, branch_weight,
                          branch_bias, center, eps, lengths)
    r, y = torch.empty_like(x), torch.empty_like(x)
    stats = x.new_empty((a.B, a.T, 4), dtype=torch.float32) if want_stats else None
    word = _status(check_status, x.device)
    _run("semicrf_residual_norm", dev, word, a, encoder._raw_stream(dev), r.data_ptr(), y.data_ptr(),
         _ptr(stats), _ptr(word))
    return r, y, stats


def residual_norm_grad(grad_r, grad_y, x, branch, weight, stats, *, bias=None, gate=None, scale=None,
                       norm_branch=False, branch_weight=None, branch_bias=None, center=True,
                       lengths=None, want_params=True, workspace=None, check_status=False) -> dict:
    """Gradients of residual_norm from those of r and y [B, T, N] (None: 0) and the stats it left: a
    dict with grad_x, grad_branch, with a gate grad_gate and, unless want_params is False,
    grad_weight, grad_bias, grad_scale and, with norm_branch, grad_branch_weight and
    grad_branch_bias [N] in the weights' type (x's where there are none).  bias counts for that type
    only: no gradient depends on it."""
    dev, a, wtype = _residual(x, branch, weight, bias, gate, scale, norm_branch, branch_weight,
                              branch_bias, center, 0.0, lengths)
    return _residual_grad(dev, a, wtype, grad_r, grad_y, x, gate, stats, want_params, workspace,
                          check_status)


def _residual_grad(dev, a, wtype, grad_r, grad_y, x, gate, stats, want_params, workspace, check_status):
    for name, g in (("grad_r", grad_r), ("grad_y", grad_y)):
        if g is not None:
            _need(name, g, x.dtype, x.shape, dev)
    _need("stats", stats, torch.float32, (a.B, a.T, 4), dev)
    n = _native.load().semicrf_residual_norm_grad_bytes(a.dtype, a.B, a.T, a.N)
    ws = _workspace("semicrf_residual_norm_grad", n, x.device, workspace)
    gx, gb = torch.empty_like(x), torch.empty_like(x)
    gg = torch.empty_like(x) if gate is not None else None
    params = x.new_empty((5, a.N), dtype=wtype) if want_params else None
    word = _status(check_status, x.device)
    _run("semicrf_residual_norm_grad", dev, word, a, stats.data_ptr(), _ptr(grad_r), _ptr(grad_y),
         encoder._raw_stream(dev), ws.data_ptr(), n, gx.data_ptr(), gb.data_ptr(), _ptr(gg),
         _ptr(params), _ptr(word))
    out = {"grad_x": gx, "grad_branch": gb}
    if gate is not None:
        out["grad_gate"] = gg
    if want_params:
        names = ("weight", "bias", "scale") + (("branch_weight", "branch_bias") if a.norm_branch else ())
        out.update(("grad_" + k, p) for k, p in zip(names, params.unbind(0)))
    return out


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, branch, weight, bias, gate, scale, branch_weight, branch_bias, norm_branch,
                center, eps, lengths, check_status):
        r, y, stats = _run_residual(x, branch, weight, bias, gate, scale, branch_weight, branch_bias,
                                    norm_branch, center, eps, lengths, True, check_status)
        ctx.save_for_backward(x, branch, weight, bias, gate, scale, branch_weight, branch_bias, lengths,
                              stats)
        ctx.norm_branch, ctx.center = norm_branch, center
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(stats)
        return r, y, stats

    @staticmethod
    def backward(ctx, g_r, g_y, _stats):
        (x, branch, weight, bias, gate, scale, branch_weight, branch_bias, lengths,
         stats) = ctx.saved_tensors
        need = dict(zip(("x", "branch", "weight", "bias", "gate", "scale", "branch_weight",
                         "branch_bias"), ctx.needs_input_grad))
        if g_r is None and g_y is None:
            return (None,) * 13

        def grads():
            dev, a, wtype = _residual(x, branch, weight, bias, gate, scale, ctx.norm_branch,
                                      branch_weight, branch_bias, ctx.center, 0.0, lengths)
            d = _residual_grad(dev, a, wtype, None if g_r is None else g_r.contiguous(),
                               None if g_y is None else g_y.contiguous(), x, gate, stats,
                               any(need[k] for k in list(need)[2:] if k != "gate"), None, False)
            return tuple(d["grad_" + k] if need[k] else None for k in need)

        d = first_order("residual_norm", grads, g_r, g_y, x, branch, weight, gate, scale, branch_weight,
                        branch_bias)
        return *d, None, None, None, None, None


# ---------------------------------------------------------------- token loss

def _nll_args(x, table, targets, lengths):
    """Device index, B, T, V, N and the targets' bits."""
    dev = _index("x", x)
    if x.dim() != 3 or not x.is_contiguous():
        raise ValueError("x must be contiguous [B, T, N]")
    B, T, N = x.shape
    try:
        V = table.shape[0]
    except (AttributeError, IndexError):
        raise ValueError("table must be [V, N]") from None
    _need("table", table, x.dtype, (V, N), dev)
    Bt, Tt, bits = _tokens(targets, dev)
    if (Bt, Tt) != (B, T):
        raise ValueError(f"targets must be [{B}, {T}], got {list(targets.shape)}")
    _lengths(lengths, B, dev)
    return dev, B, T, V, N, bits


def token_nll(x, table, targets, *, scale=1.0, lengths=None, want_lse=False, workspace=None,
              check_status=False):
    """-log softmax(scale x table^T)[target] of every position: x [B, T, N], table [V, N] of x's type
    (embed's, or another), targets [B, T] int32 or int64; loss [B, T] float32.  A negative target
    marks a position with nothing to predict: its x is not read, its loss is 0.  A target of V or
    more gives NaN.  The scores are formed in pieces and not kept.  With want_lse, (loss, lse
    [B, T] float32), which token_nll_grad takes; lse carries no gradient."""
    if _tracked(x, table):
        loss, lse = _TokenNll.apply(x, table, targets, float(scale), lengths, want_lse, check_status)
    else:
        loss, lse = _run_nll(x, table, targets, scale, lengths, want_lse, workspace, check_status)
    return (loss, lse) if want_lse else loss


def _run_nll(x, table, targets, scale, lengths, want_lse, workspace, check_status):
    dev, B, T, V, N, bits = _nll_args(x, table, targets, lengths)
    typ = _TYPES[x.dtype]
    n = _native.load().semicrf_token_nll_table_bytes(typ, B, T, V, N, table.data_ptr(), 0)
    ws = _workspace("semicrf_token_nll", n, x.device, workspace)
    loss = x.new_empty((B, T), dtype=torch.float32)
    lse = torch.empty_like(loss) if want_lse else None
    word = _status(check_status, x.device)
    _run("semicrf_token_nll", dev, word, x.data_ptr(), table.data_ptr(), typ, targets.data_ptr(), bits,
         _ptr(lengths), B, T, V, N, scale, encoder._raw_stream(dev), ws.data_ptr(), n, loss.data_ptr(),
         _ptr(lse), _ptr(word))
    return loss, lse


def token_nll_grad(grad_loss, x, table, targets, lse, *, scale=1.0, lengths=None, want_x=True,
                   want_table=True, workspace=None, check_status=False) -> dict:
    """Gradients of token_nll from those of its loss, grad_loss [B, T] float32, and the lse it left: a
    dict with grad_x [B, T, N] and grad_table [V, N] (each unless it is not wanted).  A target of V or
    more counts for nothing."""
    dev, B, T, V, N, bits = _nll_args(x, table, targets, lengths)
    if not want_x and not want_table:
        raise ValueError("one of the two gradients must be wanted")
    _need("grad_loss", grad_loss, torch.float32, (B, T), dev)
    _need("lse", lse, torch.float32, (B, T), dev)
    typ = _TYPES[x.dtype]
    n = _native.load().semicrf_token_nll_table_bytes(typ, B, T, V, N, table.data_ptr(), 1)
    ws = _workspace("semicrf_token_nll_grad", n, x.device, workspace)
    gx = torch.empty_like(x) if want_x else None
    gt = torch.empty_like(table) if want_table else None
    word = _status(check_status, x.device)
    _run("semicrf_token_nll_grad", dev, word, grad_loss.data_ptr(), x.data_ptr(), table.data_ptr(), typ,
         targets.data_ptr(), bits, _ptr(lengths), lse.data_ptr(), B, T, V, N, scale,
         encoder._raw_stream(dev), ws.data_ptr(), n, _ptr(gx), _ptr(gt), _ptr(word))
    return {k: v for k, v in (("grad_x", gx), ("grad_table", gt)) if v is not None}


class _TokenNll(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, table, targets, scale, lengths, want_lse, check_status):
        loss, lse = _run_nll(x, table, targets, scale, lengths, True, None, check_status)
        ctx.save_for_backward(x, table, targets, lengths, lse)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        if not want_lse:
            return loss, None
        ctx.mark_non_differentiable(lse)
        return loss, lse

    @staticmethod
    def backward(ctx, g, _lse):
        if g is None:
            return (None,) * 7
        x, table, targets, lengths, lse = ctx.saved_tensors
        need_x, need_table = ctx.needs_input_grad[:2]

        def grads():
            d = token_nll_grad(g.contiguous(), x, table, targets, lse, scale=ctx.scale, lengths=lengths,
                               want_x=need_x, want_table=need_table)
            return d.get("grad_x"), d.get("grad_table")

        return *first_order("token_nll", grads, g, x, table), None, None, None, None, None
