"""How the block operators stand in torch's autograd and on a GPU that is not the current one, on the
CPU: the kernels are replaced by plain torch expressions or by nothing, everything around them is
the package's own."""

import pytest
import torch

import semi_markov_crf_amd as crf
from semi_markov_crf_amd import blocks, encoder
from test_current_device import array, calls, only_there  # noqa: F401


def plain_recurrence(x, r, i, lam, state):
    h = torch.zeros(x.shape[0], x.shape[2]) if state is None else state
    out = []
    for t in range(x.shape[1]):
        s = lam * torch.sigmoid(r[:, t])
        h = torch.exp(s) * h + torch.sqrt(-torch.expm1(2 * s)) * torch.sigmoid(i[:, t]) * x[:, t]
        out.append(h)
    return torch.stack(out, 1), h


def plain_residual(x, branch, weight, bias, gate, scale):
    r = x + scale * torch.sigmoid(gate) * branch
    c = r - r.mean(-1, keepdim=True)
    return r, c * torch.rsqrt(c.square().mean(-1, keepdim=True) + 1e-5) * weight + bias


def plain_nll(x, table, targets, scale):
    z = scale * (x @ table.t())
    return torch.logsumexp(z, -1) - z.gather(-1, targets[..., None])[..., 0]


def grads_of(f, args, outs):
    with torch.enable_grad():
        a = [v.detach().requires_grad_() for v in args]
        y = f(*a)
        y, outs = (y, outs) if isinstance(y, tuple) else ((y,), (outs,))
        pairs = [(v, g) for v, g in zip(y, outs) if g is not None]
        return torch.autograd.grad([v for v, _ in pairs], a, [g for _, g in pairs], allow_unused=True)


@pytest.fixture
def plain(monkeypatch):
    def recurrence(x, r, i, lam, lengths, state, want_state, want_starts, ws, check):
        h, end = plain_recurrence(x, r, i, lam, state)
        return h, end if want_state else None, torch.zeros(1)

    def recurrence_grad(g, x, r, i, lam, starts, *, lengths, state, grad_state):
        d = grads_of(plain_recurrence, (x, r, i, lam, state), (g, grad_state))
        return dict(zip(("grad_x", "grad_decay_gate", "grad_input_gate", "grad_log_decay", "grad_state"), d))

    def residual(x, branch, weight, bias, gate, scale, bw, bb, *rest):
        return (*plain_residual(x, branch, weight, bias, gate, scale), torch.zeros(1))

    def residual_grad(dev, a, wtype, g_r, g_y, x, gate, stats, want_params, ws, check):
        d = grads_of(plain_residual, a, (g_r, g_y))
        return dict(zip(("grad_x", "grad_branch", "grad_weight", "grad_bias", "grad_gate", "grad_scale"), d))

    def check_residual(x, branch, weight, bias, gate, scale, *rest):
        return -1, (x, branch, weight, bias, gate, scale), torch.float32

    def nll(x, table, targets, scale, lengths, want_lse, ws, check):
        return plain_nll(x, table, targets, scale), torch.zeros(1)

    def nll_grad(g, x, table, targets, lse, *, scale, lengths, want_x, want_table):
        return dict(zip(("grad_x", "grad_table"), grads_of(lambda *a: plain_nll(*a, targets, scale), (x, table), g)))

    for name, f in (("_run_recurrence", recurrence), ("gated_recurrence_grad", recurrence_grad),
                    ("_run_residual", residual), ("_residual_grad", residual_grad), ("_residual", check_residual),
                    ("_run_nll", nll), ("token_nll_grad", nll_grad)):
        monkeypatch.setattr(blocks, name, f)


def cases():
    torch.manual_seed(0)
    r = lambda *s: torch.randn(*s, requires_grad=True)  # noqa: E731
    lam = (-torch.rand(3) - 0.1).requires_grad_()
    t = torch.tensor([[0, 4]])
    return {
        "gated_recurrence": ([r(2, 4, 3), r(2, 4, 3), r(2, 4, 3), lam, r(2, 3)],
                             lambda x, g, i, d, s: crf.gated_recurrence(x, g, i, d, state=s)),
        "residual_norm": ([r(1, 2, 5), r(1, 2, 5), r(5), r(5), r(1, 2, 5), r(5)],
                          lambda x, o, w, b, z, c: crf.residual_norm(x, o, w, b, gate=z, scale=c)[1]),
        "token_nll": ([r(1, 2, 3), r(5, 3)], lambda x, w: crf.token_nll(x, w, t, scale=0.5)),
    }


NAMES = ["gated_recurrence", "residual_norm", "token_nll"]


@pytest.mark.parametrize("name", NAMES)
def test_gradients_reach_their_inputs(plain, name):
    """Each input's gradient arrives at that input, wanted alone or with the others."""
    args, f = cases()[name]
    same = {"gated_recurrence": lambda *a: plain_recurrence(*a)[0], "residual_norm": lambda *a: plain_residual(*a)[1],
            "token_nll": lambda x, w: plain_nll(x, w, torch.tensor([[0, 4]]), 0.5)}[name]
    g = torch.randn_like(f(*args))
    want = torch.autograd.grad(same(*args), args, g)
    assert all(torch.allclose(a, b) for a, b in zip(torch.autograd.grad(f(*args), args, g), want))
    for k in range(len(args)):
        alone = [a if j == k else a.detach() for j, a in enumerate(args)]
        assert torch.allclose(torch.autograd.grad(f(*alone), args[k], g)[0], want[k])


@pytest.mark.parametrize("name", NAMES)
def test_second_derivatives_are_refused(plain, name):
    args, f = cases()[name]
    first = torch.autograd.grad(f(*args).pow(2).sum(), args)
    again = torch.autograd.grad(f(*args).pow(2).sum(), args, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    with pytest.raises(RuntimeError, match=f"{name} has no second derivatives"):
        torch.autograd.grad(sum((g * g).sum() for g in again) + sum((a * a).sum() for a in args), args)


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("grad", [True, False])
def test_forward_mode_is_refused(plain, name, grad):
    import torch.autograd.forward_ad as fwd
    args, f = cases()[name]
    args = [a.detach() for a in args]
    with torch.set_grad_enabled(grad), fwd.dual_level():
        for i in range(len(args)):
            dual = [fwd.make_dual(a, torch.ones_like(a)) if j == i else a for j, a in enumerate(args)]
            with pytest.raises(RuntimeError, match="forward"):
                f(*dual)


def test_outputs_and_extras(plain):
    """Extras carry no gradient; a state that is returned does."""
    args, _ = cases()["gated_recurrence"]
    h, end, starts = crf.gated_recurrence(*args[:4], state=args[4], want_state=True, want_starts=True)
    assert h.requires_grad and end.requires_grad and not starts.requires_grad
    d = torch.autograd.grad(end.sum(), args)
    want = torch.autograd.grad(plain_recurrence(*args)[1].sum(), args)
    assert all(torch.allclose(a, b) for a, b in zip(d, want))
    args, _ = cases()["residual_norm"]
    r, y, stats = crf.residual_norm(*args[:4], gate=args[4], scale=args[5], want_stats=True)
    assert r.requires_grad and y.requires_grad and not stats.requires_grad
    args, _ = cases()["token_nll"]
    loss, lse = crf.token_nll(*args, torch.tensor([[0, 4]]), want_lse=True)
    assert loss.requires_grad and not lse.requires_grad


def test_a_step_counts_as_an_in_place_write(monkeypatch):
    """And refuses a state that wants a gradient."""
    import types
    monkeypatch.setattr(blocks, "_recurrence", lambda *args: (-1, types.SimpleNamespace(B=2, N=3)))
    monkeypatch.setattr(encoder, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(encoder._native, "call", lambda dev, name, *args: 0)
    monkeypatch.setattr(blocks, "_need", lambda *args: None)
    x, state = torch.zeros(2, 3), torch.ones(2, 3)
    w = torch.ones(2, 3, requires_grad=True)
    y = w * state
    crf.gated_recurrence_step(x, x, x, None, state)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    for call in (lambda: crf.gated_recurrence_step(x, x, x, None, w),
                 lambda: crf.gated_recurrence_step(x, x, x, None, state, state_out=w)):
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
    with torch.no_grad():
        crf.gated_recurrence_step(x, x, x, None, w)


def test_calls_run_on_their_arrays_gpu(calls):  # noqa: F811
    """The library runs with the arrays' GPU current."""
    x, v, state, m = array(2, 3, 8), array(8), array(2, 8), array(2, 3)
    t = array(2, 3, dtype=torch.int32)
    ws = torch.empty(1 << 13, dtype=torch.uint8)
    ws = ws[-ws.data_ptr() % 256:]
    with torch.no_grad():
        crf.gated_recurrence(x, x, x, v, workspace=ws)
        crf.gated_recurrence_grad(x, x, x, x, v, array(2, 1, 8), workspace=ws)
        crf.gated_recurrence_step(state, state, state, v, state.clone())
        crf.residual_norm(x, x, v)
        crf.residual_norm_grad(x, x, x, x, v, array(2, 3, 4), workspace=ws)
        crf.token_nll(x, array(5, 8), t, workspace=ws)
        crf.token_nll_grad(m, x, array(5, 8), t, m, workspace=ws)
    only_there(calls, ["semicrf_gated_recurrence", "semicrf_gated_recurrence_grad", "semicrf_gated_recurrence_step",
                       "semicrf_residual_norm", "semicrf_residual_norm_grad", "semicrf_token_nll",
                       "semicrf_token_nll_grad"])
