"""How the encoder operators stand in torch's autograd, on the CPU: the kernels are replaced by
plain torch expressions, everything around them is the package's own."""

import pytest
import torch

from semi_markov_crf_amd import encoder


def plain_norm(x, weight, bias, eps):
    mean = x.mean(-1)
    rstd = torch.rsqrt((x - mean[..., None]).square().mean(-1) + eps)
    y = (x - mean[..., None]) * rstd[..., None]
    y = y if weight is None else y * weight
    return y if bias is None else y + bias, mean, rstd


def plain_attention(q, k, v, log_decay, scale, state):
    s = torch.zeros(*q.shape[:1], *q.shape[2:], v.shape[-1]) if state is None else state
    out = []
    for t in range(q.shape[1]):
        s = torch.exp(log_decay)[:, None, None] * s + k[:, t, :, :, None] * v[:, t, :, None, :]
        out.append(scale * (q[:, t, :, :, None] * s).sum(-2))
    return torch.stack(out, 1), s


@pytest.fixture
def plain(monkeypatch):
    """The package's calls with plain expressions in place of the library."""
    def embed(tokens, table, *, scale, lengths, check_status):
        return table[tokens] * scale

    def embed_grad(tokens, g, V, *, scale, lengths):
        return torch.zeros(V, g.shape[-1]).index_add_(0, tokens.reshape(-1), g.reshape(-1, g.shape[-1]) * scale)

    def layer_norm(x, weight, bias, *, eps, lengths, want_stats, check_status):
        return plain_norm(x, weight, bias, eps)

    def norm_grad(g, x, weight, wtype, mean, rstd, lengths, want_params, ws, check_status, dev, B, T, N):
        with torch.enable_grad():
            a = [x.detach().requires_grad_(), (torch.ones(N) if weight is None else weight).detach().requires_grad_(),
                 torch.zeros(N, requires_grad=True)]
            d = torch.autograd.grad(plain_norm(*a, 1e-5)[0], a, g)
        return dict(zip(("grad_x", "grad_weight", "grad_bias"), d))

    def attention(q, k, v, log_decay, *, scale, lengths, state, want_state, check_status):
        o, s = plain_attention(q, k, v, log_decay, scale, state)
        return (o, s) if want_state else o

    def attention_grad(g, q, k, v, log_decay, *, scale, lengths, state, grad_state):
        with torch.enable_grad():
            a = [x.detach().requires_grad_() for x in (q, k, v)]
            s0 = None if state is None else state.detach().requires_grad_()
            o, s = plain_attention(*a, log_decay, scale, s0)
            loss = (o * g).sum() + (0 if grad_state is None else (s * grad_state).sum())
            d = torch.autograd.grad(loss, a + ([] if s0 is None else [s0]))
        return dict(zip(("grad_q", "grad_k", "grad_v", "grad_state"), d))

    for name, f in (("embed", embed), ("embed_grad", embed_grad), ("layer_norm", layer_norm),
                    ("_norm_grad", norm_grad), ("decay_attention", attention),
                    ("decay_attention_grad", attention_grad)):
        monkeypatch.setattr(encoder, name, f)


def cases():
    torch.manual_seed(0)
    r = lambda *s: torch.randn(*s, requires_grad=True)  # noqa: E731
    tok, lengths = torch.tensor([[0, 2, 2]]), None
    log_decay = torch.tensor([-0.1, -1.0])
    return {
        "embed": ([r(4, 5)], lambda x: encoder._Embed.apply(tok, x, 2.0, lengths, False)),
        "layer_norm": ([r(1, 3, 5), r(5), r(5)],
                       lambda x, w, b: encoder._LayerNorm.apply(x, w, b, 1e-5, lengths, torch.float32, False)[0]),
        "decay_attention": ([r(1, 3, 2, 4), r(1, 3, 2, 4), r(1, 3, 2, 5), r(1, 2, 4, 5)],
                            lambda q, k, v, s: encoder._DecayAttention.apply(q, k, v, log_decay, 0.5, lengths, s, True,
                                                                             False)[0]),
    }


@pytest.mark.parametrize("name", ["embed", "layer_norm", "decay_attention"])
def test_second_derivatives_are_refused(plain, name):
    """A term of the second order is never left out silently: what depends on the inputs through a
    gradient raises, first derivatives stay what they are."""
    args, f = cases()[name]
    first = torch.autograd.grad(f(*args).pow(2).sum(), args)
    again = torch.autograd.grad(f(*args).pow(2).sum(), args, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    with pytest.raises(RuntimeError, match=f"{name} has no second derivatives"):
        torch.autograd.grad(sum((g * g).sum() for g in again) + sum((a * a).sum() for a in args), args)


@pytest.mark.parametrize("name", ["layer_norm", "decay_attention"])
def test_second_derivatives_under_a_constant_gradient(plain, name):
    """The gradient depends on the inputs also where the output's own gradient is a constant."""
    args, f = cases()[name]
    again = torch.autograd.grad(f(*args).sum(), args, create_graph=True)
    with pytest.raises(RuntimeError, match="no second derivatives"):
        torch.autograd.grad(sum((g * g).sum() for g in again) + sum((a * a).sum() for a in args), args)


def test_a_gradient_linear_in_its_table_has_none(plain):
    """embed's gradient does not depend on the table: under a constant gradient there is nothing to
    refuse."""
    (table,), f = cases()["embed"]
    g, = torch.autograd.grad(f(table).sum(), table, create_graph=True)
    assert not g.requires_grad


def test_second_derivatives_of_log_partition_are_refused(monkeypatch):
    """One position, segments of length one: log Z is the log-sum-exp of the emissions."""
    import semi_markov_crf_amd as crf

    def backward(em, lengths, trans, dur, *, proj_start, proj_end, grad_log_z, delta, want_marginals):
        p = torch.softmax(em[:, 0], -1) * grad_log_z[:, None]
        return {"grad_em": p[:, None], "grad_trans": torch.zeros_like(trans), "grad_dur": p.sum(0, keepdim=True)}

    monkeypatch.setattr(crf, "logz", lambda em, *a, **kw: torch.logsumexp(em[:, 0], -1))
    monkeypatch.setattr(crf, "backward", backward)
    torch.manual_seed(1)
    em = torch.randn(2, 1, 3, requires_grad=True)
    lengths, trans, dur = torch.ones(2, dtype=torch.int32), torch.zeros(3, 3), torch.zeros(1, 3)
    first, = torch.autograd.grad(crf.log_partition(em, lengths, trans, dur).sum(), em)
    assert torch.allclose(first[:, 0], torch.softmax(em[:, 0], -1))
    again, = torch.autograd.grad(crf.log_partition(em, lengths, trans, dur).sum(), em, create_graph=True)
    assert torch.equal(first, again)
    with pytest.raises(RuntimeError, match="log_partition has no second derivatives"):
        torch.autograd.grad((again ** 2).sum() + (em ** 2).sum(), em)


@pytest.mark.parametrize("name", ["embed", "layer_norm", "decay_attention"])
@pytest.mark.parametrize("grad", [True, False])
def test_forward_mode_is_refused(plain, monkeypatch, name, grad):
    """A dual input raises, with gradients on or off: its tangent is not dropped.  The calls go by
    _tracked, and what it sends to the autograd function is refused there."""
    import torch.autograd.forward_ad as fwd
    args, f = cases()[name]
    args = [a.detach() for a in args]
    with torch.set_grad_enabled(grad):
        assert not encoder._tracked(*args, None)
        with fwd.dual_level():
            assert not encoder._tracked(*args, None)
            for i in range(len(args)):
                dual = [fwd.make_dual(a, torch.ones_like(a)) if j == i else a for j, a in enumerate(args)]
                assert encoder._tracked(*dual, None)
                with pytest.raises(RuntimeError, match="forward"):
                    f(*dual)
        assert not encoder._tracked(*args, None)


@pytest.fixture
def step(monkeypatch):
    """decay_attention_step on CPU tensors: the library's call writes a one into the state."""
    import types

    def call(a, slots, pool, stream, out, state_out):
        call.state.data[0, 0, 0, 0] = 1.0          # .data: like a kernel's write, unseen by autograd
        return 0

    a = types.SimpleNamespace(B=2, Hq=2, Dv=5)
    monkeypatch.setattr(encoder, "_attention", lambda *args: (-1, a))
    monkeypatch.setattr(encoder, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(encoder._native, "call", lambda dev, name, *args: call(*args))
    monkeypatch.setattr(encoder, "_need", lambda *args: None)

    def run(state, state_out=None):
        call.state = state if state_out is None else state_out
        return encoder.decay_attention_step(torch.zeros(2, 2, 4), None, None, None, state, state_out=state_out)
    return run


@pytest.mark.parametrize("apart", [False, True])
def test_a_step_counts_as_an_in_place_write(plain, step, apart):
    """A state that decay_attention keeps for its backward pass and a step then overwrites: backward
    raises, as after any in-place operation."""
    torch.manual_seed(2)
    q, k, v = (torch.randn(2, 3, 2, d, requires_grad=True) for d in (4, 4, 5))
    state, other = torch.randn(2, 2, 4, 5), torch.randn(2, 2, 4, 5)
    o = encoder._DecayAttention.apply(q, k, v, torch.tensor([-0.1, -1.0]), 0.5, None, state, False, False)[0]
    step(other, state) if apart else step(state)
    assert float(state[0, 0, 0, 0]) == 1.0
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        o.sum().backward()


def test_a_step_refuses_a_state_that_wants_a_gradient(step):
    state = torch.randn(2, 2, 4, 5, requires_grad=True)
    for call in (lambda: step(state), lambda: step(state.detach(), state)):
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
    with torch.no_grad():
        step(state)
    step(state, state.detach().clone())              # only read
    with torch.inference_mode():                      # such tensors count no versions
        step(torch.randn(2, 2, 4, 5))
