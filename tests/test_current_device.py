"""Calls on arrays of a GPU that is not the current one: the library must run with theirs current,
since a default stream is a null handle that stands for the current GPU's.  The library and the
devices are stand-ins here, the binding is the package's own."""

import contextlib
import types

import pytest
import torch

import semi_markov_crf_amd as crf
from semi_markov_crf_amd import _native, encoder

WHERE = 1                                                # the arrays' GPU; 0 is current


class Array(torch.Tensor):
    """A CPU tensor that says it lies on GPU 1."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", WHERE))

    def get_device(self):
        return WHERE


def array(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Array)


@pytest.fixture
def calls(monkeypatch):
    """(function, current device) of every call of the library."""
    now, seen = [0], []

    class Lib:
        def __getattr__(self, name):
            def f(*args):
                seen.append((name, now[0]))
                return 1 << 12 if name.endswith("_bytes") else 0
            return f

    @contextlib.contextmanager
    def device(index):
        before, now[0] = now[0], torch.device("cuda", index).index
        yield
        now[0] = before

    def on_host(make):
        return lambda *a, device=None, **kw: make(*a, **kw).as_subclass(Array)

    lib = Lib()
    monkeypatch.setattr(_native, "load", lambda: lib)
    monkeypatch.setattr(_native, "_lib", lib)
    monkeypatch.setattr(_native, "_current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(encoder, "_raw_stream", lambda index: 0)
    for make in ("empty", "zeros"):
        monkeypatch.setattr(torch, make, on_host(getattr(torch, make)))
    yield seen
    assert now[0] == 0                                   # and the caller's device is current again


def only_there(seen, names):
    """Every call that launches ran on the arrays' GPU."""
    ran = [c for c in seen if not c[0].endswith("_bytes")]
    assert ran == [(n, WHERE) for n in names]


def test_encoder_operators(calls):
    tok, table, x = array(2, 3, dtype=torch.int32), array(5, 8), array(2, 3, 8)
    q, g, state, m = array(2, 3, 2, 4), array(2), array(2, 2, 4, 4), array(2, 3)
    ws = torch.empty(1 << 13, dtype=torch.uint8)
    ws = ws[-ws.data_ptr() % 256:]
    with torch.no_grad():
        crf.embed(tok, table)
        crf.embed_grad(tok, x, 5, workspace=ws)
        crf.layer_norm(x)
        crf.layer_norm_grad(x, x, None, m, m, workspace=ws)
        crf.decay_attention(q, q, q, g, workspace=ws)
        crf.decay_attention_grad(q, q, q, q, g, workspace=ws)
        crf.decay_attention_step(q[:, 0], q[:, 0], q[:, 0], g, state)
    only_there(calls, ["semicrf_embed", "semicrf_embed_grad", "semicrf_layer_norm", "semicrf_layer_norm_grad",
                       "semicrf_decay_attention", "semicrf_decay_attention_grad", "semicrf_decay_attention_step"])


def test_crf(calls):
    em, lengths, trans, dur = array(2, 3, 4), array(2, dtype=torch.int32), array(4, 4), array(5, 4)
    gold, seg = array(2, 3, dtype=torch.int32), array(2, 3, dtype=torch.uint8)
    ws = torch.empty(1 << 13, dtype=torch.uint8)
    ws = ws[-ws.data_ptr() % 256:]
    with torch.no_grad():
        crf.prefix(em, lengths, workspace=ws)
        crf.logz(em, lengths, trans, dur, workspace=ws, check_status=True)
        crf.backward(em, lengths, trans, dur, workspace=ws)
        crf.nll(em, lengths, trans, dur, gold, seg, workspace=ws)
        crf.viterbi(em, lengths, trans, dur, workspace=ws)
    only_there(calls, ["semicrf_prefix", "semicrf_logz_ex", "semicrf_read_status", "semicrf_backward_ex",
                       "semicrf_nll", "semicrf_viterbi_ex"])


def test_the_current_device_stays_where_it_is(monkeypatch):
    """No switch where the arrays' GPU is current."""
    monkeypatch.setattr(_native, "_lib", types.SimpleNamespace(f=lambda *a: a))
    monkeypatch.setattr(_native, "_current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda index: pytest.fail("switched"))
    assert _native.call(0, "f", 3, 4) == (3, 4)
