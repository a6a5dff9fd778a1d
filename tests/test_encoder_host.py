"""The encoder operators' argument checks, which need no GPU: every refused call returns
before a launch, so the pointers here are never followed.  And the references the GPU tests
use, checked against differences."""

import ctypes
import os
import re

import numpy as np
import pytest

import encoder_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, WORKSPACE, UNSUPPORTED = 0, 1, 2, 3
P, N0 = ctypes.c_void_p(0x1000), None


@pytest.fixture(scope="module")
def native():
    from semi_markov_crf_amd import _native
    return _native


def test_attention_struct_matches_header(native):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "semicrf.h")).read(), flags=re.S)
    body = re.search(r"typedef struct semicrf_attention \{(.*?)\} semicrf_attention;", text, re.S).group(1)
    names = []
    for decl in body.split(";"):
        decl = re.sub(r"^\s*(const\s+)?(void|int32_t|int64_t|float|int)\b\s*\*?", "", decl.strip())
        names += [re.sub(r"[\s*]|\[.*\]", "", n) for n in decl.split(",") if n.strip()]
    assert names == [f[0] for f in native.Attention._fields_]


def test_embed_refusals(native):
    f = native.load().semicrf_embed

    def call(tokens=P, bits=32, table=P, dtype=0, B=1, T=4, V=5, N=6, out=P):
        return f(tokens, bits, N0, table, dtype, B, T, V, N, 1.0, N0, out, N0)

    for kw in ({"tokens": N0}, {"table": N0}, {"out": N0}, {"bits": 16}, {"dtype": 2}, {"dtype": -1},
               {"B": 0}, {"T": 0}, {"V": 0}, {"N": 0}):
        assert call(**kw) == INVALID, kw
    for kw in ({"B": 1 << 15, "T": 1 << 15}, {"V": 1 << 30}):
        assert call(**kw) == UNSUPPORTED, kw


def test_embed_grad_refusals(native):
    lib = native.load()
    size = lib.semicrf_embed_grad_bytes
    need = size(0, 2, 100, 50, 8)
    assert need > 0 and need % 256 == 0
    assert size(0, 2, 200, 50, 8) > need and size(0, 2, 100, 50, 800) > need
    for bad in ((2, 2, 100, 50, 8), (0, 0, 100, 50, 8), (0, 2, 0, 50, 8), (0, 2, 100, 0, 8), (0, 2, 100, 50, 0)):
        assert size(*bad) == 0, bad

    def call(tokens=P, bits=64, g=P, ws=P, n=need, out=P, V=50):
        return lib.semicrf_embed_grad(tokens, bits, N0, g, 0, 2, 100, V, 8, 1.0, N0, ws, n, out, N0)

    assert call(tokens=N0) == call(g=N0) == call(out=N0) == call(V=0) == call(bits=8) == INVALID
    assert call(ws=N0) == call(n=need - 1) == call(ws=ctypes.c_void_p(0x1010)) == WORKSPACE


def test_layer_norm_refusals(native):
    lib = native.load()

    def call(x=P, dtype=1, wdtype=1, B=2, T=3, N=8, eps=1e-5, y=P):
        return lib.semicrf_layer_norm(x, dtype, P, P, wdtype, N0, B, T, N, eps, N0, y, N0, N0, N0)

    for kw in ({"x": N0}, {"y": N0}, {"dtype": 7}, {"dtype": 0, "wdtype": 1}, {"eps": -1.0},
               {"eps": float("nan")}, {"B": 0}, {"N": 0}):
        assert call(**kw) == INVALID, kw
    assert call(N=32769) == UNSUPPORTED
    need = lib.semicrf_layer_norm_grad_bytes(1, 2, 3, 8)
    assert need > 0 and lib.semicrf_layer_norm_grad_bytes(1, 2, 3, 32769) == 0

    def grad(g=P, mean=P, rstd=P, gx=P, ws=P, n=need):
        return lib.semicrf_layer_norm_grad(g, P, 1, P, 0, mean, rstd, N0, 2, 3, 8, N0, ws, n, gx, N0, N0, N0)

    assert grad(g=N0) == grad(mean=N0) == grad(rstd=N0) == grad(gx=N0) == INVALID
    assert grad(ws=N0) == grad(n=need - 1) == WORKSPACE


def attention(native, **kw):
    a = native.Attention()
    for n in ("q", "k", "v", "log_decay"):
        setattr(a, n, 0x1000)
    a.scale, a.dtype, a.B, a.T, a.Hq, a.Hk, a.Dk, a.Dv = 1.0, 1, 2, 3, 4, 2, 16, 16
    for n, x in kw.items():
        setattr(a, n, x)
    return a


def test_attention_refusals(native):
    lib = native.load()
    need = lib.semicrf_decay_attention_bytes(attention(native), 0)
    grad = lib.semicrf_decay_attention_bytes(attention(native), 1)
    assert 0 < need <= grad

    def fwd(a, ws=P, n=need, out=P):
        return lib.semicrf_decay_attention(a, N0, ws, n, out, N0, N0)

    def bwd(a, g=P, ws=P, n=grad, gq=P, gk=P, gv=P):
        return lib.semicrf_decay_attention_grad(a, g, N0, N0, ws, n, gq, gk, gv, N0, N0)

    for kw, want in (({"q": 0}, INVALID), ({"k": 0}, INVALID), ({"v": 0}, INVALID),
                     ({"log_decay": 0}, INVALID), ({"dtype": 3}, INVALID), ({"B": 0}, INVALID),
                     ({"T": 0}, INVALID), ({"Hq": 3}, INVALID), ({"Hk": 0}, INVALID),
                     ({"Dk": 0}, INVALID), ({"Dv": -1}, INVALID), ({"Dk": 129}, UNSUPPORTED),
                     ({"Dv": 129}, UNSUPPORTED), ({"B": 65536}, UNSUPPORTED),
                     ({"B": 60000, "T": 60000}, UNSUPPORTED)):
        assert fwd(attention(native, **kw)) == want, kw
        assert bwd(attention(native, **kw)) == want, kw
    a = attention(native)
    assert fwd(a, out=N0) == INVALID and fwd(N0) == INVALID
    assert fwd(a, ws=N0) == fwd(a, n=need - 1) == fwd(a, ws=ctypes.c_void_p(0x1008)) == WORKSPACE
    assert bwd(a, g=N0) == bwd(a, gq=N0) == bwd(a, gk=N0) == bwd(a, gv=N0) == INVALID
    assert bwd(a, ws=N0) == bwd(a, n=grad - 1) == WORKSPACE


def test_step_refusals(native):
    lib = native.load()

    def call(slots=P, pool=2, out=P, so=P, **kw):
        a = attention(native, **{"T": 1, "state": 0x1000, **kw})
        return lib.semicrf_decay_attention_step(a, slots, pool, N0, out, so)

    assert call(out=N0) == call(so=N0) == call(state=0) == call(T=2) == call(pool=0) == INVALID
    assert call(lengths=0x1000) == call(slots=N0, pool=1) == INVALID
    assert call(Dk=200) == UNSUPPORTED


def test_python_refuses_cpu_tensors():
    import torch

    import semi_markov_crf_amd as crf
    x = torch.zeros(2, 3, 8)
    for f in (lambda: crf.layer_norm(x), lambda: crf.embed(x.int()[..., 0], x[0]),
              lambda: crf.decay_attention(x[None], x[None], x[None], torch.zeros(3))):
        with pytest.raises(ValueError):
            f()


def test_reference_gradients_against_differences():
    """The 64-bit definitions that the GPU tests compare with."""
    rng = np.random.default_rng(0)
    B, T, Hq, Hk, Dk, Dv, L = 2, 6, 4, 2, 3, 5, [6, 3]
    q, k, v, do = (rng.standard_normal((B, T, h, d)) for h, d in ((Hq, Dk), (Hk, Dk), (Hk, Dv), (Hq, Dv)))
    s, ds = (rng.standard_normal((B, Hq, Dk, Dv)) for _ in range(2))
    g = np.array([0.0, -0.1, -1.0, -3.0])
    got = ref.attention_grad(do, q, k, v, g, 0.7, L, s, ds)

    def loss(x):
        o, end = ref.attention(x[0], x[1], x[2], g, 0.7, L, x[3])
        return (o * do).sum() + (end * ds).sum()

    for i in range(4):
        x = [q, k, v, s]
        D = rng.standard_normal(x[i].shape)
        up, down = ([y + t * D if j == i else y for j, y in enumerate(x)] for t in (1, -1))
        assert abs((loss(up) - loss(down)) / 2 - (got[i] * D).sum()) < 1e-10
    x, dy, w, b = rng.standard_normal((2, 3, 7)), rng.standard_normal((2, 3, 7)), rng.random(7), rng.random(7)
    _, mean, rstd = ref.layer_norm(x, w, b, 1e-5, [3, 2])
    dx, dw, db = ref.layer_norm_grad(dy, x, w, mean, rstd, [3, 2])[:3]
    D, h = rng.standard_normal(x.shape), 1e-5
    f = lambda x, w: (ref.layer_norm(x, w, b, 1e-5, [3, 2])[0] * dy).sum()  # noqa: E731
    assert abs((f(x + h * D, w) - f(x - h * D, w)) / (2 * h) - (dx * D).sum()) < 1e-7
    E = rng.standard_normal(7)
    assert abs((f(x, w + h * E) - f(x, w - h * E)) / (2 * h) - (dw * E).sum()) < 1e-7
