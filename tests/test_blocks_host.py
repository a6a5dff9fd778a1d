"""The block operators' argument checks, which need no GPU: every refused call returns before a
launch, so the pointers here are never followed.  And the references the GPU tests use, checked
against differences."""

import ctypes
import os
import re

import numpy as np
import pytest

import blocks_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, WORKSPACE, UNSUPPORTED = 1, 2, 3
P, N0 = ctypes.c_void_p(0x1000), None


@pytest.fixture(scope="module")
def native():
    from semi_markov_crf_amd import _native
    return _native


@pytest.mark.parametrize("name", ["recurrence", "residual"])
def test_structs_match_header(native, name):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "semicrf.h")).read(), flags=re.S)
    body = re.search(r"typedef struct semicrf_%s \{(.*?)\} semicrf_%s;" % (name, name), text, re.S).group(1)
    names = []
    for decl in body.split(";"):
        decl = re.sub(r"^\s*(const\s+)?(void|int32_t|int64_t|float|int)\b\s*\*?", "", decl.strip())
        names += [re.sub(r"[\s*]|\[.*\]", "", n) for n in decl.split(",") if n.strip()]
    assert names == [f[0] for f in getattr(native, name.capitalize())._fields_]


def test_span_matches_header(native):
    text = open(os.path.join(ROOT, "include", "semicrf.h")).read()
    assert int(re.search(r"#define SEMICRF_RECURRENCE_SPAN (\d+)", text).group(1)) == native.RECURRENCE_SPAN


def recurrence(native, **kw):
    a = native.Recurrence()
    for n in ("x", "decay_gate", "input_gate", "log_decay"):
        setattr(a, n, 0x1000)
    a.dtype, a.B, a.T, a.N = 1, 2, 3, 16
    for n, x in kw.items():
        setattr(a, n, x)
    return a


def test_recurrence_refusals(native):
    lib = native.load()
    size = lib.semicrf_gated_recurrence_bytes
    need, grad = size(recurrence(native), 0), size(recurrence(native), 1)
    assert need > 0 and grad > 0 and need % 256 == grad % 256 == 0

    def fwd(a, ws=P, n=need, out=P):
        return lib.semicrf_gated_recurrence(a, N0, ws, n, out, N0, N0, N0)

    def bwd(a, starts=P, g=P, ws=P, n=grad, gx=P, gr=P, gi=P):
        return lib.semicrf_gated_recurrence_grad(a, starts, g, N0, N0, ws, n, gx, gr, gi, N0, N0, N0)

    for kw, want in (({"x": 0}, INVALID), ({"decay_gate": 0}, INVALID), ({"input_gate": 0}, INVALID),
                     ({"log_decay": 0}, INVALID), ({"dtype": 3}, INVALID), ({"B": 0}, INVALID), ({"T": 0}, INVALID),
                     ({"N": 0}, INVALID), ({"N": (1 << 20) + 1}, UNSUPPORTED), ({"B": 65536}, UNSUPPORTED),
                     ({"B": 60000, "T": 60000}, UNSUPPORTED)):
        assert fwd(recurrence(native, **kw)) == bwd(recurrence(native, **kw)) == want, kw
        if not any(k in kw for k in ("x", "decay_gate", "input_gate", "log_decay")):
            assert size(recurrence(native, **kw), 0) == size(recurrence(native, **kw), 1) == 0
    for kw in ({"B": 65535, "N": 64 * 65}, {"x_stride": native.Strides2(0, 1 << 25)},
               {"input_stride": native.Strides2(0, -1)}):
        assert fwd(recurrence(native, **kw)) == bwd(recurrence(native, **kw)) == UNSUPPORTED, kw
        assert size(recurrence(native, **kw), 0) == 0
    assert size(recurrence(native, T=1, x_stride=native.Strides2(0, 1 << 40)), 0) > 0
    a = recurrence(native)
    assert fwd(a, out=N0) == fwd(N0) == bwd(N0) == INVALID
    assert fwd(a, ws=N0) == fwd(a, n=need - 1) == fwd(a, ws=ctypes.c_void_p(0x1008)) == WORKSPACE
    assert bwd(a, starts=N0) == bwd(a, g=N0) == bwd(a, gx=N0) == bwd(a, gr=N0) == bwd(a, gi=N0) == INVALID
    assert bwd(a, ws=N0) == bwd(a, n=grad - 1) == WORKSPACE


def test_recurrence_step_refusals(native):
    lib = native.load()

    def call(slots=P, pool=2, out=P, so=P, **kw):
        a = recurrence(native, **{"T": 1, "state": 0x1000, **kw})
        return lib.semicrf_gated_recurrence_step(a, slots, pool, N0, out, so)

    assert call(out=N0) == call(so=N0) == call(state=0) == call(T=2) == call(pool=0) == INVALID
    assert call(lengths=0x1000) == call(slots=N0, pool=1) == INVALID
    assert call(N=(1 << 20) + 1) == UNSUPPORTED


def residual(native, **kw):
    a = native.Residual()
    a.x = a.branch = 0x1000
    a.eps, a.dtype, a.wdtype, a.B, a.T, a.N = 1e-5, 1, 0, 2, 3, 16
    for n, x in kw.items():
        setattr(a, n, x)
    return a


def test_residual_refusals(native):
    lib = native.load()
    need = lib.semicrf_residual_norm_grad_bytes(1, 2, 3, 16)
    assert need > 0
    for bad in ((2, 2, 3, 16), (1, 0, 3, 16), (1, 2, 0, 16), (1, 2, 3, 0), (1, 2, 3, 16385)):
        assert lib.semicrf_residual_norm_grad_bytes(*bad) == 0

    def fwd(a, r=P, y=P):
        return lib.semicrf_residual_norm(a, N0, r, y, N0, N0)

    def bwd(a, stats=P, ws=P, n=need, gx=P, gb=P, gg=P):
        return lib.semicrf_residual_norm_grad(a, stats, P, P, N0, ws, n, gx, gb, gg, N0, N0)

    for kw, want in (({"x": 0}, INVALID), ({"branch": 0}, INVALID), ({"eps": -1.0}, INVALID),
                     ({"eps": float("nan")}, INVALID), ({"dtype": 2}, INVALID), ({"dtype": 0, "wdtype": 1}, INVALID),
                     ({"B": 0}, INVALID), ({"N": 16385}, UNSUPPORTED), ({"B": 1 << 15, "T": 1 << 15}, UNSUPPORTED)):
        assert fwd(residual(native, **kw)) == bwd(residual(native, **kw)) == want, kw
    a = residual(native)
    assert fwd(N0) == fwd(a, r=N0) == fwd(a, y=N0) == bwd(a, stats=N0) == bwd(a, gx=N0) == bwd(a, gb=N0) == INVALID
    assert bwd(residual(native, gate=0x1000), gg=N0) == INVALID
    assert bwd(a, ws=N0) == bwd(a, n=need - 1) == WORKSPACE


def test_token_nll_refusals(native):
    lib = native.load()
    size = lib.semicrf_token_nll_bytes
    need, grad = size(1, 2, 3, 50, 16, 0), size(1, 2, 3, 50, 16, 1)
    assert 0 < need < grad
    assert size(1, 2, 3000, 50, 16, 1) > grad and size(0, 2, 3, 50, 16, 0) > 0
    for bad in ((2, 2, 3, 50, 16), (1, 0, 3, 50, 16), (1, 2, 3, 0, 16), (1, 2, 3, 50, 0), (1, 2, 3, 50, 32769),
                (1, 2, 3, (1 << 22) + 1, 16), (1, 1 << 11, (1 << 11) + 1, 50, 16),
                (1, 1 << 11, 1 << 11, 1 << 22, 8192)):
        assert size(*bad, 0) == size(*bad, 1) == 0, bad

    def fwd(x=P, w=P, dtype=1, t=P, bits=32, B=2, T=3, V=50, N=16, scale=1.0, ws=P, n=need, loss=P):
        return lib.semicrf_token_nll(x, w, dtype, t, bits, N0, B, T, V, N, scale, N0, ws, n, loss, N0, N0)

    def bwd(x=P, w=P, dtype=1, t=P, bits=32, B=2, T=3, V=50, N=16, scale=1.0, ws=P, n=grad, g=P, lse=P, gx=P, gw=P):
        return lib.semicrf_token_nll_grad(g, x, w, dtype, t, bits, N0, lse, B, T, V, N, scale, N0, ws, n, gx, gw, N0)

    for f in (fwd, bwd):
        for kw in ({"x": N0}, {"w": N0}, {"t": N0}, {"bits": 16}, {"dtype": 5}, {"B": 0}, {"V": 0},
                   {"scale": float("nan")}, {"scale": float("inf")}):
            assert f(**kw) == INVALID, kw
        for kw in ({"N": 32769}, {"V": (1 << 22) + 1}, {"B": 1 << 11, "T": (1 << 11) + 1}):
            assert f(**kw) == UNSUPPORTED, kw
        assert f(ws=N0) == f(n=need - 1) == f(ws=ctypes.c_void_p(0x1010)) == WORKSPACE
    assert fwd(loss=N0) == bwd(g=N0) == bwd(lse=N0) == bwd(gx=N0, gw=N0) == INVALID


def test_python_refuses_cpu_tensors():
    import torch

    import semi_markov_crf_amd as crf
    x = torch.zeros(2, 3, 8)
    for f in (lambda: crf.gated_recurrence(x, x, x, x[0, 0]), lambda: crf.residual_norm(x, x),
              lambda: crf.token_nll(x, x[0], x[..., 0].int()),
              lambda: crf.gated_recurrence_step(x[0], x[0], x[0], x[0, 0], x[0])):
        with pytest.raises(ValueError):
            f()


def test_reference_gradients_against_differences():
    """The 64-bit definitions that the GPU tests compare with."""
    rng = np.random.default_rng(0)
    B, T, N, L = 2, 6, 3, [6, 3]
    x, r, i, g = (rng.standard_normal((B, T, N)) for _ in range(4))
    lam, s, gs = -rng.random(N) - 0.1, rng.standard_normal((B, N)), rng.standard_normal((B, N))
    got = ref.recurrence_grad(g, x, r, i, lam, L, s, gs)[0]
    args, step = [x, r, i, lam, s], 1e-6

    def loss(a):
        h, end = ref.recurrence(*a[:4], L, a[4])[:2]
        return (h * g).sum() + (end * gs).sum()

    def slope(f, a, k, D):
        ends = [f([v + t * step * D if j == k else v for j, v in enumerate(a)]) for t in (1, -1)]
        return (ends[0] - ends[1]) / (2 * step)

    for k, name in enumerate(("x", "decay_gate", "input_gate", "log_decay", "state")):
        D = rng.standard_normal(args[k].shape)
        assert abs(slope(loss, args, k, D) - (got[name] * D).sum()) < 1e-7, name

    names = ["x", "branch", "weight", "bias", "gate", "scale", "branch_weight", "branch_bias"]
    a = [rng.standard_normal((4, 7)) if n in ("x", "branch", "gate") else rng.random(7) + 0.5 for n in names]
    gr, gy = rng.standard_normal((2, 4, 7))
    for center in (True, False):
        def f(v):
            x, o, w, b, z, c, p, q = v
            return ref.residual(x, o, w, b, z, c, True, p, q, center, 1e-5, gr, gy)[0]

        d = f(a)
        for k, name in enumerate(names):
            D = rng.standard_normal(a[k].shape)
            got = slope(lambda v: (f(v)["r"] * gr).sum() + (f(v)["y"] * gy).sum(), a, k, D)
            assert abs(got - (d["grad_" + name] * D).sum()) < 1e-7, (center, name)

    x, w, t, g = rng.standard_normal((5, 4)), rng.standard_normal((9, 4)), rng.integers(0, 9, 5), rng.random(5)
    dx, dw = ref.nll(x, w, t, 0.7, lambda n: n, 1.0, g)[4:6]
    for k, d in enumerate((dx, dw)):
        D = rng.standard_normal(d.shape)
        got = slope(lambda v: (ref.nll(v[0], v[1], t, 0.7, lambda n: n, 1.0)[0] * g).sum(), [x, w], k, D)
        assert abs(got - (d * D).sum()) < 1e-7
