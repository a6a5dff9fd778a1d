"""Decayed linear attention against its 64-bit definition, as closely as its arithmetic allows.

Tolerances, fixed from the arithmetic.  u = 2^-24 and w = 2^-8 are the largest relative errors of
rounding to float32 and to bfloat16; `mag` is the sum of the absolute values of the terms that a
result adds up.
  * an fp32 sum of n terms is within n u mag of the exact one, and a decay gamma^n within 64 u (as
    in test_gpu_encoder.py);
  * in bfloat16 the masked products and the state are sums of two bfloat16 numbers when they are
    multiplied: w^2 of each term, 1.1 w^2 mag in all;
  * the output is rounded once: w |result| in bfloat16;
  * below 2^-126 float32 is rounded to multiples of 2^-149: an output's own rounding is 2^-150 at least.
"""

import numpy as np
import pytest

import encoder_ref as ref
from test_gpu_encoder import U, W, att_inputs, close, crf, dev, opt, poison, rounding  # noqa: F401

pytestmark = pytest.mark.gpu

f32 = np.float32


def tol(typ, T, D, want, mag):
    """Of a result that is rounded to `typ`: D terms of a product, 64 positions of a chunk twice,
    a chain of chunks."""
    return ((D + 2 * 64 + T // 32 + 64) * U + (1.1 * W ** 2 if typ == "bf16" else 0)) * mag + \
        np.maximum(rounding(typ, want), 2.0 ** -150)


def check(crf, case, seed=0, g=None, scale=0.25):  # noqa: F811
    """Outputs, final state and gradients of a case (as in ATT of test_gpu_encoder.py) element by
    element, and the same bits again."""
    B, T, Hq, Hk, Dk, Dv, typ, kind, _ = case
    print(f"\n[decay_attention {case}]", flush=True)
    lengths, q, k, v, do, g0, st, gs = att_inputs(case, seed)
    g = g0 if g is None else np.asarray(g, f32)
    qd, kd, vd, dd = (dev(poison(a.copy(), lengths).astype(f32), typ) for a in (q, k, v, do))
    ln, gd = dev(lengths), dev(g)
    o, end = crf.decay_attention(qd, kd, vd, gd, scale=scale, lengths=ln, state=opt(st), want_state=True,
                                 check_status=True)
    wo, ws = ref.attention(q, k, v, g, scale, lengths, st)
    a = ref.absolute(q, k, v, st)
    mo, ms = ref.attention(a[0], a[1], a[2], g, scale, lengths, a[3])
    close(o, wo, tol(typ, T, Dk, wo, mo), "o")
    close(end, ws, tol("f32", T, 1, ws, ms), "state")
    d = crf.decay_attention_grad(dd, qd, kd, vd, gd, scale=scale, lengths=ln, state=opt(st), grad_state=opt(gs),
                                 check_status=True)
    want = ref.attention_grad(do, q, k, v, g, scale, lengths, st, gs)
    a = ref.absolute(do, q, k, v, st, gs)
    mag = ref.attention_grad(a[0], a[1], a[2], a[3], g, scale, lengths, a[4], a[5])
    for n, x, m, D in zip(("grad_q", "grad_k", "grad_v"), want, mag, (Dv, Dv, Dk)):
        close(d[n], x, tol(typ, T, D + Hq // Hk, x, m), n)
    if st is not None:
        close(d["grad_state"], want[3], tol("f32", T, 1, want[3], mag[3]), "grad_state")
    again = crf.decay_attention_grad(dd, qd, kd, vd, gd, scale=scale, lengths=ln, state=opt(st), grad_state=opt(gs))
    assert all((again[n] == d[n]).all() for n in d)


def name(c):
    return f"B{c[0]}T{c[1]}H{c[2]}_{c[3]}D{c[4]}_{c[5]}{c[6]}"


BF16 = [  # B, T, Hq, Hk, Dk, Dv, typ, lengths, initial state: every width, one token to several chunks
    (2, 1, 2, 2, 64, 64, "bf16", "full", False),
    (2, 5, 2, 1, 32, 32, "bf16", "full", False),
    (3, 100, 2, 2, 32, 32, "bf16", "ragged", True),
    (3, 190, 4, 2, 64, 64, "bf16", "ragged", True),
    (3, 140, 2, 1, 128, 128, "bf16", "ragged", True),
    (2, 150, 2, 2, 39, 17, "bf16", "ragged", True),
    (2, 130, 2, 1, 24, 16, "bf16", "ragged", False),
    (2, 200, 2, 2, 64, 100, "bf16", "ragged", True),
]


@pytest.mark.parametrize("case", BF16, ids=[name(c) for c in BF16])
def test_bfloat16_is_as_exact_as_its_outputs(crf, case):  # noqa: F811
    check(crf, case)


@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_a_long_stream_keeps_its_state(crf, typ):  # noqa: F811
    """8,000 tokens one by one: the state follows the 64-bit recurrence and the sequence form.

    A step rounds each element by at most u |s| and the decay forgets that as it forgets the rest.  In
    float32, where k v has as many bits as the state, the errors are independent: those of
    m = min(T, 1 / 2|log decay|) steps have a standard deviation of u / sqrt(3) sqrt(m) max|s|, and six
    times u sqrt(m + 1) max|s| is ten of them.  An error of the decay itself would add up in one
    direction, m times.  Products of bfloat16 numbers lie on a grid that is coarse beside an ulp of the
    state; what is rounded there is the decay's share alone, alike from step to step, so only the sum
    of all errors bounds them: u max|s| min(T, 1 / |log decay|)."""
    import torch
    B, T, H, Dk, Dv = 2, 8000, 6, 8, 12
    rng = np.random.default_rng(8)
    from test_gpu_encoder import host
    r = lambda *s: host(dev(rng.standard_normal(s).astype(f32), typ))  # noqa: E731
    q, k, v = r(B, T, H, Dk), r(B, T, H, Dk) * 0.125, r(B, T, H, Dv)
    g = np.array([-2.0 ** -13, -3.3e-4, -1e-5, -1e-6, -3e-8, -0.2], f32)
    st = (4 + rng.standard_normal((B, H, Dk, Dv))).astype(f32)
    gamma = np.exp(g.astype(np.float64))[None, :, None, None]
    s, top = st.astype(np.float64), np.abs(st).astype(np.float64)
    for t in range(T):
        s = gamma * s + k[:, t, :, :, None] * v[:, t, :, None, :]
        top = np.maximum(top, np.abs(s))
    a = np.abs(g.astype(np.float64))[None, :, None, None]
    bound = 6 * U * np.sqrt(np.minimum(T, 0.5 / a) + 1) * top if typ == "f32" else \
        U * (np.minimum(T, 1 / a) + 2) * top
    qd, kd, vd = (dev(x.astype(f32), typ) for x in (q, k, v))
    gd, state = dev(g), dev(st)
    for t in range(T):
        o = crf.decay_attention_step(qd[:, t], kd[:, t], vd[:, t], gd, state, scale=1.0)
    torch.cuda.synchronize()
    close(state, s, bound, "state")
    want, end = crf.decay_attention(qd, kd, vd, gd, scale=1.0, state=dev(st), want_state=True)
    close(end, s, bound, "state of the sequence form")
    mag = (np.abs(q[:, -1, :, :, None]) * (bound + Dk * U * np.abs(s))).sum(2)
    x = (q[:, -1, :, :, None] * s).sum(2)
    close(o, x, mag + rounding(typ, x), "last output")


def test_forward_mode_is_refused(crf):  # noqa: F811
    import torch
    import torch.autograd.forward_ad as fwd
    x = torch.randn(1, 3, 8, device="cuda")
    tok = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    g = torch.zeros(2, device="cuda")
    with fwd.dual_level():
        d = fwd.make_dual(x, torch.ones_like(x))
        h, p = (a.unflatten(-1, (2, 4)) for a in (d, x))
        dg = fwd.make_dual(g, torch.ones_like(g))
        for err, f in ((RuntimeError, lambda: crf.embed(tok, d[0])), (RuntimeError, lambda: crf.layer_norm(d)),
                       (RuntimeError, lambda: crf.decay_attention(p, h, p, g)),
                       (ValueError, lambda: crf.decay_attention(p, p, p, dg))):
            with pytest.raises(err):
                f()
        crf.layer_norm(x)
        crf.decay_attention(p, p, p, g)


def test_a_step_counts_as_an_in_place_write(crf):  # noqa: F811
    import torch
    torch.manual_seed(2)
    q, k, v = (torch.randn(2, 3, 2, 8, device="cuda", requires_grad=True) for _ in range(3))
    g, state = torch.tensor([-0.1, -1.0], device="cuda"), torch.randn(2, 2, 8, 8, device="cuda")
    o = crf.decay_attention(q, k, v, g, state=state)
    one = [x[:, 0].detach() for x in (q, k, v)]
    crf.decay_attention_step(*one, g, state.clone())
    crf.decay_attention_step(*one, g, state)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        o.sum().backward()
    state.requires_grad_()
    with pytest.raises(ValueError):
        crf.decay_attention_step(*one, g, state)
    with torch.inference_mode():
        crf.decay_attention_step(*one, g, torch.zeros(2, 2, 8, 8, device="cuda"))
    torch.cuda.synchronize()


def segments(crf, B, T, Hq, Hk, Dk, Dv, typ, grad=False):  # noqa: F811
    """Segments that a call is cut into, from the states that its workspace holds."""
    a = crf._native.Attention()
    a.dtype, a.B, a.T, a.Hq, a.Hk, a.Dk, a.Dv = int(typ == "bf16"), B, T, Hq, Hk, Dk, Dv
    n = crf._native.load().semicrf_decay_attention_bytes(a, int(grad))
    if grad and Hq > Hk:
        n -= sum(-(-B * T * Hq * 4 * D // 256) * 256 for D in (Dk, Dv))
    return max(1, n // (1 + grad) // (B * Hq * Dk * Dv * 4))


def test_segments_join_without_drift(crf):  # noqa: F811
    """A state that only decays, over a hundred segments and more: every join rounds it once, errors of
    independent sign (as in test_a_long_stream_keeps_its_state), and exp(log decay * segment) adds
    nothing of one sign.  grad_state is the same sum backward."""
    import torch
    B, T, H, D = 1, 100_000, 8, 16
    rng = np.random.default_rng(11)
    n = min(segments(crf, B, T, H, H, D, D, "f32", grad) for grad in (False, True))
    assert n >= 40
    g = -np.exp2(rng.uniform(-24, -17, H)).astype(f32)
    st = rng.standard_normal((B, H, D, D)).astype(f32)
    want = st * np.exp(g.astype(np.float64) * T)[None, :, None, None]
    bound = 6 * U * np.sqrt(max(segments(crf, B, T, H, H, D, D, "f32", x) for x in (False, True)) + 1)
    zero = torch.zeros(B, T, H, D, device="cuda")
    _, end = crf.decay_attention(zero, zero, zero, dev(g), state=dev(st), want_state=True)
    close(end, want, bound * np.abs(want), "state")
    d = crf.decay_attention_grad(zero, zero, zero, zero, dev(g), state=dev(st), grad_state=dev(st))
    close(d["grad_state"], want, bound * np.abs(want), "grad_state")


def test_float32_rounds_a_long_memory_once_a_chunk(crf):  # noqa: F811
    """Time constants of 8,192 positions, where the state is the sum of many chunks.  Rounding a number
    gives a relative error of 0.42 u on average (u / sqrt(3), less over a binade).  If each chunk of 32
    rounds the state once, what the decay leaves of the errors is 0.42 u sqrt(8192 / 64) = 4.7 u of it;
    joins of segments add 1.5 u, a product of 64 terms 2.4 u, weights about 1 u: 5.6 u in all, of the
    result as of the state.  9 u is half as much again; one rounding for every product of a chunk
    would give 14 u and more."""
    from test_gpu_encoder import host
    B, T, H, D = 1, 20_000, 2, 64
    rng = np.random.default_rng(13)
    q, k, v, do = (host(dev(rng.standard_normal((B, T, H, D)).astype(f32))) for _ in range(4))
    g = np.array([-2.0 ** -13, -1.25 * 2.0 ** -13], f32)
    a = [dev(x.astype(f32)) for x in (q, k, v)] + [dev(g)]
    got = {"out": crf.decay_attention(*a, scale=1.0), **crf.decay_attention_grad(dev(do.astype(f32)), *a, scale=1.0)}
    want = dict(zip(("grad_q", "grad_k", "grad_v"), ref.attention_grad(do, q, k, v, g, 1.0, [T])))
    want["out"] = ref.attention(q, k, v, g, 1.0, [T])[0]
    for n, x in want.items():
        off = np.linalg.norm(host(got[n]) - x) / np.linalg.norm(x)
        print(f"{n}: {off / U:.2f} u", flush=True)
        assert off <= 9 * U, (n, off / U)


# rows that fill the padded width, cut into segments of several chunks: B, T, Hq, Hk, D, typ
LONG = [
    (2, 9000, 4, 2, 64, "f32"), (2, 9000, 4, 2, 64, "bf16"),
    (2, 9000, 4, 2, 32, "f32"), (2, 9000, 4, 2, 32, "bf16"),
    (2, 9000, 2, 1, 128, "f32"), (2, 9000, 2, 1, 128, "bf16"),
    (1, 9000, 4, 4, 64, "bf16"), (1, 9000, 8, 1, 64, "bf16"),
]


@pytest.mark.parametrize("case", LONG, ids=[f"B{c[0]}T{c[1]}H{c[2]}_{c[3]}D{c[4]}{c[5]}" for c in LONG])
def test_segments_of_several_chunks(crf, case):  # noqa: F811
    """Slow heads among them one that keeps everything, ragged lengths, initial and final states.
    Element by element within `tol`; and the norm of all errors of an array, which a lost part of the
    state or of the masked products would raise, although sums over thousands of positions leave
    `tol` wide:
      * rounding to bfloat16 gives 0.42 w of the result on average (w / sqrt(3), less over a binade);
        5 % more leave room for a third of it besides;
      * in float32, 9 u as in test_float32_rounds_a_long_memory_once_a_chunk.  A head without decay rounds
        its growing state T / 32 times, the same as 140 times at its final size: 5 u; a product of 128
        terms 3.4 u; joins and weights 1.8 u: 6.3 u in all."""
    import encoder_ref64 as ref64
    from test_gpu_encoder import host
    B, T, Hq, Hk, D, typ = case
    for grad in (False, True):
        n, C = segments(crf, B, T, Hq, Hk, D, D, typ, grad), 64 if typ == "bf16" else 32
        print(f"\n[decay_attention {case}: {n} segments]", flush=True)
        assert n >= 4 and -(-T // C) / n > 2
    rng = np.random.default_rng(T + D)
    r = lambda *s: host(dev(rng.standard_normal(s).astype(f32), typ))  # noqa: E731
    q, k, v, do = r(B, T, Hq, D), r(B, T, Hk, D), r(B, T, Hk, D), r(B, T, Hq, D)
    g = np.resize(np.array([0.0, -2.0 ** -12, -2.0 ** -6, -0.5], f32), Hq)
    st, gs = (rng.standard_normal((B, Hq, D, D)).astype(f32) for _ in range(2))
    lengths = np.array([T, T * 2 // 3 + 7], np.int32)[:B]
    scale, ln = 0.25, dev(lengths)
    a = [dev(poison(x.copy(), lengths).astype(f32), typ) for x in (q, k, v)] + [dev(g)]
    got = dict(zip(("o", "state"), crf.decay_attention(*a, scale=scale, lengths=ln, state=dev(st), want_state=True)))
    want = dict(zip(got, ref64.attention(q, k, v, g, scale, lengths, st, "cuda")))
    p = ref.absolute(do, q, k, v, st, gs)
    mag = dict(zip(got, ref64.attention(p[1], p[2], p[3], g, scale, lengths, p[4], "cuda")))
    got.update(crf.decay_attention_grad(dev(poison(do.copy(), lengths).astype(f32), typ), *a, scale=scale, lengths=ln,
                                        state=dev(st), grad_state=dev(gs)))
    grads = ("grad_q", "grad_k", "grad_v", "grad_state")
    want.update(zip(grads, ref64.attention_grad(do, q, k, v, g, scale, lengths, st, gs, "cuda")))
    mag.update(zip(grads, ref64.attention_grad(p[0], p[1], p[2], p[3], g, scale, lengths, p[4], p[5], "cuda")))
    for n, x in want.items():
        t = "f32" if "state" in n else typ
        off = np.linalg.norm(host(got[n]) - x) / np.linalg.norm(x)
        print(f"{n}: {off / (W if t == 'bf16' else U):.2f} of its unit", flush=True)
        close(got[n], x, tol(t, T, D + Hq // Hk, x, mag[n]), n)
        if t == typ:
            assert off <= (1.05 * 0.425 * W if t == "bf16" else 9 * U), (n, off)


STRONG = [(2, 200, 6, 6, 32, 32, "bf16", "ragged", True), (2, 150, 6, 3, 64, 64, "bf16", "full", True),
          (2, 70, 6, 6, 128, 128, "bf16", "ragged", True), (2, 200, 6, 3, 39, 20, "bf16", "full", True),
          (2, 150, 6, 6, 64, 64, "f32", "full", True)]


@pytest.mark.parametrize("case", STRONG, ids=[name(c) for c in STRONG])
def test_strong_decays(crf, case):  # noqa: F811
    """gamma from 0 and e^-80 to 1.  The gradient of the initial state is of order gamma, down to 10^-35,
    and as exact as any: the low parts of what is added to it must not underflow."""
    check(crf, case, g=[-np.inf, -80.0, -30.0, -12.0, -1e-6, 0.0])


SHARED = [(2, 200, 16, 1, 128, 128, "bf16", "ragged", True), (2, 100, 16, 1, 64, 64, "f32", "ragged", True),
          (2, 130, 33, 1, 64, 64, "bf16", "full", True), (2, 90, 12, 1, 128, 100, "f32", "full", False),
          (1, 1500, 34, 2, 32, 32, "bf16", "full", True)]


@pytest.mark.parametrize("case", SHARED, ids=[name(c) for c in SHARED])
def test_many_query_heads_on_one(crf, case):  # noqa: F811
    check(crf, case)
