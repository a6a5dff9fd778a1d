"""Decayed linear attention against its 64-bit definition, as closely as its arithmetic allows.

Tolerances, fixed from the arithmetic.  u = 2^-24 and w = 2^-8 are the largest relative errors of
rounding to float32 and to bfloat16; `mag` is the sum of the absolute values of the terms that a
result adds up.
  * an fp32 sum of n terms is within n u mag of the exact one, and a decay gamma^n within 64 u (as
    in test_gpu_encoder.py);
  * in bfloat16 the masked products and the state are sums of two bfloat16 numbers when they are
    multiplied: w^2 of each term, 1.1 w^2 mag in all;
  * the output is rounded once: w |result| in bfloat16.
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
    return ((D + 2 * 64 + T // 32 + 64) * U + (1.1 * W ** 2 if typ == "bf16" else 0)) * mag + rounding(typ, want)


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
