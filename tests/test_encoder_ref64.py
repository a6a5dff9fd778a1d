"""The two 64-bit definitions of decayed linear attention against each other."""

import numpy as np

import encoder_ref as ref
import encoder_ref64 as ref64


def test_the_definitions_agree():
    rng = np.random.default_rng(3)
    B, T, Hq, Hk, Dk, Dv, L = 3, 9, 4, 2, 3, 5, np.array([9, 0, 4], np.int32)
    r = rng.standard_normal
    q, k, v, do = r((B, T, Hq, Dk)), r((B, T, Hk, Dk)), r((B, T, Hk, Dv)), r((B, T, Hq, Dv))
    g = np.array([0.0, -0.1, -3.0, -np.inf], np.float32)
    for s, ds in ((None, None), (r((B, Hq, Dk, Dv)), r((B, Hq, Dk, Dv)))):
        for a, b in zip(ref.attention(q, k, v, g, 0.7, L, s), ref64.attention(q, k, v, g, 0.7, L, s)):
            np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-12)
        for a, b in zip(ref.attention_grad(do, q, k, v, g, 0.7, L, s, ds),
                        ref64.attention_grad(do, q, k, v, g, 0.7, L, s, ds)):
            np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-12)
