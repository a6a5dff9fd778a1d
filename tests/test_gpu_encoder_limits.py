"""The encoder operators at the largest sizes that their interface accepts: what a single launch
does not hold."""

import pytest

from test_gpu_encoder import U, crf  # noqa: F401

pytestmark = pytest.mark.gpu


def test_embed_of_more_rows_than_a_launch_has_threads(crf):  # noqa: F811
    """2^27 + 5 rows of 264 bfloat16, 32 threads each: 2^32 threads and more, 71 GB of output."""
    import torch
    n, N, V = 2 ** 27 + 5, 264, 7
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    print(f"\n[embed n={n} N={N}]", flush=True)
    tok = (torch.arange(n, device="cuda", dtype=torch.int32) % V).view(1, n)
    table = torch.randn(V, N, device="cuda").bfloat16()
    y = crf.embed(tok, table)
    for rows in (slice(0, 300), slice(n // 2, n // 2 + 300), slice(n - 300, n)):
        assert torch.equal(y[0, rows], table[tok[0, rows].long()])


def test_embed_grad_of_the_widest_rows(crf):  # noqa: F811
    """300 rows of 2^23 - 3 bfloat16 into two: as many column slabs as a grid takes, and a run over
    two chunks.  Sums of small whole numbers are exact."""
    import torch
    n, N, V = 300, 2 ** 23 - 3, 3
    print(f"\n[embed_grad n={n} N={N}]", flush=True)
    tok = torch.zeros(1, n, dtype=torch.int32, device="cuda")
    tok[0, -4:] = 2
    g = (torch.arange(N, device="cuda") % 2).to(torch.bfloat16)[None, None].expand(1, n, N).contiguous()
    d = crf.embed_grad(tok, g, V)
    assert torch.equal(d, torch.tensor([n - 4, 0, 4], device="cuda", dtype=torch.bfloat16)[:, None] * g[0, :1])


def test_attention_of_more_heads_than_a_launch_has_threads(crf):  # noqa: F811
    """65,535 sequences of one position, 129 query heads on one: 8.5 million workgroups of 512 threads,
    three times as many for the gradients.  One position alone is o = scale (q k) v."""
    import torch
    B, H, D, scale = 65535, 129, 66, 0.5
    torch.manual_seed(3)
    print(f"\n[decay_attention B={B} H={H} D={D}]", flush=True)
    q, do = (torch.randn(B, 1, H, D, device="cuda").bfloat16() for _ in range(2))
    k, v = (torch.randn(B, 1, 1, D, device="cuda").bfloat16() for _ in range(2))
    g = torch.full((H,), -0.1, device="cuda")
    w = 2.0 ** -8

    def near(got, a, b, c, what, sums=False):
        """got = scale (a . b) c; with sums, over the heads: errors of test_gpu_decay_attention.py."""
        a, b, c = (x.float() for x in (a, b, c))
        want, mag = scale * (a * b).sum(-1, keepdim=True) * c, scale * (a * b).abs().sum(-1, keepdim=True) * c.abs()
        if sums:
            want, mag = want.sum(2, keepdim=True), mag.sum(2, keepdim=True)
        off = (got.float() - want).abs() - w * want.abs() - (1.1 * w * w + (D + H + 400) * U) * mag
        assert float(off.max()) <= 0 and bool(torch.isfinite(got).all()), what

    near(crf.decay_attention(q, k, v, g, scale=scale), q, k, v, "o")
    d = crf.decay_attention_grad(do, q, k, v, g, scale=scale)
    near(d["grad_q"], do, v, k, "grad_q")
    near(d["grad_k"], do, v, q, "grad_k", True)
    near(d["grad_v"], q, k, do, "grad_v", True)


def test_sum_over_more_shared_heads_than_a_launch_has_threads(crf):  # noqa: F811
    """2^26 + 64 positions with two query heads on one of 128 value columns: the sum over the heads
    takes 2^31 threads and more.  Heads that forget at once leave dv = sum over heads scale (q k) do."""
    import torch
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 170 << 30:
        pytest.skip("needs 170 GB")
    B, T, D = 64, 2 ** 20 + 1, 128
    torch.manual_seed(4)
    print(f"\n[decay_attention_grad B={B} T={T}]", flush=True)
    q, k = (torch.randn(B, T, h, 1, device="cuda").bfloat16() for h in (2, 1))
    do, v = (torch.zeros(B, T, h, D, device="cuda", dtype=torch.bfloat16) for h in (2, 1))
    rows = [(0, slice(0, 99)), (31, slice(T - 99, T)), (63, slice(T // 2, T // 2 + 99)), (63, slice(T - 99, T))]
    for b, t in rows:
        do[b, t].normal_()
    g = torch.full((2,), -float("inf"), device="cuda")
    d = crf.decay_attention_grad(do, q, k, v, g, scale=0.5)["grad_v"]
    w = 2.0 ** -8
    for b, t in rows:
        terms = 0.5 * q[b, t].float() * k[b, t].float() * do[b, t].float()
        want, mag = terms.sum(1, keepdim=True), terms.abs().sum(1, keepdim=True)
        off = (d[b, t].float() - want).abs() - w * want.abs() - (1.1 * w * w + 300 * U) * mag
        assert float(off.max()) <= 0, (b, t)
    assert int(torch.count_nonzero(d[:, 200:T // 2 - 200])) == 0
