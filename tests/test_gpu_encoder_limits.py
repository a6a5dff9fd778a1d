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
