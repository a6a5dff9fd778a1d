"""The token loss writes to its workspace and nowhere else, with a table that it reads where it lies or copies."""

import pytest

from test_gpu_encoder import crf  # noqa: F401

pytestmark = pytest.mark.gpu

CASES = [(2, 70, 64, 300, "f32"), (2, 70, 64, 300, "bf16"), (1, 300, 128, 1000, "bf16"), (1, 300, 100, 513, "bf16"),
         (1, 600, 256, 4097, "f32")]


@pytest.mark.parametrize("offset", [0, 1, 8])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_workspace_of_the_size_asked_for(crf, case, offset):  # noqa: F811
    import torch
    from semi_markov_crf_amd import _native
    B, T, N, V, typ = case
    dt = torch.float32 if typ == "f32" else torch.bfloat16
    print(f"\n[token_nll workspace {case} table at {offset}]", flush=True)
    torch.manual_seed(T + N)
    x = torch.randn(B, T, N, device="cuda").to(dt)
    table = torch.empty(V * N + offset, device="cuda", dtype=dt)[offset:].view(V, N)
    table.copy_(torch.randn(V, N, device="cuda") * N ** -0.5)
    t, g = torch.randint(-50, V, (B, T), device="cuda"), torch.rand(B, T, device="cuda")
    aligned = table.clone()
    want, lse = crf.token_nll(x, aligned, t, want_lse=True)
    d = crf.token_nll_grad(g, x, aligned, t, lse)
    ws = {}
    for grad in (0, 1):
        n = _native.load().semicrf_token_nll_table_bytes(_native.F32 if typ == "f32" else _native.BF16, B, T, V, N,
                                                         table.data_ptr(), grad)
        room = torch.full((n + 8192,), 0xa5, dtype=torch.uint8, device="cuda")
        at = 4096 - room.data_ptr() % 256
        ws[grad] = room[at:at + n], room[:at], room[at + n:]
    assert torch.equal(crf.token_nll(x, table, t, workspace=ws[0][0]), want)
    e = crf.token_nll_grad(g, x, table, t, lse, workspace=ws[1][0])
    assert all(torch.equal(d[k], e[k]) for k in d)
    for _, before, after in ws.values():
        assert bool((before == 0xa5).all()) and bool((after == 0xa5).all())
    with pytest.raises(ValueError):
        crf.token_nll(x, table, t, workspace=ws[0][0][:-256])
