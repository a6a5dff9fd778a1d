"""Gated recurrence, residual norm and token loss where offsets pass 32 bits, at the borders of their
tiles, with a workspace of the caller's and captured with their gradients."""

import numpy as np
import pytest

import blocks_ref as ref
from test_gpu_blocks import decays, dev, near, put, values
from test_gpu_encoder import crf  # noqa: F401

pytestmark = pytest.mark.gpu


def room(gigabytes):
    import torch
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip(f"needs {gigabytes} GB")


def test_recurrence_past_32_bits(crf):  # noqa: F811
    """1.3 * 10^9 elements a sequence, three of them: the same bits as the last sequence by itself, whose
    tiles of channels are as many that the gradient takes them in the same way (each by one workgroup; fewer are
    cut along T, whose joins round otherwise)."""
    import torch
    room(130)
    B, T, N = 3, 26_000, 49_152
    print(f"\n[gated_recurrence B={B} T={T} N={N}]", flush=True)
    torch.manual_seed(5)
    x, r, i = (torch.randn(B, T, N, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    ld = dev(decays(N, "spread"))
    h, starts = crf.gated_recurrence(x, r, i, ld, want_starts=True)
    d = crf.gated_recurrence_grad(x, x, r, i, ld, starts)
    part = [v[-1:].contiguous() for v in (x, r, i)]
    want, some = crf.gated_recurrence(*part, ld, want_starts=True)
    assert torch.equal(h[-1:], want) and torch.equal(starts[-1:], some)
    e = crf.gated_recurrence_grad(part[0], *part, ld, some)
    for name in ("grad_x", "grad_decay_gate", "grad_input_gate"):
        assert torch.equal(d[name][-1:], e[name]), name
    del d, h, e, want, part
    views = [torch.empty(2, 2 ** 26 + 70, 64, device="cuda", dtype=torch.bfloat16)[:, -70:] for _ in range(3)]
    for v in views:                                          # sequences more than 2^32 elements apart
        v.copy_(torch.randn(2, 70, 64, device="cuda"))
    got = crf.gated_recurrence(*views, ld[:64].contiguous())
    assert torch.equal(got, crf.gated_recurrence(*(v.contiguous() for v in views), ld[:64].contiguous()))


def test_recurrence_of_rows_far_apart(crf):  # noqa: F811
    """Positions 2^25 - 1 elements apart, the most that is taken: 300 of them span 20 GB."""
    import torch
    room(70)
    T, N = 300, 40
    print(f"\n[gated_recurrence rows far apart T={T}]", flush=True)
    far = torch.empty(T * (2 ** 25 - 1), device="cuda", dtype=torch.bfloat16).view(1, T, -1)[..., -N:]
    far.copy_(torch.randn(1, T, N, device="cuda"))
    ld = dev(decays(N, "spread"))
    near_by = far.contiguous()
    h, starts = crf.gated_recurrence(far, near_by, far, ld, want_starts=True)
    assert torch.equal(h, crf.gated_recurrence(near_by, near_by, near_by, ld))
    d = crf.gated_recurrence_grad(h, far, near_by, far, ld, starts)
    e = crf.gated_recurrence_grad(h, near_by, near_by, near_by, ld, starts)
    assert all(torch.equal(d[k], e[k]) for k in e)
    further = torch.empty(2 ** 26, device="cuda", dtype=torch.bfloat16).view(1, 2, -1)[..., :N]
    with pytest.raises(crf.SemiCRFError):
        crf.gated_recurrence(further, further, further, ld)


def test_residual_norm_past_32_bits(crf):  # noqa: F811
    """300,000 rows of 16,384: the last rows as by themselves, in both directions."""
    import torch
    room(120)
    B, T, N, n = 2, 150_000, 16_384, 70
    print(f"\n[residual_norm B={B} T={T} N={N}]", flush=True)
    torch.manual_seed(6)
    x, o = (torch.randn(B, T, N, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    w = torch.randn(N, device="cuda")
    kw = dict(norm_branch=True, branch_weight=w)
    r, y, stats = crf.residual_norm(x, o, w, gate=x, want_stats=True, **kw)
    last = [v[-1:, -n:].contiguous() for v in (x, o)]
    s, z, some = crf.residual_norm(*last, w, gate=last[0], want_stats=True, **kw)
    assert torch.equal(r[-1:, -n:], s) and torch.equal(y[-1:, -n:], z) and torch.equal(stats[-1:, -n:], some)
    del r
    d = crf.residual_norm_grad(None, y, x, o, w, stats, gate=x, **kw)
    e = crf.residual_norm_grad(None, z, *last, w, some, gate=last[0], **kw)
    for name in ("grad_x", "grad_branch", "grad_gate"):
        assert torch.equal(d[name][-1:, -n:], e[name]), name


def test_token_nll_past_32_bits(crf):  # noqa: F811
    """A table of 2^33 elements: losses and the gradient's rows against float32 sums by torch."""
    import torch
    room(110)
    V, N, M = 2 ** 20, 8192, 40
    print(f"\n[token_nll V={V} N={N}]", flush=True)
    torch.manual_seed(7)
    table = torch.randn(V, N, device="cuda", dtype=torch.bfloat16).mul_(N ** -0.5)
    x = torch.randn(1, M, N, device="cuda", dtype=torch.bfloat16)
    t = torch.randint(V - 5, V, (1, M), device="cuda")
    loss, lse = crf.token_nll(x, table, t, want_lse=True)
    x64 = x[0].double()
    z = torch.cat([x64 @ piece.double().t() for piece in table.split(2 ** 14)], 1)
    want = torch.logsumexp(z, 1)
    # scores of about 1 to within 2^-20, sums of 2^20 positive terms in pieces
    assert float((lse[0] - want).abs().max()) < 1e-4
    assert float((loss[0] - (want - z.gather(1, t[0][:, None])[:, 0])).abs().max()) < 1e-4
    g = torch.rand(1, M, device="cuda") + 0.5
    d = crf.token_nll_grad(g, x, table, t, lse)
    p = torch.exp(z - want[:, None])
    p[torch.arange(M, device="cuda"), t[0]] -= 1
    p *= g[0].double()[:, None]
    rows = torch.arange(V - 9, V, device="cuda")
    exact = p[:, rows].t().contiguous() @ x64
    # half a step of bfloat16 of each value, and 2^-11 of its terms in fp16
    assert float((d["grad_table"][rows].double() - exact).norm() / exact.norm()) < 2.0 ** -8
    exact = sum(p[:, i:i + 2 ** 14] @ piece.double() for i, piece in zip(range(0, V, 2 ** 14), table.split(2 ** 14)))
    assert float((d["grad_x"][0].double() - exact).norm() / exact.norm()) < 2.0 ** -8


BORDERS = [(1, 191, 70, "f32"), (2, 192, 64, "bf16"), (1, 193, 31, "f32"), (1, 384, 3, "bf16"), (2, 2049, 33, "f32"),
           (1, 6145, 2, "f32"), (1, 2048, 1, "bf16"), (1, 6300, 1, "f32")]


@pytest.mark.parametrize("case", BORDERS, ids=lambda c: "-".join(map(str, c)))
def test_recurrence_at_the_borders_of_tiles(crf, case):  # noqa: F811
    import torch
    B, T, N, typ = case
    rng = np.random.default_rng(T + N)
    x, r, i, g = (values(rng, (B, T, N), typ) for _ in range(4))
    lam, L = decays(N, "spread"), np.full(B, T)
    state, gs = rng.standard_normal((2, B, N)).astype(np.float32)
    h, last, eh, elast, _ = ref.recurrence(x, r, i, lam, L, state)
    args = [put(v, typ) for v in (x, r, i)] + [dev(lam)]
    got, end, starts = crf.gated_recurrence(*args, state=dev(state), want_state=True, want_starts=True)
    near(got, h, eh, typ, "h")
    near(end, last, elast, "f32", "state")
    d = crf.gated_recurrence_grad(put(g, typ), *args, starts, state=dev(state), grad_state=dev(gs))
    want, bound = ref.recurrence_grad(g, x, r, i, lam, L, state, gs)
    for k, v in want.items():
        near(d["grad_" + k], v, bound[k], "f32" if k in ("log_decay", "state") else typ, k)
    cut = T // 3                                             # carried on in a call with borders elsewhere
    one, two = ([v[:, s].contiguous() for v in args[:3]] + [args[3]] for s in (slice(0, cut), slice(cut, T)))
    first, mid = crf.gated_recurrence(*one, state=dev(state), want_state=True)
    near(torch.cat([first, crf.gated_recurrence(*two, state=mid)], 1), h, eh, typ, "h in two")


def test_a_workspace_of_the_callers(crf):  # noqa: F811
    """One workspace, larger than needed and holding anything, for one call after another."""
    import torch
    torch.manual_seed(8)
    B, T, N, V = 2, 500, 100, 700
    x, r, i = (torch.randn(B, T, N, device="cuda") for _ in range(3))
    ld, w = dev(decays(N, "spread")), torch.randn(N, device="cuda")
    table, t = torch.randn(V, N, device="cuda"), torch.randint(-9, V, (B, T), device="cuda")

    def work(**kw):
        h, starts = crf.gated_recurrence(x, r, i, ld, want_starts=True, **kw)
        d = crf.gated_recurrence_grad(x, x, r, i, ld, starts, **kw)
        s, y, stats = crf.residual_norm(x, h, w, want_stats=True)
        e = crf.residual_norm_grad(r, i, x, h, w, stats, **kw)
        loss, lse = crf.token_nll(y, table, t, want_lse=True, **kw)
        f = crf.token_nll_grad(loss, y, table, t, lse, **kw)
        return [h, starts, *d.values(), s, y, *e.values(), loss, lse, *f.values()]

    want = work()
    for fill in (0xff, 0x00, 0x3c):
        ws = torch.full((64 << 20,), fill, dtype=torch.uint8, device="cuda")
        assert all(torch.equal(a, b) for a, b in zip(want, work(workspace=ws)))


def test_inputs_of_another_stream(crf):  # noqa: F811
    """Inputs made on another stream that is waited for; the result used on it."""
    import torch
    torch.manual_seed(9)
    B, T, N = 2, 900, 64
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x, r, i = (torch.randn(B, T, N, device="cuda") for _ in range(3))
    ld = dev(decays(N, "spread"))
    torch.cuda.current_stream().wait_stream(side)
    want = crf.gated_recurrence(x, r, i, ld)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = crf.gated_recurrence(x, r, i, ld)
        table = torch.randn(77, N, device="cuda")
        t = torch.randint(-3, 77, (B, T), device="cuda")
        losses = [crf.token_nll(again, table, v) for v in (t, t.int())]
    torch.cuda.synchronize()
    assert torch.equal(want, again) and torch.equal(*losses)
