"""What the token loss asks for as its workspace.  Sizes need no GPU, and refused calls follow no pointer."""

import ctypes

import pytest

WORKSPACE = 2
P = ctypes.c_void_p(0x1000)


@pytest.fixture(scope="module")
def lib():
    from semi_markov_crf_amd import _native
    return _native.load()


@pytest.mark.parametrize("dtype,e", [(0, 4), (1, 2)])
@pytest.mark.parametrize("shape", [(1, 16, 50_001, 1024), (1, 40, 2 ** 20, 8192), (2, 300, 700, 64)])
def test_an_aligned_table_is_not_copied(lib, dtype, e, shape):
    B, T, V, N = shape
    table = V * N * e
    for grad in (0, 1):
        any_table = lib.semicrf_token_nll_bytes(dtype, *shape, grad)
        assert any_table == lib.semicrf_token_nll_table_bytes(dtype, *shape, None, grad)
        assert any_table == lib.semicrf_token_nll_table_bytes(dtype, *shape, 0x1002, grad)
        this = lib.semicrf_token_nll_table_bytes(dtype, *shape, 0x1010, grad)
        if grad and e == 4:
            assert this == any_table
        else:
            assert any_table - this >= table
            if not grad and V > 2 ** 16:
                assert this < table / 4
        # a call takes what its own table needs, and no less
        for at, need in ((0x1010, this), (0x1002, any_table)):
            if grad:
                rc = lib.semicrf_token_nll_grad(P, P, at, dtype, P, 32, None, P, *shape, 1.0, None, P, need - 1, P, P,
                                                None)
            else:
                rc = lib.semicrf_token_nll(P, at, dtype, P, 32, None, *shape, 1.0, None, P, need - 1, P, None, None)
            assert rc == WORKSPACE


def test_a_width_of_no_whole_steps_is_copied(lib):
    for N in (63, 65, 100):
        size = lib.semicrf_token_nll_bytes(1, 2, 3, 50, N, 0)
        assert lib.semicrf_token_nll_table_bytes(1, 2, 3, 50, N, 0x1000, 0) == size
    assert lib.semicrf_token_nll_table_bytes(1, 2, 3, 50, 0, 0x1000, 0) == 0


def test_softmaxes_take_two_gigabytes_or_256_words(lib):
    """As the header says, beside the copies, the lists and the shared-out tiles' sums (below 1 GB here)."""
    for dtype, e in ((0, 4), (1, 2)):
        for rows, V in ((1 << 22, 4096), (1 << 16, 1 << 19), (1 << 20, 1 << 12)):
            n = lib.semicrf_token_nll_bytes(dtype, 1, rows, V, 16, 1)
            p = max(2 << 30, 256 * rows * e)
            pieces = -(-V * rows * e // p)
            copies = 2 * rows * 64 * e + V * 64 * 2 * e + (rows * 16 * 4 if pieces > 1 else 0)
            assert n <= p + copies + (1 << 30), (dtype, rows, V)
