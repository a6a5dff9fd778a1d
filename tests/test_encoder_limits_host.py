"""Sizes past what the encoder operators take, refused before a launch: no pointer here is
followed."""

import ctypes

import pytest

UNSUPPORTED = 3
P = ctypes.c_void_p(0x1000)


@pytest.fixture(scope="module")
def lib():
    from semi_markov_crf_amd import _native
    return _native.load()


def test_embed_refuses_rows_of_2_30_elements(lib):
    for N in (1 << 30, (1 << 31) - 1):
        assert lib.semicrf_embed(P, 32, None, P, 1, 1, 1, 1, N, 1.0, None, P, None) == UNSUPPORTED


def test_embed_grad_refuses_rows_past_2_23_elements(lib):
    """The second dimension of its grids would not hold their slabs of 256 columns."""
    n = lib.semicrf_embed_grad_bytes(0, 1, 1, 1, 1 << 23)
    assert n > 0
    for N in ((1 << 23) + 1, 1 << 25, 1 << 30):
        assert lib.semicrf_embed_grad_bytes(0, 1, 1, 1, N) == 0
        assert lib.semicrf_embed_grad(P, 32, None, P, 0, 1, 1, 1, N, 1.0, None, P, 1 << 40, P, None) == UNSUPPORTED
