"""A step without rows: the attention entry points accept it, as the indexer's do, also where
there is no sequence, page or table (CPU: nothing is launched)."""
import ctypes

import pytest

OK, INVALID = 0, 1
A = ctypes.c_void_p(1 << 20)


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_fp4_gb300 import build
    build.build()
    from sparse_attention_fp4_gb300 import fp4idx
    return fp4idx._lib


def selected(lib, n, seqs, pages, cols, table):
    return lib.fp4idx_latent_attn_topk(A, n, 64, 576, A, pages, table, seqs, cols, A, A, 16, None, 0.1, A, 1 << 40, A, None, None, None)


def whole(lib, n, seqs, pages, cols, table):
    return lib.fp4idx_latent_attn(A, n, 64, 576, A, pages, table, seqs, cols, A, A, 0, None, 0, 0.1, A, 1 << 40, A, None, None, None)


@pytest.mark.parametrize("call", [selected, whole])
def test_no_rows(lib, call):
    assert call(lib, 0, 0, 8, 4, None) == OK
    assert call(lib, 0, 0, 0, 0, None) == OK
    assert call(lib, 0, 2, 0, 4, A) == OK
    for seqs, pages, cols in ((-1, 8, 4), (2, -1, 4), (2, 8, -1)):
        assert call(lib, 0, seqs, pages, cols, A) == INVALID
    for seqs, pages, cols in ((0, 8, 4), (2, 0, 4), (2, 8, 0)):
        assert call(lib, 1, seqs, pages, cols, A) == INVALID
