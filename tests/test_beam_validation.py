"""Host-side refusals of the beam selection and of the page pool's entry points, on CPU (nothing is launched)."""
import ctypes

import pytest

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4
V = ctypes.c_void_p
A, B, M4, M2, M1 = V(1 << 20), V(1 << 21), V((1 << 20) + 4), V((1 << 20) + 2), V((1 << 20) + 1)


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_fp4_gb300 import build
    build.build()
    from sparse_attention_fp4_gb300 import fp4idx
    return fp4idx._lib


def call(fn, base, **kw):
    assert set(kw) <= set(base)
    return fn(*[kw.get(n, v) for n, v in base.items()])


def test_beam_select(lib):
    base = dict(logits=A, type=0, stride=1000, vocab=1000, scores=A, n=8, beams=4, k=8, done=A, end=5, ws=A, ws_bytes=1 << 40, os=A,
                rows=A, tokens=A, done_out=A, status=None, stream=None)
    f = lambda **kw: call(lib.fp4idx_beam_select, base, **kw)  # noqa: E731
    assert f(n=0, logits=None, ws=None) == OK
    for kw in (dict(n=-4), dict(n=7), dict(beams=0), dict(k=0), dict(vocab=0), dict(stride=999), dict(end=-2), dict(end=1000), dict(end=-1),
               dict(logits=M1), dict(type=2, logits=M2), dict(done=M1), dict(done_out=M2), dict(status=M1), dict(ws=M4)):
        assert f(**kw) == INVALID, kw
    for name in ("logits", "scores", "ws", "os", "rows", "tokens"):
        assert f(**{name: None}) == INVALID, name
    for name in ("scores", "os", "rows", "tokens"):
        assert f(**{name: M2}) == INVALID, name
    for kw in (dict(type=-1), dict(type=3), dict(beams=65, n=65), dict(k=65), dict(vocab=(1 << 19) + 1, stride=1 << 20), dict(n=1 << 21),
               dict(stride=1 << 41)):
        assert f(**kw) == UNSUPPORTED, kw
    need = lib.fp4idx_beam_select_workspace_bytes(8, 1000, 8)
    assert need > 0 and f(ws_bytes=need - 1) == WORKSPACE


def test_workspace_queries(lib):
    q = lib.fp4idx_beam_select_workspace_bytes
    assert q(-1, 10, 1) == 0 and q(1, 0, 1) == 0 and q(1, (1 << 19) + 1, 1) == 0 and q(1, 10, 0) == 0 and q(1, 10, 65) == 0
    assert q((1 << 20) + 1, 10, 1) == 0 and q(0, 1, 1) > 0
    for rows in (1, 3, 16, 100, 151, 152, 153, 400, 5000):
        for vocab in (1, 100, 4097, 50001, 131072, 1 << 19):
            assert q(rows + 1, vocab, 8) >= q(rows, vocab, 8), (rows, vocab)  # (a program takes one for its most rows)
    c = lib.fp4idx_compact_pages_workspace_bytes
    assert c(0) == 0 and c((1 << 23) + 1) == 0 and c(1) > 0 and c(1 << 23) >= 1 << 25


def test_fork_pages(lib):
    base = dict(table=A, cached=A, n_old=3, max_pages=8, ratio=4, parents=A, n_new=4, pool=100, pinned=A, free=A, n_free=9, head=A,
                table_out=B, cached_out=B, src=A, dst=A, counts=A, status=None, stream=None)
    f = lambda **kw: call(lib.fp4idx_fork_pages, base, **kw)  # noqa: E731
    for kw in (dict(n_old=-1), dict(n_new=-1), dict(max_pages=0), dict(ratio=0), dict(ratio=65), dict(pool=0), dict(n_free=-1),
               dict(free=None), dict(table_out=A), dict(cached_out=A)):
        assert f(**kw) == INVALID, kw
    for name in ("table", "cached", "parents", "table_out", "cached_out", "src", "dst", "counts"):
        assert f(**{name: None}) == INVALID, name
    for name in ("table", "cached", "parents", "pinned", "free", "head", "table_out", "cached_out", "src", "dst", "counts", "status"):
        assert f(**{name: M2}) == INVALID, name
    for kw in (dict(n_old=8193), dict(n_new=8193), dict(pool=(1 << 23) + 1), dict(max_pages=1 << 26), dict(n_free=1 << 31)):
        assert f(**kw) == UNSUPPORTED, kw


def test_copy_pages(lib):
    def f(src=A, dst=A, n=4, count=None, bases=(1 << 20, 1 << 21), sizes=(4096, 256), m=None, pool=10, status=None, null=False):
        m = len(bases) if m is None else m
        r, s = (V * max(1, len(bases)))(*bases), (ctypes.c_int64 * max(1, len(sizes)))(*sizes)
        return lib.fp4idx_copy_pages(src, dst, n, count, None if null else r, None if null else s, m, pool, status, None)
    assert f(n=0) == OK and f(m=0, null=True) == OK and f(pool=0) == OK and f(n=0, src=None, dst=None) == OK
    for kw in (dict(n=-1), dict(m=-1), dict(pool=-1), dict(null=True), dict(src=None), dict(dst=None), dict(src=M2), dict(dst=M1),
               dict(count=M2), dict(status=M2), dict(bases=(None, 1 << 21)), dict(bases=((1 << 20) + 8, 1 << 21)), dict(sizes=(4096, 0)),
               dict(sizes=(4096, 250)), dict(sizes=(-16, 16))):
        assert f(**kw) == INVALID, kw
    for kw in (dict(n=(1 << 24) + 1), dict(bases=(1 << 20,) * 257, sizes=(16,) * 257), dict(pool=1 << 31), dict(sizes=(4096, (1 << 30) + 16))):
        assert f(**kw) == UNSUPPORTED, kw


def test_compact_pages(lib):
    base = dict(table=A, cached=A, n=3, max_pages=8, ratio=4, pool=100, pinned=A, ws=A, ws_bytes=1 << 30, free=A, n_free=9, table_out=B, src=A,
                dst=A, moves=4, counts=A, status=None, stream=None)
    f = lambda **kw: call(lib.fp4idx_compact_pages, base, **kw)  # noqa: E731
    for kw in (dict(n=-1), dict(max_pages=0), dict(ratio=0), dict(ratio=65), dict(pool=0), dict(n_free=-1), dict(free=None), dict(table_out=A),
               dict(moves=-1), dict(ws=None), dict(ws=M4)):
        assert f(**kw) == INVALID, kw
    for name in ("table", "cached", "table_out", "src", "dst", "counts"):
        assert f(**{name: None}) == INVALID, name
    for name in ("table", "cached", "pinned", "free", "table_out", "src", "dst", "counts", "status"):
        assert f(**{name: M2}) == INVALID, name
    for kw in (dict(n=65537), dict(pool=(1 << 23) + 1), dict(max_pages=1 << 26), dict(n_free=1 << 31), dict(moves=1 << 31)):
        assert f(**kw) == UNSUPPORTED, kw
    assert f(ws_bytes=399) == WORKSPACE
