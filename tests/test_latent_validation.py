"""Host-side refusals of the latent-attention entry points, on CPU (nothing is launched)."""
import ctypes
import math

import pytest

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4
V = ctypes.c_void_p
A, M4, M1 = V(1 << 20), V((1 << 20) + 4), V((1 << 20) + 1)


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_fp4_gb300 import build
    build.build()
    from sparse_attention_fp4_gb300 import fp4idx
    return fp4idx._lib


def call(fn, base, **kw):
    assert set(kw) <= set(base)
    return fn(*[kw.get(n, v) for n, v in base.items()])


def test_plan_step(lib):
    base = dict(cached=A, new=A, n=3, ratio=4, free=A, n_free=9, head=A, table=A, max_pages=8, qp=A, rs=A, cl=A, rows=5,
                sp=A, ss=A, stores=5, cu=A, cuc=A, counts=A, status=None, stream=None)
    f = lambda **kw: call(lib.fp4idx_plan_step, base, **kw)  # noqa: E731
    for kw in (dict(n=-1), dict(ratio=0), dict(ratio=65), dict(n_free=-1), dict(max_pages=0), dict(rows=-1), dict(stores=-1)):
        assert f(**kw) == INVALID, kw
    for name in ("cached", "new", "free", "table", "qp", "rs", "cl", "sp", "ss", "cu", "cuc", "counts"):
        assert f(**{name: None}) == INVALID, name
        assert f(**{name: M1}) == INVALID, name
    assert f(head=M1) == INVALID and f(status=M1) == INVALID
    for kw in (dict(n=65537), dict(max_pages=1 << 26), dict(rows=1 << 31), dict(stores=1 << 31), dict(n_free=1 << 31)):
        assert f(**kw) == UNSUPPORTED, kw


def test_store_latent(lib):
    base = dict(kv=A, n=4, width=576, pos=A, slots=A, w=A, eps=1e-6, cs=A, max_pos=16, cache=A, pages=8, status=None, stream=None)
    f = lambda **kw: call(lib.fp4idx_store_latent, base, **kw)  # noqa: E731
    assert f(n=0, kv=None) == OK
    for kw in (dict(n=-1), dict(pages=-1), dict(max_pos=0), dict(status=M1), dict(pos=M1), dict(slots=M1)):
        assert f(**kw) == INVALID, kw
    for name in ("kv", "w", "cs", "cache"):
        assert f(**{name: None}) == INVALID and f(**{name: M4}) == INVALID, name
    assert f(width=640) == UNSUPPORTED and f(width=128) == UNSUPPORTED and f(pages=1 << 26) == UNSUPPORTED


def attn_cases(f, lib):
    need = lib.fp4idx_latent_attn_workspace_bytes(4, 64)
    assert need > 0 and f(ws_bytes=need - 1) == WORKSPACE
    assert f(n=0, q=None, out=None) == OK
    for kw in (dict(n=-1), dict(heads=0), dict(pages=0), dict(seqs=0), dict(max_pages=0), dict(scale=math.nan), dict(scale=math.inf),
               dict(status=M1), dict(lse=M1)):
        assert f(**kw) == INVALID, kw
    for name in ("q", "cache", "ws", "out"):
        assert f(**{name: None}) == INVALID and f(**{name: M4}) == INVALID, name
    for name in ("table", "rs"):
        assert f(**{name: None}) == INVALID and f(**{name: M1}) == INVALID, name
    for kw in (dict(width=448), dict(heads=129), dict(n=(1 << 20) + 1), dict(pages=1 << 26), dict(max_pages=1 << 26)):
        assert f(**kw) == UNSUPPORTED, kw


def test_latent_attn_topk(lib):
    base = dict(q=A, n=4, heads=64, width=576, cache=A, pages=8, table=A, seqs=2, max_pages=4, rs=A, idx=A, k=16, cl=A, scale=0.1,
                ws=A, ws_bytes=1 << 40, out=A, lse=A, status=None, stream=None)
    f = lambda **kw: call(lib.fp4idx_latent_attn_topk, base, **kw)  # noqa: E731
    attn_cases(f, lib)
    assert f(k=0) == INVALID and f(k=4097) == INVALID and f(idx=None) == INVALID and f(idx=M1) == INVALID and f(cl=M1) == INVALID


def test_latent_attn(lib):
    base = dict(q=A, n=4, heads=64, width=576, cache=A, pages=8, table=A, seqs=2, max_pages=4, rs=A, cl=A, max_context=256, tree=A,
                words=1, scale=0.1, ws=A, ws_bytes=1 << 40, out=A, lse=A, status=None, stream=None)
    f = lambda **kw: call(lib.fp4idx_latent_attn, base, **kw)  # noqa: E731
    attn_cases(f, lib)
    for kw in (dict(max_context=-1), dict(max_context=257), dict(words=-1), dict(words=0), dict(tree=None), dict(tree=M1), dict(cl=None), dict(cl=M1)):
        assert f(**kw) == INVALID, kw
    assert f(words=9) == UNSUPPORTED


def test_workspace_query(lib):
    q = lib.fp4idx_latent_attn_workspace_bytes
    assert q(-1, 64) == 0 and q(4, 0) == 0 and q(4, 129) == 0 and q((1 << 20) + 1, 64) == 0 and q(1, 1) > 0
    assert q(100, 64) >= q(1, 64)


def test_latent_prefill(lib):
    base = dict(q=A, nq=64, heads=4, kv=A, nkv=64, kr=A, cq=A, ck=A, seqs=2, max_q=40, max_kv=40, scale=0.1, out=A, lse=A, status=None,
                stream=None)
    f = lambda **kw: call(lib.fp4idx_latent_prefill, base, **kw)  # noqa: E731
    assert f(nq=0, q=None) == OK and f(seqs=0) == OK and f(max_q=0) == OK
    for kw in (dict(nq=-1), dict(nkv=-1), dict(heads=0), dict(seqs=-1), dict(max_q=-1), dict(max_kv=-1), dict(scale=math.nan),
               dict(lse=M1), dict(status=M1)):
        assert f(**kw) == INVALID, kw
    for name in ("q", "kv", "kr", "out"):
        assert f(**{name: None}) == INVALID and f(**{name: M4}) == INVALID, name
    for name in ("cq", "ck"):
        assert f(**{name: None}) == INVALID and f(**{name: M1}) == INVALID, name
    assert f(heads=1025) == UNSUPPORTED and f(seqs=65536) == UNSUPPORTED and f(nq=(1 << 24) + 1) == UNSUPPORTED


def test_plan_step_limits(lib):
    """Row and store counters are 32 bits and advance by a grid of threads: half of them stay free."""
    base = dict(cached=A, new=A, n=3, ratio=4, free=A, n_free=9, head=A, table=A, max_pages=8, qp=A, rs=A, cl=A, rows=5,
                sp=A, ss=A, stores=5, cu=A, cuc=A, counts=A, status=None, stream=None)
    assert call(lib.fp4idx_plan_step, base, rows=(1 << 30) + 1) == UNSUPPORTED
    assert call(lib.fp4idx_plan_step, base, stores=(1 << 30) + 1) == UNSUPPORTED
