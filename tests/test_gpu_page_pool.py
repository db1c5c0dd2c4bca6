"""Fork, copy and compaction of the page pool against plain references (whole numbers)."""
import random

import pytest
import torch

from tests import beam_ref as ref

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def guarded(n):
    return torch.full((n + 7,), -77, dtype=torch.int32, device="cuda")


def whole(v, n):
    assert bool((v[n:] == -77).all())
    return v[:n].tolist()


def state(seed, rows, most, ratio, pool, share=0.7, same=False):
    """Rows that share full pages with a row before them, partly filled pages of their own."""
    r = random.Random(seed)
    ids = list(range(pool))
    r.shuffle(ids)
    table, cached = [], []
    length = r.randrange(0, most * 64 * ratio + 1)
    for b in range(rows):
        c = length if same else r.randrange(0, most * 64 * ratio + 1)
        n, full = -(-(c // ratio) // 64), c // ratio // 64
        row = []
        if table and r.random() < share:
            up = r.randrange(len(table))
            row = table[up][:r.randrange(0, min(full, cached[up] // ratio // 64) + 1)]
        row = row + [ids.pop() for _ in range(n - len(row))]
        table.append(row + [r.choice([-1, 10 ** 9, 5]) for _ in range(most - n)])
        cached.append(c)
    return table, cached, ids


def run_fork(table, cached, ratio, parents, pool, free, head, pinned=(), most=None, stream=None):
    from sparse_attention_fp4_gb300 import fp4idx
    A, B = len(table), len(parents)
    most = most or len(table[0])
    t = i32(table).view(A, most) if A else torch.empty((0, most), dtype=torch.int32, device="cuda")
    f = i32(free)
    out, cout, src, dst, counts = (guarded(n) for n in (B * most, B, B, B, 4))
    status = i32([0])
    pins = i32(ref.words(pinned, pool)) if pinned else None
    c, p, h = i32(cached), i32(parents), None if head is None else i32([head])
    keep = t.clone()
    for _ in range(2):  # repeated: the same
        fp4idx.fork_pages(t, c, ratio, p, pool, f, out[:B * most].view(B, most), cout[:B], src[:B], dst[:B], counts[:4], free_head=h,
                          pinned=pins, status=status, stream=stream)
    torch.cuda.synchronize()
    assert bool((t == keep).all()) and c.tolist() == cached
    flat = whole(out, B * most)
    return dict(table=[flat[i * most:(i + 1) * most] for i in range(B)], cached=whole(cout, B), src=whole(src, B), dst=whole(dst, B),
                counts=whole(counts, 4), free=f.tolist()), fp4idx.read_status(status)


def check_fork(table, cached, ratio, parents, pool, free, head=None, pinned=(), **kw):
    want = ref.fork(table, cached, ratio, parents, pool, free, head or 0, set(pinned)) if table else None
    got, status = run_fork(table, cached, ratio, parents, pool, free, head, pinned, **kw)
    if want:
        bad = want.pop("bad")
        assert (status in bad) if bad else status == 0, (status, bad)
        for n in want:
            assert got[n] == want[n], n
    return got


def pick(seed, rows, new, ended=0.0):
    r = random.Random(seed)
    return [-1 if r.random() < ended else r.randrange(rows) for _ in range(new)]


@pytest.mark.parametrize("rows,most,ratio,new,ended", [
    (1, 1, 1, 1, 0), (1, 1, 64, 3, 0), (4, 3, 4, 4, 0), (4, 8, 1, 4, 0.3), (8, 5, 2, 8, 0), (3, 40, 1, 12, 0), (64, 20, 4, 64, 0.1),
    (64, 130, 1, 64, 0), (5, 300, 1, 5, 0.5), (33, 129, 3, 70, 0.2), (1, 2000, 1, 4, 0), (2, 30000, 1, 3, 0.3), (200, 128, 1, 130, 0.4), (7, 9, 1, 0, 0)])
def test_fork(rows, most, ratio, new, ended):
    for seed in range(3):
        table, cached, ids = state(seed, rows, most, ratio, rows * most + new + 9, same=seed == 1)
        parents = pick(seed + 5, rows, new, ended)
        check_fork(table, cached, ratio, parents, rows * most + new + 9, [-9] * (rows * most) + ids, rows * most)


@pytest.mark.parametrize("rows", [1023, 1024, 1025, 4000])
def test_fork_of_many_rows(rows):
    table, cached, ids = state(rows, rows, 3, 1, rows * 5)
    parents = pick(rows, rows, rows + 3, 0.1)
    check_fork(table, cached, 1, parents, rows * 5, [-9] * rows * 3 + ids, rows * 3)


def test_fork_of_the_most_rows():
    rows = 8192
    table, cached, ids = state(8, rows, 2, 1, rows * 3 + 5)
    check_fork(table, cached, 1, pick(1, rows, rows, 0.1), rows * 3 + 5, [-9] * rows * 2 + ids, rows * 2)


@pytest.mark.parametrize("pool", [33, 1 << 12, (1 << 20) + 17, 1 << 23])
def test_fork_in_pools_of_any_size(pool):
    r = random.Random(pool)
    ids = sorted(r.sample(range(pool), 32), reverse=True) if pool == 33 else [pool - 1 - 131 * i % pool for i in range(100)]
    ids = list(dict.fromkeys(ids))
    table = [[ids[0], ids[1], -1], [ids[0], ids[2], -1], [ids[3], ids[4], ids[5]], [ids[6], -1, -1]]
    check_fork(table, [100, 128, 190, 64], 1, [1, 1, 3, 3, 2, 2], pool, [7] * 5 + ids[7:], 5)
    check_fork(table, [100, 128, 190, 64], 1, [0, 0, 0, -1], pool, [7] * 9 + ids[7:], 9)


def test_fork_of_the_most_rows_in_the_largest_pool():
    rows, pool = 8192, 1 << 23
    table, cached, ids = state(9, rows, 2, 1, rows * 3)
    far = lambda p: pool - 1 - 331 * p if p >= 0 else p  # noqa: E731
    table = [[far(p) if 0 <= p < rows * 3 else p for p in t] for t in table]
    got = check_fork(table, cached, 1, pick(2, rows, rows, 0.1), pool, [-9] * rows * 2 + [far(p) for p in ids], rows * 2)
    assert got["counts"][0] > 1000 and got["counts"][1] > 1000


def test_fork_identity_and_release():
    """Rows that go on from themselves cost nothing; a batch that ends gives every page back."""
    table, cached, ids = state(3, 12, 30, 1, 500)
    got = check_fork(table, cached, 1, list(range(12)), 500, [-9] * 400 + ids, 400)
    assert got["counts"] == [0, 0, 0, 12]
    got = check_fork(table, cached, 1, [-1] * 12, 500, [-9] * 400 + ids, 400)
    held = {p for t, c in zip(table, cached) for p in t[:-(-c // 64)]}
    assert got["counts"] == [0, len(held), -len(held), 0]
    got = check_fork(table, cached, 1, [], 500, [-9] * 400 + ids, 400, most=30)
    assert got["counts"][1] == len(held)


def test_fork_of_nothing():
    got, status = run_fork([], [], 1, [-1, -1], 10, [3, 4], 0, most=4)
    assert status == 0 and got["table"] == [[-1] * 4] * 2 and got["counts"] == [0, 0, 0, 0] and got["free"] == [3, 4]
    got, status = run_fork([], [], 1, [], 10, [], None, most=4)
    assert status == 0 and got["counts"] == [0, 0, 0, 0]


def test_fork_pinned():
    """Pinned pages are not given back; a pinned page that is partly filled is copied for the first row too."""
    table, cached, ids = state(4, 20, 12, 1, 400)
    r = random.Random(2)
    pages = [p for t, c in zip(table, cached) for p in t[:-(-c // 64)]]
    pinned = r.sample(pages, len(pages) // 2) + ids[:3]
    check_fork(table, cached, 1, pick(3, 20, 20, 0.2), 400, [-9] * 300 + ids[3:], 300, pinned=pinned)
    check_fork(table, cached, 1, list(range(20)), 400, [-9] * 300 + ids[3:], 300, pinned=pinned)


@pytest.mark.parametrize("avail", [0, 1, 3, 100])
def test_fork_out_of_pages(avail):
    table, cached = [[4, 5, 6], [7, 8, -1]], [150, 100]
    check_fork(table, cached, 1, [0, 0, 0, 1, 1, 1, -1, 1], 200, list(range(100, 100 + avail)), 0)
    check_fork(table, cached, 1, [0] * 6, 200, list(range(100, 100 + avail)), 0)


@pytest.mark.parametrize("head", [0, 1, 4, 5])
def test_fork_out_of_room_below_the_head(head):
    table, cached = [[4, 5, 6], [7, 8, -1], [10, 11, 12]], [150, 100, 192]
    check_fork(table, cached, 1, [1, 1, -1], 50, list(range(20, 25)) + [30, 31], head)


@pytest.mark.parametrize("head", [-1, 8, -2 ** 31, 2 ** 31 - 1])
def test_fork_bad_head(head):
    table, cached = [[4, 5, 6], [7, 8, -1]], [150, 100]
    check_fork(table, cached, 1, [1, 1, 1, 1, 1], 50, list(range(20, 27)), head)
    check_fork(table, cached, 1, [-1, 0], 50, list(range(20, 27)), head)


def test_fork_bad_parents_lengths_and_ids():
    table = [[1, 2, 3], [4, -5, 6], [7, 8, 9], [10, 99, 11], [12, 13, 400]]
    cached = [150, 192, -1, 193, 130]
    for parents in ([0, 1, 2, 3, 4], [5, -2, 2 ** 31 - 1, -2 ** 31, 0], [4, 4, 4, 1, 1], [2, 2, 3, 3, 0], [-1] * 5):
        check_fork(table, cached, 1, parents, 99, [50, 51, 52, 53], 2)


def test_fork_largest_lengths():
    table = [[1, 2], [3, 4]]
    check_fork(table, [2 ** 31 - 1, 100], 64, [0, 0, 1, 1], 20, [9, 10, 11], 1)
    check_fork(table, [8191, 8192], 64, [0, 0, 1, 1], 20, [9, 10, 11], 1)


def test_fork_streams_and_graph():
    from sparse_attention_fp4_gb300 import fp4idx
    table, cached, ids = state(6, 40, 50, 1, 2200)
    parents = pick(6, 40, 40, 0.1)
    free = [-9] * 2000 + ids
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    check_fork(table, cached, 1, parents, 2200, free, 2000, stream=side)
    t, c, p, f, h = i32(table), i32(cached), i32(parents), i32(free), i32([2000])
    out, cout, src, dst, counts = torch.empty_like(t), torch.empty_like(c), torch.empty_like(p), torch.empty_like(p), i32([0] * 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp4idx.fork_pages(t, c, 1, p, 2200, f, out, cout, src, dst, counts, free_head=h)
    for seed in (6, 7, 8):
        p.copy_(i32(pick(seed, 40, 40, 0.1)))
        f.copy_(i32(free))
        graph.replay()
        want = ref.fork(table, cached, 1, p.tolist(), 2200, free, 2000)
        assert out.tolist() == want["table"] and f.tolist() == want["free"] and counts.tolist() == want["counts"]
        assert src.tolist() == want["src"] and dst.tolist() == want["dst"]


# ---------------------------------------------------------------- compaction
def run_compact(table, cached, ratio, pool, free, moves, pinned=(), most=None, stream=None):
    from sparse_attention_fp4_gb300 import fp4idx
    B = len(table)
    most = most or len(table[0])
    t = i32(table).view(B, most) if B else torch.empty((0, most), dtype=torch.int32, device="cuda")
    out, src, dst, counts, f = (guarded(n) for n in (B * most, moves, moves, 4, len(free)))
    f[:len(free)] = i32(free)
    status = i32([0])
    ws = torch.full((fp4idx.compact_pages_workspace_bytes(pool),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        fp4idx.compact_pages(t, i32(cached), ratio, pool, ws, f[:len(free)], out[:B * most].view(B, most), src[:moves], dst[:moves], counts[:4],
                             pinned=i32(ref.words(pinned, pool)) if pinned else None, status=status, stream=stream)
    torch.cuda.synchronize()
    flat = whole(out, B * most)
    return dict(table=[flat[i * most:(i + 1) * most] for i in range(B)], src=whole(src, moves), dst=whole(dst, moves), counts=whole(counts, 4),
                free=whole(f, len(free))), fp4idx.read_status(status)


def check_compact(table, cached, ratio, pool, free, moves, pinned=(), **kw):
    want = ref.compact(table, cached, ratio, pool, free, moves, set(pinned))
    got, status = run_compact(table, cached, ratio, pool, free, moves, pinned, **kw)
    bad = want.pop("bad")
    assert (status in bad) if bad else status == 0, (status, bad)
    for n in want:
        assert got[n] == want[n], n
    return got


@pytest.mark.parametrize("rows,most,ratio,pool,moves", [
    (1, 1, 1, 1, 1), (1, 1, 1, 40, 1), (4, 3, 4, 33, 9), (4, 8, 1, 500, 3), (64, 20, 4, 4096, 2000), (64, 130, 1, 9000, 9000),
    (5, 300, 1, 1600, 100), (33, 129, 3, 70001, 5000), (300, 128, 1, 300000, 40000), (7, 9, 1, 64, 0), (2000, 3, 2, 6001, 50)])
def test_compact(rows, most, ratio, pool, moves):
    for seed in range(3):
        table, cached, _ = state(seed, rows, most, ratio, pool, share=0.5)
        check_compact(table, cached, ratio, pool, [-3] * pool, moves)
        check_compact(table, cached, ratio, pool, [-3] * (pool + 5), moves)


def test_compact_twice_moves_nothing_more():
    table, cached, _ = state(5, 30, 20, 1, 3000)
    once = check_compact(table, cached, 1, 3000, [-3] * 3000, 1000)
    again = check_compact(once["table"], cached, 1, 3000, once["free"], 1000)
    assert again["counts"][0] == 0 and again["table"] == once["table"] and again["free"] == once["free"]
    assert once["counts"][2] == once["counts"][1] == 3000 - (3000 - once["counts"][3])


def test_compact_pinned():
    table, cached, ids = state(6, 30, 20, 1, 3000)
    pages = [p for t, c in zip(table, cached) for p in t[:-(-c // 64)]]
    for seed in range(4):
        pinned = random.Random(seed).sample(pages, len(pages) // 3) + ids[:40]
        check_compact(table, cached, 1, 3000, [-3] * 3000, 1000, pinned=pinned)
    check_compact([[5, 6]], [0], 1, 40, [-3] * 40, 7, pinned=[39, 0, 31, 32])


def test_compact_empty():
    got = check_compact([[5, 6, 7]], [0], 1, 100, [-3] * 100, 4)
    assert got["counts"] == [0, 0, 0, 0] and got["free"] == list(range(100))
    got, status = run_compact([], [], 1, 10, [-3] * 10, 2, most=3)
    assert status == 0 and got["free"] == list(range(10))


def test_compact_free_list_too_short():
    table, cached, _ = state(7, 10, 6, 1, 200)
    for n in (0, 1, 50):
        check_compact(table, cached, 1, 200, [-3] * n, 100)


def test_compact_bad_lengths_and_ids():
    table = [[1, 92, 3], [4, -5, 6], [7, 8, 9], [10, 99, 11], [12, 13, 400]]
    check_compact(table, [150, 192, -1, 193, 130], 1, 99, [-3] * 99, 10)
    check_compact(table, [150, 192, 2 ** 31 - 1, 193, 130], 1, 95, [-3] * 95, 1)


@pytest.mark.parametrize("pool", [(1 << 20) + 17, 1 << 23])
def test_compact_in_large_pools(pool):
    ids = [pool - 1 - 1237 * i for i in range(150)]
    table = [ids[:50], ids[:20] + ids[50:80], ids[80:130]]
    check_compact(table, [50 * 64, 49 * 64 + 1, 3000], 1, pool, [-3] * pool, 200, pinned=[ids[3], ids[140], 77])


def test_compact_streams_and_graph():
    from sparse_attention_fp4_gb300 import fp4idx
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    table, cached, _ = state(8, 40, 50, 1, 5000)
    check_compact(table, cached, 1, 5000, [-3] * 5000, 2000, stream=side)
    t, c = i32(table), i32(cached)
    ws = torch.empty(fp4idx.compact_pages_workspace_bytes(5000), dtype=torch.uint8, device="cuda")
    out, f, src, dst, counts = torch.empty_like(t), i32([-3] * 5000), i32([0] * 2000), i32([0] * 2000), i32([0] * 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp4idx.compact_pages(t, c, 1, 5000, ws, f, out, src, dst, counts)
    for seed in (8, 9):
        table, cached, _ = state(seed, 40, 50, 1, 5000)
        t.copy_(i32(table)), c.copy_(i32(cached))
        f.fill_(-3)
        graph.replay()
        want = ref.compact(table, cached, 1, 5000, [-3] * 5000, 2000)
        assert out.tolist() == want["table"] and f.tolist() == want["free"] and counts.tolist() == want["counts"]
        assert src.tolist() == want["src"] and dst.tolist() == want["dst"]


# ---------------------------------------------------------------- copies
def filled(seed, *shape, dtype=torch.uint8):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = torch.empty(0, dtype=dtype).element_size()
    raw = torch.randint(0, 256, (*shape[:-1], shape[-1] * n), generator=g, device="cuda", dtype=torch.uint8)
    return raw.view(dtype)


def caches_of(seed, pool, kinds):
    shapes = dict(payload=((4, 64, 16), torch.uint8), scale=((4, 64), torch.uint8), latent=((64, 576), torch.bfloat16),
                  narrow=((64, 512), torch.bfloat16), fp8=((8448,), torch.uint8), tiny=((16,), torch.uint8), odd=((5, 7, 12), torch.float32))
    return [filled(seed + i, pool, *shapes[k][0], dtype=shapes[k][1]) for i, k in enumerate(kinds)]


def raw(c):
    return c.reshape(c.shape[0], -1).view(torch.uint8)


def check_copy(src, dst, caches, count=None, want_status=0, stream=None):
    from sparse_attention_fp4_gb300 import fp4idx
    want = [raw(c).clone() for c in caches]
    pool = caches[0].shape[0] if caches else 0
    for s, d in list(zip(src, dst))[:len(src) if count is None else max(0, count)]:
        if 0 <= s < pool and 0 <= d < pool:
            for w, c in zip(want, caches):
                w[d] = raw(c)[s]
    status = i32([0])
    fp4idx.copy_pages(i32(src), i32(dst), caches, count=None if count is None else i32([count]), status=status, stream=stream)
    torch.cuda.synchronize()
    assert fp4idx.read_status(status) == want_status
    for w, c in zip(want, caches):
        assert bool((w == raw(c)).all())


KINDS = [("payload",), ("scale",), ("tiny",), ("odd",), ("latent",), ("payload", "scale"), ("payload", "scale", "latent"),
         ("fp8", "narrow"), ("tiny", "latent", "odd", "scale")]


@pytest.mark.parametrize("kinds", KINDS, ids=lambda k: "-".join(k))
@pytest.mark.parametrize("n", [0, 1, 2, 37, 300])
def test_copy(kinds, n):
    pool = 2 * n + 3
    ids = random.Random(n).sample(range(pool), 2 * n)
    check_copy(ids[:n], ids[n:], caches_of(n, pool, kinds))


def test_copy_many_regions():
    pool = 50
    ids = random.Random(1).sample(range(pool), 30)
    check_copy(ids[:15], ids[15:], caches_of(1, pool, ("payload", "scale", "tiny", "fp8") * 64))


def test_copy_large_pages():
    caches = [filled(8, 6, 3 << 20), filled(9, 6, 5, 4000016, dtype=torch.float32)]
    assert raw(caches[1]).shape[1] % 16 == 0
    check_copy([0, 3], [5, 1], caches)


def test_copy_padding_count_and_bad_ids():
    caches = caches_of(3, 20, ("payload", "scale", "latent"))
    check_copy([1, -1, 3, 4, -1, 6], [11, 12, -1, 14, -1, 16], caches)
    check_copy([1, 2, 3, 4], [11, 12, 13, 14], caches, count=2)
    check_copy([1, 2, 3, 4], [15, 16, 17, 18], caches, count=0)
    check_copy([1, 2, 3, 4], [15, 16, 17, 18], caches, count=-3)
    check_copy([1, 2, 3, 4], [11, 12, 13, 14], caches, count=2 ** 31 - 1)
    check_copy([1, 20, 3, 2 ** 31 - 1], [15, 16, 20, 17], caches, want_status=5)
    check_copy([7, 8], [7, 9], caches)  # a page onto itself
    check_copy([5, 5, 5], [10, 11, 12], caches)  # one page to several


def test_copy_one_source_to_many():
    caches = caches_of(4, 400, ("latent", "scale"))
    check_copy([3] * 300, list(range(50, 350)), caches)


def test_copy_past_32_bit_offsets():
    """A pool of more than 4 GB."""
    pool = 70000
    c = torch.zeros((pool, 64, 512), dtype=torch.bfloat16, device="cuda")
    c[0], c[pool - 2], c[40000] = 1.0, 2.0, 3.0
    from sparse_attention_fp4_gb300 import fp4idx
    fp4idx.copy_pages(i32([0, pool - 2, 40000]), i32([pool - 1, 1, 65537]), [c])
    torch.cuda.synchronize()
    assert [float(c[p].float().mean()) for p in (pool - 1, 1, 65537, 2)] == [1.0, 2.0, 3.0, 0.0]


def test_copy_streams_and_graph():
    from sparse_attention_fp4_gb300 import fp4idx
    caches = caches_of(5, 60, ("payload", "scale", "latent"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    check_copy([1, 2], [30, 31], caches, stream=side)
    src, dst, n = i32([1, 2, 3]), i32([40, 41, 42]), i32([3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp4idx.copy_pages(src, dst, caches, count=n)
    for k in (2, 3):
        n.fill_(k)
        src += 4
        want = [raw(c).clone() for c in caches]
        for s, d in list(zip(src.tolist(), dst.tolist()))[:k]:
            for w, c in zip(want, caches):
                w[d] = raw(c)[s]
        graph.replay()
        torch.cuda.synchronize()
        assert all(bool((w == raw(c)).all()) for w, c in zip(want, caches))


def test_copy_without_pages_or_caches():
    from sparse_attention_fp4_gb300 import fp4idx
    fp4idx.copy_pages(i32([1]), i32([2]), [])
    fp4idx.copy_pages(i32([]), i32([]), [torch.empty((0, 4, 64, 16), dtype=torch.uint8, device="cuda")])
    fp4idx.copy_pages(i32([1]), i32([0]), [torch.empty((0, 4, 64, 16), dtype=torch.uint8, device="cuda")])


def test_refusals_of_the_binding():
    from sparse_attention_fp4_gb300 import fp4idx
    a = caches_of(6, 8, ("payload",))[0]
    one, two = i32([1]), i32([2])
    for bad in ([a[:, :2]], [a, a[:4]], [a.cpu()]):
        with pytest.raises(ValueError):
            fp4idx.copy_pages(one, two, bad)
    with pytest.raises(ValueError):
        fp4idx.copy_pages(one, i32([]), [a])
    for bad in ([a.view(-1)], [a] * 257):
        with pytest.raises(fp4idx.Fp4IdxError):
            fp4idx.copy_pages(one, two, bad)
    t, c = i32([[1, 2]]), i32([70])
    out, counts, free = torch.empty_like(t), i32([0] * 4), i32([3, 4])
    fork = lambda t=t, c=c, p=one, out=out, cout=torch.empty_like(c), src=one, dst=two, **kw: fp4idx.fork_pages(  # noqa: E731
        t, c, 1, i32([0]), 8, free, out, cout, src, dst, counts, **kw)
    fork()
    for kw in (dict(out=i32([[1, 2, 3]])), dict(out=i32([[1, 2], [1, 2]])), dict(src=i32([])), dict(t=t[0]), dict(pinned=i32([]))):
        with pytest.raises(ValueError):
            fork(**kw)
    for kw in (dict(out=t), dict(cout=c)):
        with pytest.raises(fp4idx.Fp4IdxError):
            fork(**kw)
    ws = torch.empty(fp4idx.compact_pages_workspace_bytes(8), dtype=torch.uint8, device="cuda")
    pack = lambda out=out, ws=ws, dst=two: fp4idx.compact_pages(t, c, 1, 8, ws, free, out, one, dst, counts)  # noqa: E731
    pack()
    for kw in (dict(out=t), dict(ws=ws[:-4].clone())):
        with pytest.raises(fp4idx.Fp4IdxError):
            pack(**kw)
    with pytest.raises(ValueError):
        pack(dst=i32([]))
