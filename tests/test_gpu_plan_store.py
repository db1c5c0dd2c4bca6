"""Step plan and latent store against plain references (integers; float64)."""
import random

import pytest
import torch

from tests import latent_ref as ref

pytestmark = pytest.mark.gpu

NAMES = ("q_positions", "row_seq", "context_lens", "store_positions", "store_slots", "cu_rows", "cu_context", "counts")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def run_plan(cached, new, ratio, free, table, max_rows, max_stores, head=None, stream=None):
    from sparse_attention_fp4_gb300 import fp4idx
    B = len(cached)
    sizes = (max_rows, max_rows, max_rows, max_stores, max_stores, B + 1, B + 1, 4)
    out = [torch.full((n + 3,), -77, dtype=torch.int32, device="cuda")[:n] for n in sizes]
    t = i32(table).view(B, -1) if B else torch.empty((0, 1), dtype=torch.int32, device="cuda")
    status = i32([0])
    args = (i32(cached), i32(new), ratio, i32(free), t, *out)
    fp4idx.plan_step(*args, free_head=None if head is None else i32([head]), status=status, stream=stream)
    fp4idx.plan_step(*args, free_head=None if head is None else i32([head]), status=status, stream=stream)  # repeated: the same
    got = {n: v.tolist() for n, v in zip(NAMES, out)}
    got["table"] = t.tolist()
    assert all(int(v._base[n:].min()) == -77 == int(v._base[n:].max()) for v, n in zip(out, sizes))
    return got, fp4idx.read_status(status)


def case(seed, B, lo, hi, new_hi, ratio, max_pages):
    r = random.Random(seed)
    cached = [r.randrange(lo, hi + 1) for _ in range(B)]
    new = [r.randrange(0, new_hi + 1) for _ in range(B)]
    ids = list(range(B * max_pages + B * (new_hi // 64 + 2)))
    r.shuffle(ids)
    table = []
    for b in range(B):
        held = -(-(cached[b] // ratio) // 64)
        table.append([ids.pop() if j < held else -5 for j in range(max_pages)])
    return cached, new, ids, table


@pytest.mark.parametrize("B,lo,hi,new_hi,ratio,max_pages", [
    (1, 0, 0, 1, 1, 2), (1, 63, 63, 2, 1, 4), (1, 64, 64, 1, 1, 4), (3, 0, 300, 0, 4, 4), (64, 500, 3000, 1, 4, 20),
    (64, 0, 130, 70, 1, 8), (1023, 0, 20, 3, 2, 3), (1024, 0, 200, 1, 1, 5), (1025, 0, 200, 5, 3, 5),
    (2500, 0, 64, 9, 1, 3), (7, 0, 6000, 3000, 1, 160), (2, 0, 40000, 9000, 64, 20)])
def test_plan(B, lo, hi, new_hi, ratio, max_pages):
    cached, new, free, table = case(B * 7 + ratio, B, lo, hi, new_hi, ratio, max_pages)
    rows = sum(new) + 5
    stores = sum((c + n) // ratio - c // ratio for c, n in zip(cached, new)) + 3
    for head in (None, 2):
        want = ref.plan(cached, new, ratio, free, head or 0, [list(t) for t in table], rows, stores)
        got, status = run_plan(cached, new, ratio, free, table, rows, stores, head)
        assert status == 0 and not want["full"]
        for n in NAMES + ("table",):
            assert got[n] == want[n], n


@pytest.mark.parametrize("rows,stores,pages", [(0, 100, 100), (40, 1000, 100), (1000, 17, 100), (1000, 1000, 1), (1000, 1000, 0)])
def test_plan_out_of_capacity(rows, stores, pages):
    """The sequences that fit are planned; the first that does not, and all behind it, get nothing."""
    cached, new, free, table = case(5, 40, 0, 200, 40, 2, 6)
    want = ref.plan(cached, new, 2, free[:pages], 0, [list(t) for t in table], rows, stores)
    got, status = run_plan(cached, new, 2, free[:pages], table, rows, stores)
    assert want["full"] and status == 11
    for n in NAMES + ("table",):
        assert got[n] == want[n], n


def test_plan_bad_lengths():
    """A sequence with a bad length gets nothing; those around it are planned."""
    cached = [10, -1, 20, 5, 300, 2 ** 31 - 2, 7]
    new = [3, 1, -2, 1, 100, 5, 2]
    table = [[100 + 10 * b + j if j < -(-max(0, min(c, 300)) // 64) else -1 for j in range(6)] for b, c in enumerate(cached)]
    free = list(range(20))
    want = ref.plan(cached, new, 1, free, 0, [list(t) for t in table], 30, 30)
    got, status = run_plan(cached, new, 1, free, table, 30, 30)
    assert want["bad"] and not want["full"] and status == 8
    for n in NAMES + ("table",):
        assert got[n] == want[n], n


def test_plan_bad_page_and_head():
    # the page of the existing entries is missing: slots -1, BAD_PAGE
    got, status = run_plan([10], [4], 1, [3], [[-1, -1]], 4, 4)
    assert status == 5 and got["store_slots"] == [-1] * 4 and got["q_positions"] == [10, 11, 12, 13]
    # a page id whose slots would not fit in 32 bits
    got, status = run_plan([0], [2], 1, [1 << 25], [[-1]], 2, 2)
    assert status == 5 and got["store_slots"] == [-1, -1]
    for head in (-1, 5):  # outside the list: nothing to take
        got, status = run_plan([0, 64], [1, 0], 1, [1, 2, 3], [[-1, -1], [9, -1]], 2, 2, head)
        assert status == 11 and got["counts"] == [0, 0, 0, 0] and got["table"] == [[-1, -1], [9, -1]]


def test_plan_nothing():
    got, status = run_plan([], [], 1, [], [], 3, 2)
    assert status == 0 and got["context_lens"] == [0, 0, 0] and got["store_slots"] == [-1, -1]
    assert got["cu_rows"] == [0] and got["cu_context"] == [0] and got["counts"] == [0, 0, 0, 0]


def cos_sin_table(n):
    f = 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
    a = torch.arange(n, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).to(torch.bfloat16).cuda()


def store_inputs(n, width, pages, seed):
    g = torch.Generator().manual_seed(seed)
    kv = (torch.randn((n, width), generator=g) * 3).to(torch.bfloat16).cuda()
    kv[n // 2] = 0
    w = (1 + 0.1 * torch.randn(512, generator=g)).to(torch.bfloat16).cuda()
    pos = torch.randint(0, 5000, (n,), generator=g).to(torch.int32).cuda()
    slots = torch.randperm(pages * 64, generator=g)[:n].to(torch.int32).cuda()
    return kv, w, pos, slots


@pytest.mark.parametrize("n,width", [(1, 512), (1, 576), (2, 576), (7, 512), (63, 576), (513, 512), (3001, 576)])
def test_store_latent(n, width):
    from sparse_attention_fp4_gb300 import fp4idx
    pages = 60
    kv, w, pos, slots = store_inputs(n, width, pages, n)
    cs = cos_sin_table(5000)
    cache = torch.full((pages, 64, width), 7.5, dtype=torch.bfloat16, device="cuda")
    status = i32([0])
    skipped = []
    if n > 5:  # padding, a slot past the cache, positions outside the table
        slots[1], slots[2], pos[3], pos[4] = -1, pages * 64, -1, 5000
        skipped = [1, 2, 3, 4]
    fp4idx.store_latent(kv, pos, slots, w, 1e-6, cs, cache, status=status)
    assert fp4idx.read_status(status) in ((5, 7) if skipped else (0,))
    keep = [i for i in range(n) if i not in skipped]
    want, tol = ref.store(kv[keep], pos[keep], w, 1e-6, cs)
    flat = cache.view(-1, width)
    got = flat[slots[keep].long()].double()
    assert bool(((got - want).abs() <= tol).all()), float((got - want).abs().max())
    rest = torch.ones(pages * 64, dtype=torch.bool, device="cuda")
    rest[slots[keep].long()] = False
    assert bool((flat[rest] == 7.5).all())


def test_store_latent_far_slots():
    """Slots whose element offset passes 32 bits."""
    from sparse_attention_fp4_gb300 import fp4idx
    pages, width = 120000, 576  # 4.4e9 elements
    kv, w, pos, slots = store_inputs(9, width, 10, 3)
    slots = torch.arange(9, dtype=torch.int32, device="cuda") * 3 + pages * 64 - 40
    cs = cos_sin_table(5000)
    cache = torch.empty((pages, 64, width), dtype=torch.bfloat16, device="cuda")
    cache[-1].fill_(1)
    fp4idx.store_latent(kv, pos, slots, w, 1e-6, cs, cache)
    want, tol = ref.store(kv, pos, w, 1e-6, cs)
    got = cache.view(-1, width)[slots.long()].double()
    assert bool(((got - want).abs() <= tol).all())
