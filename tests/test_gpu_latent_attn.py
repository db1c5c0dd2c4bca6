"""Absorbed latent attention (selected tokens, whole context, drafted trees) against the
formula in float64, row by row."""
import math
import random

import pytest
import torch

from tests import latent_ref as ref

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Batch:
    """Rows over a paged cache; every page that no sequence owns, and every token behind a
    sequence's end, holds NaN."""

    def __init__(self, seed, lens, rows_per_seq, heads, width, qscale=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = random.Random(seed)
        self.lens, self.n, self.H, self.width = lens, rows_per_seq, heads, width
        B = len(lens)
        pages = [max(1, -(-v // 64)) for v in lens]
        pool = sum(pages) + 5
        ids = list(range(pool))
        r.shuffle(ids)
        most = max(pages) + 1
        table, owned = [], torch.zeros((pool, 64), dtype=torch.bool)
        for b in range(B):
            mine = [ids.pop() for _ in range(pages[b])]
            for s in range(lens[b]):
                owned[mine[s // 64], s % 64] = True
            table.append(mine + [-1] * (most - pages[b]))
        self.cache = torch.randn((pool, 64, width), generator=g, device="cuda").to(torch.bfloat16)
        self.cache[~owned.cuda()] = math.nan
        self.table = i32(table)
        T = B * rows_per_seq
        self.T = T
        self.row_seq = i32([b for b in range(B) for _ in range(rows_per_seq)])
        self.q = (qscale * torch.randn((T, heads, width), generator=g, device="cuda")).to(torch.bfloat16)
        self.scale = 192 ** -0.5

    def buffers(self):
        out = torch.full((self.T + 1, self.H, 512), 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.T + 1, self.H), 3.0, dtype=torch.float32, device="cuda")
        return out, lse

    def row(self, t, positions):
        k = ref.tokens(self.cache, self.table[int(self.row_seq[t])], positions)
        return ref.attend(self.q[t].double(), k, k[:, :512], self.scale)

    def check(self, out, lse, positions, rows=None):
        for t in range(self.T) if rows is None else rows:
            ref.check(out[t], None if lse is None else lse[t], self.row(t, positions[t]), "row %d" % t)
        assert bool((out[self.T:] == 3).all()) and (lse is None or bool((lse[self.T:] == 3).all()))


def workspace(b):
    from sparse_attention_fp4_gb300 import fp4idx
    return torch.full((fp4idx.latent_attn_workspace_bytes(b.T, b.H),), 0xFF, dtype=torch.uint8, device="cuda")


def selection(b, k, seed, lens):
    r = random.Random(seed)
    idx, want = [], []
    for t in range(b.T):
        L = lens[t]
        pick = sorted(r.sample(range(L), min(k, L)))
        want.append(pick)
        idx.append(pick + [-1] * (k - len(pick)))
    return i32(idx), want


@pytest.mark.parametrize("heads,width", [(64, 512), (64, 576), (128, 576), (16, 512), (1, 576), (5, 512), (40, 576), (100, 512), (8, 576)])
@pytest.mark.parametrize("lens,n,k", [([1], 1, 1), ([200, 0, 63, 64, 65], 1, 64), ([700, 3], 3, 130), ([2500], 1, 2048)])
def test_selected(heads, width, lens, n, k):
    from sparse_attention_fp4_gb300 import fp4idx
    b = Batch(heads + width + k, lens, n, heads, width)
    idx, want = selection(b, k, 1, [v for v in lens for _ in range(n)])
    ws, status = workspace(b), i32([0])
    for ctx in (None, i32([min(len(p), k) for p in want])):
        out, lse = b.buffers()
        fp4idx.latent_attn_topk(b.q, b.cache, b.table, b.row_seq, idx, b.scale, ws, out, lse=lse, context_lens=ctx, status=status)
        b.check(out, lse, want)
    out, _ = b.buffers()
    fp4idx.latent_attn_topk(b.q, b.cache, b.table, b.row_seq, idx, b.scale, ws, out, status=status)
    b.check(out, None, want)
    assert fp4idx.read_status(status) == 0


def test_selected_gaps_duplicates_order():
    """Entries < 0 anywhere are skipped, a position listed twice counts twice, any order."""
    from sparse_attention_fp4_gb300 import fp4idx
    b = Batch(3, [500, 90, 300], 1, 16, 512)
    k = 150
    r = random.Random(5)
    want, idx = [], []
    for L in b.lens:
        row = [r.randrange(L) if r.random() < 0.6 else -r.randrange(1, 9) for _ in range(k)]
        if L == 300:
            row[:70] = [-1] * 70  # a whole tile of nothing first
        idx.append(row)
        want.append([p for p in row if p >= 0])
    out, lse = b.buffers()
    fp4idx.latent_attn_topk(b.q, b.cache, b.table, b.row_seq, i32(idx), b.scale, workspace(b), out, lse=lse)
    b.check(out, lse, want)


def test_selected_bad_entries():
    """Bad positions and pages are skipped and reported; a bad sequence leaves the row empty."""
    from sparse_attention_fp4_gb300 import fp4idx
    b = Batch(4, [400, 400, 400], 1, 8, 576)
    idx, want = selection(b, 100, 2, b.lens)
    idx[0, 7] = b.table.shape[1] * 64            # past the table
    want[0].pop(7)
    gone = want[1][50] // 64
    b.table[1, gone] = b.cache.shape[0]          # a page outside the cache
    want[1] = [p for p in want[1] if p // 64 != gone]
    seqs = b.row_seq.clone()
    seqs[2] = 3
    want[2] = []
    for rows, code in (((0,), 8), ((1,), 5), ((2,), 5)):
        status = i32([0])
        out, lse = b.buffers()
        sel = torch.full_like(idx, -1)
        for t in rows:
            sel[t] = idx[t]
        fp4idx.latent_attn_topk(b.q, b.cache, b.table, seqs if 2 in rows else b.row_seq, sel, b.scale, workspace(b), out, lse=lse, status=status)
        b.check(out, lse, [want[t] if t in rows else [] for t in range(3)])
        assert fp4idx.read_status(status) == code


@pytest.mark.parametrize("heads,width", [(16, 576), (64, 512), (128, 576), (1, 512), (24, 512), (8, 576)])
@pytest.mark.parametrize("lens,n", [([1], 1), ([0, 1, 63, 64, 65, 129], 1), ([300, 700], 3), ([5000], 1), ([17, 0, 900], 9)])
def test_whole_context(heads, width, lens, n):
    from sparse_attention_fp4_gb300 import fp4idx
    b = Batch(heads + width + n, lens, n, heads, width)
    # rows of one sequence see different lengths, the longest the whole of it
    L = [max(0, v - (n - 1 - i)) for v in lens for i in range(n)]
    status = i32([0])
    out, lse = b.buffers()
    fp4idx.latent_attn(b.q, b.cache, b.table, b.row_seq, i32(L), max(lens), b.scale, workspace(b), out, lse=lse, status=status)
    b.check(out, lse, [list(range(v)) for v in L])
    assert fp4idx.read_status(status) == 0


@pytest.mark.parametrize("heads,width", [(16, 512), (8, 576), (64, 576), (128, 512), (3, 576)])
@pytest.mark.parametrize("prefix,n,words", [([0], 1, 1), ([100, 0, 64, 63], 13, 1), ([1000, 30], 32, 1), ([65, 200], 45, 2), ([10], 100, 8)])
def test_tree(heads, width, prefix, n, words):
    from sparse_attention_fp4_gb300 import fp4idx
    b = Batch(heads + n, [p + n for p in prefix], n, heads, width)
    r = random.Random(n)
    masks, want = [], []
    for p in prefix:
        up = [-1] + [r.randrange(i) for i in range(1, n)]
        for i in range(n):
            path, j = 0, i
            while j >= 0:
                path |= 1 << j
                j = up[j]
            masks.append(path)
            want.append(list(range(p)) + [p + j for j in range(n) if path >> j & 1])
    packed = [[(m >> 32 * w) & 0xFFFFFFFF for w in range(words)] for m in masks]
    tree = i32([[v - (1 << 32) if v >> 31 else v for v in row] for row in packed])
    ctx = i32([p for p in prefix for _ in range(n)])
    status = i32([0])
    out, lse = b.buffers()
    fp4idx.latent_attn(b.q, b.cache, b.table, b.row_seq, ctx, max(prefix) + n, b.scale, workspace(b), out, lse=lse, tree_mask=tree, status=status)
    b.check(out, lse, want)
    assert fp4idx.read_status(status) == 0


def test_tree_without_any_token():
    """Context length 0 and an empty mask: the row is empty, whatever its neighbours see."""
    from sparse_attention_fp4_gb300 import fp4idx
    b = Batch(8, [20, 20], 4, 16, 512)
    ctx = i32([0, 0, 0, 0, 5, 0, 5, 0])
    tree = i32([[0], [1 << 3], [0], [-(1 << 31) + 0], [0], [0], [6], [0]])
    tree[3, 0] = 1 << 19
    want = [[], [3], [], [19], list(range(5)), [], list(range(5)) + [6, 7], []]
    out, lse = b.buffers()
    fp4idx.latent_attn(b.q, b.cache, b.table, b.row_seq, ctx, 25, b.scale, workspace(b), out, lse=lse, tree_mask=tree)
    b.check(out, lse, want)


def test_masked_draft_is_nan():
    """A drafted token that holds NaN reaches the rows that see it and no other."""
    from sparse_attention_fp4_gb300 import fp4idx
    b = Batch(9, [70 + 6], 6, 8, 576)
    b.cache[int(b.table[0, 1]), (70 + 2) % 64] = math.nan
    b.cache[int(b.table[0, 1]), (70 + 4) % 64, 3] = math.inf
    masks = [0b000001, 0b000011, 0b000101, 0b001011, 0b010011, 0b100001]
    want = [list(range(70)) + [70 + j for j in range(6) if m >> j & 1] for m in masks]
    out, lse = b.buffers()
    fp4idx.latent_attn(b.q, b.cache, b.table, b.row_seq, i32([70] * 6), 76, b.scale, workspace(b), out, lse=lse, tree_mask=i32([[m] for m in masks]))
    b.check(out, lse, want, rows=(0, 1, 3, 5))
    assert bool(out[2].isnan().all()) and bool(lse[2].isnan().all())


def test_whole_context_bad_rows():
    """A bad length, sequence or page is reported; other rows are not touched by it."""
    from sparse_attention_fp4_gb300 import fp4idx
    b = Batch(10, [200, 200, 200, 200], 1, 16, 512)
    tree = i32([[0], [0], [0], [1 << 30]])
    good = list(range(150))
    for ctx, seqs, code, empty in (([150, -1, 150, 0], [0, 1, 2, 3], 8, (1,)), ([150, 201, 150, 0], [0, 1, 2, 3], 8, (1,)),
                                   ([150, 150, 150, 180], [0, 1, 2, 3], 8, (3,)), ([150, 150, 150, 0], [0, -1, 2, 3], 5, (1,)),
                                   ([150, 150, 150, 0], [0, 4, 2, 3], 5, (1,))):
        status = i32([0])
        out, lse = b.buffers()
        fp4idx.latent_attn(b.q, b.cache, b.table, i32(seqs), i32(ctx), 200, b.scale, workspace(b), out, lse=lse, tree_mask=tree, status=status)
        want = [good, good, good, [30]]
        for t in empty:
            want[t] = []
        b.check(out, lse, want)
        assert fp4idx.read_status(status) == code
    table = b.table.clone()
    table[2, 1] = -1
    status = i32([0])
    out, lse = b.buffers()
    fp4idx.latent_attn(b.q, b.cache, table, b.row_seq, i32([150] * 4), 200, b.scale, workspace(b), out, lse=lse, status=status)
    b.check(out, lse, [good, good, [p for p in good if p // 64 != 1], good])
    assert fp4idx.read_status(status) == 5


def test_large_scores_and_growing_maximum():
    """Scores in the hundreds whose maximum grows from tile to tile."""
    from sparse_attention_fp4_gb300 import fp4idx
    b = Batch(11, [1000], 1, 16, 576, qscale=4.0)
    ramp = torch.linspace(0.05, 4.0, 1000, device="cuda")
    at = torch.arange(1000, device="cuda")
    pages = b.table[0].long()[at // 64]
    b.cache[pages, at % 64] = (b.q[0, 3].float()[None, :] * ramp[:, None] * 0.5).to(torch.bfloat16)
    out, lse = b.buffers()
    fp4idx.latent_attn(b.q, b.cache, b.table, b.row_seq, i32([1000]), 1000, b.scale, workspace(b), out, lse=lse)
    b.check(out, lse, [list(range(1000))])
    assert float(lse[0, 3]) > 300


def test_far_pages():
    """Pages whose element offset passes 32 bits, 70,000 tokens, scores split over the card."""
    from sparse_attention_fp4_gb300 import fp4idx
    g = torch.Generator(device="cuda").manual_seed(1)
    pages, width, H, L = 120000, 576, 16, 70001
    cache = torch.empty((pages, 64, width), dtype=torch.bfloat16, device="cuda")
    need = -(-L // 64)
    ids = pages - 1 - 2 * torch.arange(need, device="cuda")
    cache[ids] = torch.randn((need, 64, width), generator=g, device="cuda").to(torch.bfloat16)
    cache[ids[-1], L % 64:] = math.nan
    table = ids.to(torch.int32)[None, :].contiguous()
    q = torch.randn((1, H, width), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty((1, H, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((1, H), dtype=torch.float32, device="cuda")
    ws = torch.empty(fp4idx.latent_attn_workspace_bytes(1, H), dtype=torch.uint8, device="cuda")
    fp4idx.latent_attn(q, cache, table, i32([0]), i32([L]), L, 192 ** -0.5, ws, out, lse=lse)
    k = ref.tokens(cache, table[0], torch.arange(L, device="cuda"))
    ref.check(out[0], lse[0], ref.attend(q[0].double(), k, k[:, :512], 192 ** -0.5), "whole")
    pick = torch.arange(0, L, 41, device="cuda").to(torch.int32)[None, :].contiguous()
    fp4idx.latent_attn_topk(q, cache, table, i32([0]), pick, 192 ** -0.5, ws, out, lse=lse)
    k = k[pick[0].long()]
    ref.check(out[0], lse[0], ref.attend(q[0].double(), k, k[:, :512], 192 ** -0.5), "picked")


def test_graph_stream_and_repeat():
    """Captured and replayed on another stream with changed inputs; the same bits each time."""
    from sparse_attention_fp4_gb300 import fp4idx
    b = Batch(12, [900, 300, 77], 2, 32, 512)
    k = 200
    L = [v for v in b.lens for _ in range(2)]
    idx, want = selection(b, k, 4, L)
    ws = workspace(b)
    out, lse = b.buffers()
    out2, lse2 = b.buffers()
    ctx = i32(L)

    def both():
        fp4idx.latent_attn_topk(b.q, b.cache, b.table, b.row_seq, idx, b.scale, ws, out, lse=lse)
        fp4idx.latent_attn(b.q, b.cache, b.table, b.row_seq, ctx, 900, b.scale, ws, out2, lse=lse2)
    both()
    torch.cuda.synchronize()
    first = [v.clone() for v in (out, lse, out2, lse2)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        both()
    for v in (out, lse, out2, lse2):
        v[: b.T].zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(3):
            graph.replay()
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, (out, lse, out2, lse2)))
    idx2, want2 = selection(b, k, 5, L)
    idx.copy_(idx2)
    ctx.copy_(i32([v // 2 for v in L]))
    graph.replay()
    torch.cuda.synchronize()
    b.check(out, lse, want2)
    b.check(out2, lse2, [list(range(v // 2)) for v in L])


def test_many_rows():
    """More rows than the card holds at once; a sample is checked, and every row against the
    selection of everything."""
    from sparse_attention_fp4_gb300 import fp4idx
    lens = [64 + 3 * i for i in range(120)]
    b = Batch(13, lens, 5, 16, 576)
    L = [v for v in lens for _ in range(5)]
    k = max(lens)
    idx = i32([list(range(v)) + [-1] * (k - v) for v in L])
    ws = workspace(b)
    out, lse = b.buffers()
    out2, lse2 = b.buffers()
    fp4idx.latent_attn_topk(b.q, b.cache, b.table, b.row_seq, idx, b.scale, ws, out, lse=lse)
    fp4idx.latent_attn(b.q, b.cache, b.table, b.row_seq, i32(L), k, b.scale, ws, out2, lse=lse2)
    b.check(out, lse, [list(range(v)) for v in L], rows=range(0, b.T, 37))
    b.check(out2, lse2, [list(range(v)) for v in L], rows=range(5, b.T, 41))
    # both are within the bound of the exact value, so within twice the bf16 step of each other
    assert float((out[: b.T].float() - out2[: b.T].float()).abs().max()) <= 0.05
    assert float((lse[: b.T] - lse2[: b.T]).abs().max()) <= 1e-3


def test_no_rows():
    from sparse_attention_fp4_gb300 import fp4idx
    b = Batch(14, [64], 1, 16, 512)
    e = torch.empty((0, 16, 512), dtype=torch.bfloat16, device="cuda")
    ws = workspace(b)
    fp4idx.latent_attn_topk(e, b.cache, b.table, i32([]), torch.empty((0, 8), dtype=torch.int32, device="cuda"), 1.0, ws, e)
    fp4idx.latent_attn(e, b.cache, b.table, i32([]), i32([]), 64, 1.0, ws, e)


def test_binding_refusals():
    from sparse_attention_fp4_gb300 import fp4idx
    b = Batch(15, [64], 1, 16, 512)
    ws = workspace(b)
    out, lse = b.buffers()
    idx = i32([[0, 1]])
    ok = dict(q=b.q, cache=b.cache, page_table=b.table, row_seq=b.row_seq, topk_idx=idx, scale=1.0, workspace=ws, out=out)
    for key, bad in (("q", b.q[:, :, :500]), ("q", b.q.float()), ("q", b.q.cpu()), ("cache", b.cache[:, :32]),
                     ("page_table", b.table[0]), ("row_seq", b.row_seq.long()), ("topk_idx", idx.t().contiguous()),
                     ("out", out[:0]), ("topk_idx", idx.expand(1, 2).cpu()), ("q", b.q.transpose(1, 2))):
        with pytest.raises(ValueError):
            fp4idx.latent_attn_topk(**{**ok, key: bad})
    with pytest.raises(fp4idx.Fp4IdxError):
        fp4idx.latent_attn_topk(**{**ok, "workspace": ws[:16]})
    with pytest.raises(ValueError):
        fp4idx.latent_attn(b.q, b.cache, b.table, b.row_seq, i32([64]), 64, 1.0, ws, out, tree_mask=i32([1]))
