"""Pieces of a unit are joined whole: inputs whose result shows a piece that is lost, doubled or
weighted wrongly, however long the context is.

The 64-token tiles of a sequence are marked: a token's latent row is 1 in its tile's dim (the
tiles are spread over the 512 value dims in order) and 0 elsewhere.  A query holds a whole number
at every dim, which is then the score of that dim's tokens (in units of ln 2), so that
  out[d] = count[d] 2^n[d] / sum,  lse = log(sum),  sum = sum_d count[d] 2^n[d]
and a tile that is missing takes a third or more of its dim's output away."""
import math
import random

import pytest
import torch

BF16 = torch.finfo(torch.bfloat16).eps / 2
NAN = float("nan")
LN2 = math.log(2.0)


def dims_of_tiles(length):
    """The dim of each tile; at most three tiles share one up to 98,304 tokens."""
    tiles = -(-length // 64)
    j = torch.arange(tiles)
    return j if tiles <= 512 else j * 512 // tiles


def profile(heads, kind):
    """The queries' whole numbers [heads, 512]: 0, or 0..14 in an order of each head's own."""
    if kind == "even":
        return torch.zeros((heads, 512), dtype=torch.float64)
    d, h = torch.arange(512), torch.arange(heads)[:, None]
    return ((d * d * 7 + h * 11 + d // 37) % 15).double()


def counts(dims, positions):
    return torch.bincount(dims[positions // 64], minlength=512).double()


def expected(n, count):
    """out [heads, 512] and lse [heads], and their bounds.

    A score is one product and exact.  Its exponent n scale log2(e) - m has three roundings of
    the factors and one of the fused product, each 2^-24 of at most 14: a weight is off by
    14 4 2^-24 ln 2 < 2^-18, the exponential by 2^-21.  A weight is 2^integer up to that, so its
    rounding to bf16 leaves 2^integer.  Up to three factors 2^(m - m') are off alike, and the sums
    (at most 300 additions in a row, of positive terms) by 300 2^-24: together below 2^-15.
    Without scores all weights are 1, all sums whole numbers below 2^24, and only the division,
    the product and the logarithm are rounded."""
    w = count * torch.exp2(n)
    total = w.sum(1, keepdim=True)
    even = bool((n == 0).all())
    out = w / total
    lse = torch.log(total).squeeze(1)
    return out, lse, (BF16 + (2.0 ** -22 if even else 2.0 ** -15)) * out, 2.0 ** -20 * lse.abs() + (0.0 if even else 2.0 ** -15)


def holds(out, lse, want):
    o, l, tol, tol_l = want
    return bool(((out.double() - o).abs() <= tol).all()) and bool(((lse.double() - l).abs() <= tol_l).all())


@pytest.mark.parametrize("kind", ["even", "scores"])
@pytest.mark.parametrize("length,pieces", [(70001, 152), (70001, 76), (9000, 16), (17001, 10), (4000, 2)])
def test_bounds_show_a_wrong_piece(kind, length, pieces):
    """(CPU) A result without a piece, or with one twice, is outside the bounds; the right one, rounded, is within."""
    dims, n = dims_of_tiles(length), profile(3, kind)
    at = torch.arange(length)
    whole = counts(dims, at)
    want = expected(n, whole)
    assert holds(want[0].float().to(torch.bfloat16), want[1].float(), want)
    tiles = dims.numel()
    for i in range(pieces):
        t0, t1 = tiles * i // pieces, tiles * (i + 1) // pieces
        part = counts(dims, at[t0 * 64:t1 * 64])
        for wrong in (whole - part, whole + part):
            out, lse, _, _ = expected(n, wrong)
            assert not holds(out.float().to(torch.bfloat16), lse.float(), want)
            # the sum right and the output not, and the other way round
            assert not holds(out.float().to(torch.bfloat16), want[1].float(), want)
    # one tile of 64 tokens
    out, lse, _, _ = expected(n, whole - counts(dims, at[64 * 5:64 * 6]))
    assert not holds(out.float().to(torch.bfloat16), lse.float(), want)


class Marked:
    def __init__(self, seed, lens, heads, width, kind):
        r = random.Random(seed)
        pages = [max(1, -(-v // 64)) for v in lens]
        ids = list(range(sum(pages) + 3))
        r.shuffle(ids)
        self.cache = torch.full((len(ids), 64, width), NAN, dtype=torch.bfloat16, device="cuda")
        table = torch.full((len(lens), max(pages)), -1, dtype=torch.int32)
        self.dims, self.lens = [dims_of_tiles(v) for v in lens], lens
        for b, v in enumerate(lens):
            mine = [ids.pop() for _ in range(pages[b])]
            table[b, :pages[b]] = torch.tensor(mine)
            if v == 0:
                continue
            at = torch.tensor(mine, device="cuda")
            self.cache[at] = 0
            self.cache[at, :, self.dims[b].cuda()] = 1
            if v % 64:
                self.cache[mine[-1], v % 64:] = NAN
        self.table = table.cuda()
        self.heads, self.width, self.n = heads, width, profile(heads, kind)

    def queries(self, rows):
        q = torch.zeros((rows, self.heads, self.width), dtype=torch.bfloat16)
        q[:, :, :512] = self.n
        return q.cuda()

    def buffers(self, rows):
        from sparse_attention_fp4_gb300 import fp4idx
        ws = torch.full((fp4idx.latent_attn_workspace_bytes(rows, self.heads),), 0xFF, dtype=torch.uint8, device="cuda")
        out = torch.full((rows, self.heads, 512), NAN, dtype=torch.bfloat16, device="cuda")
        return ws, out, torch.full((rows, self.heads), NAN, dtype=torch.float32, device="cuda")

    def check(self, out, lse, seqs, positions):
        out, lse = out.cpu(), lse.cpu()
        for t, (b, p) in enumerate(zip(seqs, positions)):
            if p.numel() == 0:
                assert bool((out[t] == 0).all()) and bool((lse[t] == -math.inf).all()), t
            else:
                assert holds(out[t], lse[t], expected(self.n, counts(self.dims[b], p))), "row %d" % t


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["even", "scores"])
@pytest.mark.parametrize("lens,rows,heads,width", [
    ([70001], 1, 128, 576), ([45000], 1, 16, 512), ([33000], 1, 64, 576), ([50000], 3, 8, 576), ([40001, 0, 35000], 1, 40, 512),  # many pieces a unit
    ([17001 + 64 * i for i in range(15)], 1, 64, 576),
    ([5000 + 61 * i for i in range(40)], 1, 32, 512), ([100 + 19 * i for i in range(200)], 1, 64, 576),                            # a few
    ([900 + 7 * i for i in range(90)], 4, 16, 512),
    ([9000], 1, 64, 576), ([2000, 1999, 70, 1], 1, 128, 512), ([1500], 5, 8, 576), ([640] * 30, 1, 16, 512)])                     # clusters
def test_whole_contexts(lens, rows, heads, width, kind):
    from sparse_attention_fp4_gb300 import fp4idx
    m = Marked(len(lens) + heads, lens, heads, width, kind)
    seqs = [b for b in range(len(lens)) for _ in range(rows)]
    L = [max(0, lens[b] - (rows - 1 - i)) for b in range(len(lens)) for i in range(rows)]
    ws, out, lse = m.buffers(len(seqs))
    status = i32([0])
    fp4idx.latent_attn(m.queries(len(seqs)), m.cache, m.table, i32(seqs), i32(L), max(lens), LN2, ws, out, lse=lse, status=status)
    assert fp4idx.read_status(status) == 0
    m.check(out, lse, seqs, [torch.arange(v) for v in L])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["even", "scores"])
@pytest.mark.parametrize("seqs,rows,heads,k", [(1, 1, 128, 4096), (1, 1, 16, 4000), (9, 1, 64, 2048), (100, 1, 64, 4096), (61, 2, 128, 1111), (40, 10, 16, 700)])
def test_selections(seqs, rows, heads, k, kind):
    from sparse_attention_fp4_gb300 import fp4idx
    r = random.Random(k)
    lens = [k // 2 + 17 * i for i in range(seqs)] if seqs > 1 else [20000]
    m = Marked(seqs + k, lens, heads, 512, kind)
    of = [b for b in range(seqs) for _ in range(rows)]
    pick = [torch.tensor(sorted(r.sample(range(lens[b]), min(k, lens[b])))) for b in of]
    idx = torch.full((len(of), k), -1, dtype=torch.int32)
    for t, p in enumerate(pick):
        idx[t, :p.numel()] = p
    ws, out, lse = m.buffers(len(of))
    status = i32([0])
    fp4idx.latent_attn_topk(m.queries(len(of)), m.cache, m.table, i32(of), idx.cuda(), LN2, ws, out, lse=lse, status=status)
    assert fp4idx.read_status(status) == 0
    m.check(out, lse, of, pick)
