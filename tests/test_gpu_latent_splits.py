"""Row counts around every way the attention work is cut (clusters, CTAs of a unit's own,
whole rounds, an even cut), and the bounded waits of the attention kernels."""
import pytest
import torch

from tests.test_gpu_latent_attn import Batch, i32, selection, workspace
from tests.test_gpu_latent_prefill import Prompts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [2, 19, 38, 39, 76, 77, 100, 151, 152, 153, 200, 304, 305, 460])
@pytest.mark.parametrize("heads,k", [(8, 300), (70, 130)])
def test_selected_rows(rows, heads, k):
    from sparse_attention_fp4_gb300 import fp4idx
    lens = [1 + (37 * i) % 500 for i in range(rows)]
    b = Batch(rows, lens, 1, heads, 512)
    idx, want = selection(b, k, 2, lens)
    status = i32([0])
    out, lse = b.buffers()
    fp4idx.latent_attn_topk(b.q, b.cache, b.table, b.row_seq, idx, b.scale, workspace(b), out, lse=lse, status=status)
    assert fp4idx.read_status(status) == 0
    b.check(out, lse, want, rows=range(0, rows, 1 + rows // 60))


@pytest.mark.parametrize("seqs,n", [(1, 1), (3, 5), (40, 1), (40, 4), (152, 1), (153, 1), (200, 2), (64, 7)])
@pytest.mark.parametrize("heads", [8, 24, 64])
def test_whole_context_rows(seqs, n, heads):
    from sparse_attention_fp4_gb300 import fp4idx
    lens = [(i * i * 13) % 900 for i in range(seqs)]
    lens[0] = 1500
    b = Batch(seqs, lens, n, heads, 576)
    L = [max(0, v - (n - 1 - i)) for v in lens for i in range(n)]
    status = i32([0])
    out, lse = b.buffers()
    fp4idx.latent_attn(b.q, b.cache, b.table, b.row_seq, i32(L), 1500, b.scale, workspace(b), out, lse=lse, status=status)
    assert fp4idx.read_status(status) == 0
    b.check(out, lse, [list(range(v)) for v in L], rows=range(0, b.T, 1 + b.T // 60))


def test_rows_of_mixed_sequences():
    """Runs of one sequence of every length up to more than a pass holds, sequences that come
    back, and rows of a bad sequence between them."""
    from sparse_attention_fp4_gb300 import fp4idx
    b = Batch(3, [200, 300, 70], 12, 8, 512)
    seqs = [0] * 3 + [1] * 11 + [0] + [2] * 2 + [5] * 2 + [1] + [2] * 9 + [0] * 7
    L = [(i * 53) % 70 + 1 for i in range(len(seqs))]
    assert len(seqs) == b.T
    b.row_seq = i32([s if s < 3 else 0 for s in seqs])
    status = i32([0])
    out, lse = b.buffers()
    fp4idx.latent_attn(b.q, b.cache, b.table, i32(seqs), i32(L), 80, b.scale, workspace(b), out, lse=lse, status=status)
    assert fp4idx.read_status(status) == 5
    b.check(out, lse, [list(range(v)) if s < 3 else [] for v, s in zip(L, seqs)])


def test_same_bits_every_time():
    """Pieces are joined in a fixed order, whatever runs beside them."""
    from sparse_attention_fp4_gb300 import fp4idx
    b = Batch(7, [3000, 20, 700], 1, 40, 576)
    idx, _ = selection(b, 700, 2, b.lens)
    ws, ws2 = workspace(b), workspace(b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    first = None
    for _ in range(6):
        out, lse = b.buffers()
        out2, lse2 = b.buffers()
        torch.cuda.synchronize()
        fp4idx.latent_attn(b.q, b.cache, b.table, b.row_seq, i32(b.lens), 3000, b.scale, ws, out, lse=lse)
        fp4idx.latent_attn_topk(b.q, b.cache, b.table, b.row_seq, idx, b.scale, ws2, out2, lse=lse2, stream=side)
        torch.cuda.synchronize()
        got = [v.clone() for v in (out, lse, out2, lse2)]
        first = first or got
        assert all(torch.equal(x, y) for x, y in zip(first, got))


def test_waits_run_out():
    """With loads that never come every call ends with a status, and the next calls are right."""
    from sparse_attention_fp4_gb300 import fp4idx
    b = Batch(9, [500, 300], 1, 16, 576)
    many = Batch(10, [400] * 90, 1, 64, 512)
    p = Prompts(11, [200, 40], [300, 40], 2)
    idx, want = selection(b, 200, 1, b.lens)
    midx, mwant = selection(many, 200, 1, many.lens)

    def calls(check):
        for x, sel, w in ((b, idx, want), (many, midx, mwant)):  # a cluster a row; CTAs of a row's own
            status = i32([0])
            out, lse = x.buffers()
            fp4idx.latent_attn_topk(x.q, x.cache, x.table, x.row_seq, sel, x.scale, workspace(x), out, lse=lse, status=status)
            assert fp4idx.read_status(status) == (0 if check else 6)
            if check:
                x.check(out, lse, w, rows=range(0, x.T, 30))
        status = i32([0])
        out, lse = b.buffers()
        fp4idx.latent_attn(b.q, b.cache, b.table, b.row_seq, i32(b.lens), 500, b.scale, workspace(b), out, lse=lse, status=status)
        assert fp4idx.read_status(status) == (0 if check else 6)
        if check:
            b.check(out, lse, [list(range(v)) for v in b.lens])
        status = i32([0])
        out, lse = p.run(status)
        assert fp4idx.read_status(status) == (0 if check else 6)
        if check:
            p.check(out, lse, every=23)

    calls(True)
    try:
        fp4idx.test_pipeline_waits(True, 30_000_000)
        calls(False)
    finally:
        fp4idx.test_pipeline_waits(False, 0)
    calls(True)


def alternating(heads, width, n=24, most=500):
    """Rows whose sequence changes from row to row: as many units as rows, more than two
    sequences of twelve rows would have."""
    b = Batch(12, [most, most - 7], n // 2, heads, width)
    seqs = [(i * 5 % 7) & 1 for i in range(n)]
    assert b.T == n
    b.row_seq = i32(seqs)
    L = [(i * 131) % most if i % 5 else 0 for i in range(n)]
    return b, L


@pytest.mark.parametrize("heads,width", [(8, 512), (12, 576), (32, 512), (40, 576), (128, 512)])
def test_whole_contexts_in_clusters(heads, width):
    """Few short units share a cluster each; units that outnumber the clusters come round after
    round, and clusters without one write nothing."""
    from sparse_attention_fp4_gb300 import fp4idx
    b, L = alternating(heads, width)
    status = i32([0])
    out, lse = b.buffers()
    fp4idx.latent_attn(b.q, b.cache, b.table, b.row_seq, i32(L), 500, b.scale, workspace(b), out, lse=lse, status=status)
    assert fp4idx.read_status(status) == 0
    b.check(out, lse, [list(range(v)) for v in L])
    # 12 rows of the last of seven sequences: two units where up to seven and more could be
    c = Batch(13, [3, 4, 5, 6, 7, 8, 450], 2, heads, width)
    c.row_seq = i32([6] * c.T)
    L = [450 - (c.T - 1 - i) for i in range(c.T)]
    out, lse = c.buffers()
    fp4idx.latent_attn(c.q, c.cache, c.table, c.row_seq, i32(L), 450, c.scale, workspace(c), out, lse=lse, status=status)
    assert fp4idx.read_status(status) == 0
    c.check(out, lse, [list(range(v)) for v in L])


@pytest.mark.parametrize("heads", [8, 64])
def test_waits_run_out_in_clusters(heads):
    from sparse_attention_fp4_gb300 import fp4idx
    b, L = alternating(heads, 576)

    def call(want):
        status = i32([0])
        out, lse = b.buffers()
        fp4idx.latent_attn(b.q, b.cache, b.table, b.row_seq, i32(L), 500, b.scale, workspace(b), out, lse=lse, status=status)
        assert fp4idx.read_status(status) == want
        if want == 0:
            b.check(out, lse, [list(range(v)) for v in L])

    call(0)
    try:
        fp4idx.test_pipeline_waits(True, 30_000_000)
        call(6)
    finally:
        fp4idx.test_pipeline_waits(False, 0)
    call(0)


def test_whole_units():
    """More selections than CTAs: captured and replayed, two at once, and with loads that never
    come; whatever the workspace holds."""
    from sparse_attention_fp4_gb300 import fp4idx
    rows = 608
    lens = [1 + (37 * i) % 500 for i in range(rows)]
    b = Batch(14, lens, 1, 24, 576)
    idx, want = selection(b, 150, 2, lens)
    ws = [workspace(b) for _ in range(2)]
    bufs = [b.buffers() for _ in range(2)]
    status = i32([0])

    def call(i, stream=None):
        fp4idx.latent_attn_topk(b.q, b.cache, b.table, b.row_seq, idx, b.scale, ws[i], bufs[i][0], lse=bufs[i][1],
                                status=status, stream=stream)

    call(0)
    call(1)
    b.check(*bufs[0], want, rows=range(0, rows, 17))
    first = [v.clone() for v in bufs[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0)
    side = torch.cuda.Stream()
    for fill in (0, 255, 7):
        for w, (out, lse) in zip(ws, bufs):
            w.view(torch.uint8).fill_(fill)
            out.fill_(3.0)
            lse.fill_(3.0)
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        call(1, stream=side)
        torch.cuda.synchronize()
        assert fp4idx.read_status(status) == 0
        for out, lse in bufs:
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    try:
        fp4idx.test_pipeline_waits(True, 30_000_000)
        call(0)
        assert fp4idx.read_status(status) == 6
    finally:
        fp4idx.test_pipeline_waits(False, 0)
    status.zero_()
    call(0)
    assert fp4idx.read_status(status) == 0
    assert torch.equal(bufs[0][0], first[0]) and torch.equal(bufs[0][1], first[1])


@pytest.mark.parametrize("heads", [8, 32, 128])
def test_empty_units_among_long_ones(heads):
    """Sequences of no tokens, one and many, in runs, before, between and behind the long ones."""
    from sparse_attention_fp4_gb300 import fp4idx
    lens = [0] * 9 + [2900] + [1] * 30 + [0] * 40 + [2500, 64, 65] + [0] * 25
    b = Batch(16, lens, 1, heads, 512)
    status = i32([0])
    out, lse = b.buffers()
    fp4idx.latent_attn(b.q, b.cache, b.table, b.row_seq, i32(lens), 2900, b.scale, workspace(b), out, lse=lse, status=status)
    assert fp4idx.read_status(status) == 0
    b.check(out, lse, [list(range(v)) for v in lens])
