"""Beam selection against float64."""
import math

import numpy as np
import pytest
import torch

from tests import beam_ref as ref

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
INF = math.inf


def run(logits, scores, beams, k, done=None, end=-1, stream=None, with_done=True):
    from sparse_attention_fp4_gb300 import fp4idx
    R, V = logits.shape
    n = R // beams * k
    out = [torch.full((n + 5,), -77, dtype=d, device="cuda") for d in (FP32, torch.int32, torch.int32, torch.int32)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    # (a workspace that holds nothing)
    ws = torch.full((fp4idx.beam_select_workspace_bytes(R, V, k),), 255, dtype=torch.uint8, device="cuda")
    s = torch.tensor(scores, dtype=FP32, device="cuda")
    d = None if done is None else torch.tensor(done, dtype=torch.int32, device="cuda")
    fp4idx.beam_select(logits, s, beams, k, ws, out[0][:n], out[1][:n], out[2][:n], done=d, end_token=end,
                       done_out=out[3][:n] if with_done else None, status=status, stream=stream)
    torch.cuda.synchronize()
    assert all(bool((o[n:] == -77).all()) for o in out)  # nothing behind the outputs
    got = [o[:n].cpu().numpy().reshape(R // beams, k) for o in out]
    return got if with_done else got[:3] + [None], fp4idx.read_status(status)


def rows(seed, R, V, kind, pad=0, offset=0, spread=2.0):
    """Logits as a view of rows that lie `pad` elements apart, the first `offset` elements into its buffer."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    stride = V + pad
    buf = (spread * torch.randn(offset + R * stride, generator=g, device="cuda")).to(kind)
    x = buf.as_strided((R, V), (stride, 1), offset)
    peaks = torch.randint(0, V, (R, 5), generator=g, device="cuda")
    x.scatter_(1, peaks, (8 + torch.randn(R, 5, generator=g, device="cuda")).to(kind))
    scores = (-10 * torch.rand(R, generator=g, device="cuda") - 0.5).tolist()
    return x, scores


def check(x, scores, beams, k, done=None, end=-1, want_status=0, **kw):
    got, status = run(x, scores, beams, k, done, end, **kw)
    assert status == want_status
    s32 = np.array(scores, dtype=np.float32)
    ref.check_select(got, x.float().cpu().numpy(), s32, beams, k, done, end)
    return got


@pytest.mark.parametrize("kind", [BF16, FP16, FP32])
@pytest.mark.parametrize("groups,beams,V,k,pad,offset", [
    (1, 1, 1, 1, 0, 0), (1, 1, 2, 5, 0, 0), (3, 2, 7, 4, 0, 0), (2, 3, 8, 6, 3, 1), (1, 4, 255, 4, 0, 0), (2, 4, 257, 8, 1, 3),
    (1, 4, 32000, 4, 0, 0), (2, 5, 4097, 10, 0, 5), (3, 1, 16384, 64, 0, 0), (2, 2, 16385, 64, 7, 2), (1, 64, 1000, 64, 0, 0),
    (1, 3, 50001, 6, 0, 1), (5, 6, 9999, 12, 8, 8), (40, 4, 2049, 7, 5, 0), (200, 2, 33000, 4, 0, 0), (1, 2, 262144, 33, 0, 0)])
def test_sizes(kind, groups, beams, V, k, pad, offset):
    x, scores = rows(groups + 7 * beams + V, groups * beams, V, kind, pad, offset)
    check(x, scores, beams, k)


@pytest.mark.parametrize("kind", [BF16, FP32])
def test_largest(kind):
    x, scores = rows(3, 128, 1 << 19, kind)
    check(x, scores, 64, 64)


@pytest.mark.parametrize("kind", [BF16, FP16, FP32])
@pytest.mark.parametrize("V,k", [(300, 8), (40000, 64), (131072, 10)])
def test_ties_go_to_the_lowest(kind, V, k):
    """Equal logits everywhere; only a few values; equal rows with equal scores."""
    x = torch.full((4, V), 1.5, dtype=kind, device="cuda")
    got = check(x, [-1.0, -3.0, -1.0, -2.0], 2, k)
    assert got[2][0].tolist() == list(range(k)) and got[1][0].tolist() == [0] * k
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randint(0, 3, (6, V), generator=g, device="cuda").to(kind)
    check(x, [-1.0, -1.5, -9.0, -2.0, -2.5, -0.25], 3, k)
    one = x[:1].repeat(3, 1)
    got = check(one, [-1.0] * 3, 3, k)
    n = min(k, int((one[0] == 2).sum()))
    top = torch.nonzero(one[0] == 2).flatten().tolist()[:n]
    assert list(zip(got[1][0].tolist(), got[2][0].tolist()))[:n] == [(0, t) for t in top]  # the lower row first


@pytest.mark.parametrize("order", ["up", "down"])
def test_sorted_rows(order):
    v = torch.linspace(-20, 20, 70000, device="cuda")
    x = (v if order == "up" else v.flip(0)).repeat(4, 1).contiguous()
    check(x, [-1.0, -1.1, -1.7, -4.0], 2, 40)


def test_zeros_of_both_signs_are_equal():
    x = torch.zeros((1, 100), device="cuda")
    x[0, ::2] = -0.0
    got = check(x, [0.0], 1, 6)
    assert got[2][0].tolist() == [0, 1, 2, 3, 4, 5]


@pytest.mark.parametrize("kind", [BF16, FP16, FP32])
@pytest.mark.parametrize("kept", [0, 1, 3, 70, 3000])
def test_masked_tokens(kind, kept):
    """-inf rules a token out; fewer candidates than asked for; a row with none left."""
    x, scores = rows(kept, 6, 40000, kind)
    g = torch.Generator(device="cuda").manual_seed(9)
    for r in range(6):
        n = 0 if r in (2, 3) else kept
        keep = torch.randperm(40000, generator=g, device="cuda")[:n]
        m = torch.ones(40000, dtype=torch.bool, device="cuda")
        m[keep] = False
        x[r][m] = -INF
    check(x, scores, 2, 16)


def test_one_run_of_allowed_tokens():
    x, scores = rows(4, 4, 50000, BF16)
    m = torch.ones(50000, dtype=torch.bool, device="cuda")
    m[17000:18500] = False
    x[:, m] = -INF
    check(x, scores, 2, 64)


def test_lowest_values_are_candidates():
    """The type's lowest finite value is a value, not a mask."""
    for kind in (BF16, FP16, FP32):
        x = torch.full((2, 500), torch.finfo(kind).min, dtype=kind, device="cuda")
        x[0, 300] = 1.0
        got, status = run(x, [-1.0, -2.0], 2, 5)
        assert status == 0
        assert got[1][0].tolist()[0] == 0 and got[2][0].tolist()[0] == 300
        assert got[0][0].tolist()[0] == pytest.approx(-1.0, abs=1e-6)
        # row 1: 500 equal tokens
        assert got[1][0].tolist()[1:] == [1] * 4 and got[2][0].tolist()[1:] == [0, 1, 2, 3]
        assert got[0][0].tolist()[1] == pytest.approx(-2.0 - math.log(500), abs=1e-5)


def test_large_logits():
    x = torch.tensor([[3e38, -3e38, 2.9e38], [1e30, 1e30, -1e30]], device="cuda")
    got, status = run(x, [-1.0, -2.0], 1, 2)
    assert status == 0
    assert got[2].tolist()[0][0] == 0 and got[0][0, 0] == -1.0
    assert got[2].tolist()[1] == [0, 1] and got[0][1, 0] == pytest.approx(-2.0 - math.log(2), abs=1e-6)


def test_rows_without_candidates():
    """Dead rows, NaN and +inf in scores and logits: the row has no candidate, its neighbours are not touched."""
    x, scores = rows(11, 8, 20000, BF16)
    for r, v in ((1, math.nan), (3, INF)):
        x[r, 12345] = v
    check(x, scores, 4, 6, want_status=12)
    x, scores = rows(11, 8, 20000, BF16)
    scores[0], scores[5] = math.nan, INF
    check(x, scores, 4, 6, want_status=12)
    # what a dead row holds is not read
    x, scores = rows(11, 8, 20000, BF16)
    scores[2] = -INF
    x[2] = math.nan
    check(x, scores, 4, 6)
    scores = [-INF] * 8
    got = check(x, scores, 4, 6)
    assert (got[1] == -1).all()


def test_nan_only_and_mixed():
    x, scores = rows(12, 3, 5000, FP32)
    x[0] = math.nan
    x[1] = -INF
    x[1, 77] = math.nan
    x[2, 4] = -INF
    check(x, scores, 3, 4, want_status=12)


@pytest.mark.parametrize("end", [0, 999, 4999])
def test_finished_rows(end):
    x, scores = rows(13, 12, 5000, FP16)
    done = [0, 1, 0, 0, 1, 1, 1, 1, 0, 0, 0, 1]
    scores[1], scores[6] = -0.01, -INF
    x[1] = math.nan  # not read
    check(x, scores, 4, 9, done=done, end=end)
    check(x, scores, 1, 2, done=done, end=end)
    check(x, scores, 12, 64, done=done, end=end)
    scores[4] = math.nan
    check(x, scores, 4, 9, done=done, end=end, want_status=12)


def test_end_token_without_finished_rows():
    x, scores = rows(14, 4, 300, FP32)
    x[2, 7] = 30.0
    got = check(x, scores, 2, 5, end=7)
    assert got[3][1].any()
    check(x, scores, 2, 5, end=7, with_done=False)


def test_totals_across_rows_that_are_far_apart():
    x, scores = rows(15, 6, 3001, FP32)
    check(x, [-1e30, -5.0, -2e30, 3e30, -1e-30, 1e10], 2, 5)


@pytest.mark.parametrize("kind", [BF16, FP32])
def test_a_row_is_the_same_in_any_batch(kind):
    x, scores = rows(16, 300, 20000, kind)
    whole, _ = run(x, scores, 1, 3)
    for r in (0, 7, 299):
        alone, _ = run(x[r:r + 1].contiguous(), scores[r:r + 1], 1, 3)
        assert whole[2][r].tolist() == alone[2][0].tolist()
        assert abs(whole[0][r] - alone[0][0]).max() <= 1e-5


def test_rows_past_32_bit_offsets():
    from sparse_attention_fp4_gb300 import fp4idx
    R, V = 8196, 1 << 18  # 2^31 + 2^20 logits
    x = torch.zeros((R, V), dtype=BF16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for r in (0, 8190, 8191, 8192, 8195):
        x[r] = torch.randn(V, generator=g, device="cuda")
    s = torch.full((R,), -1.0, device="cuda")
    out = [torch.empty(R, dtype=d, device="cuda") for d in (FP32, torch.int32, torch.int32)]
    ws = torch.empty(fp4idx.beam_select_workspace_bytes(R, V, 2), dtype=torch.uint8, device="cuda")
    fp4idx.beam_select(x, s, 2, 2, ws, *out)
    got = [o.cpu().numpy().reshape(-1, 2) for o in out]
    for first in (0, 8190, 8192, 8194):
        pair = x[first:first + 2].float().cpu().numpy()
        mine = [v[first // 2:first // 2 + 1].copy() for v in got]
        mine[1] -= first
        ref.check_select(mine + [None], pair, np.float32([-1, -1]), 2, 2)
    assert (got[2][1] == [0, 1]).all() and (got[1][1] == 2).all()  # rows of zeros


@pytest.mark.parametrize("beams", [1, 64])
def test_the_most_rows(beams):
    from sparse_attention_fp4_gb300 import fp4idx
    R, V, k = 1 << 20, 3, 1
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((R, V), generator=g, device="cuda")
    s = -torch.rand(R, generator=g, device="cuda")
    out = [torch.empty(R // beams, dtype=d, device="cuda") for d in (FP32, torch.int32, torch.int32)]
    ws = torch.empty(fp4idx.beam_select_workspace_bytes(R, V, k), dtype=torch.uint8, device="cuda")
    fp4idx.beam_select(x, s, beams, k, ws, *out)
    total = (s.double()[:, None] + torch.log_softmax(x.double(), 1)).view(R // beams, -1)
    want, at = total.max(1)
    assert float((out[0].double() - want).abs().max()) < 3e-6
    first = torch.arange(R // beams, device="cuda") * beams
    flat = (out[1] - first) * V + out[2]
    assert bool(((flat >= 0) & (flat < beams * V)).all())
    chosen = total.gather(1, flat.long()[:, None])[:, 0]
    assert float((want - chosen).max()) < 3e-6  # the best, but for totals that close


def test_two_streams_at_once():
    from sparse_attention_fp4_gb300 import fp4idx
    a, sa = rows(30, 64, 60000, BF16)
    b, sb = rows(31, 40, 50001, FP32)
    calls = []
    for x, scores, beams, k in ((a, sa, 4, 8), (b, sb, 20, 20)):
        n = x.shape[0] // beams * k
        out = [torch.empty(n, dtype=d, device="cuda") for d in (FP32, torch.int32, torch.int32)]
        ws = torch.empty(fp4idx.beam_select_workspace_bytes(*x.shape, k), dtype=torch.uint8, device="cuda")
        calls.append((x, torch.tensor(scores, device="cuda"), beams, k, ws, out, scores))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (x, s, beams, k, ws, out, _) in zip(streams, calls):
            fp4idx.beam_select(x, s, beams, k, ws, *out, stream=st)
    torch.cuda.synchronize()
    for x, s, beams, k, ws, out, scores in calls:
        ref.check_select([o.cpu().numpy().reshape(-1, k) for o in out] + [None], x.float().cpu().numpy(), np.float32(scores), beams, k)


def test_streams_graph_and_repeats():
    from sparse_attention_fp4_gb300 import fp4idx
    x, scores = rows(17, 32, 30000, BF16)
    want = check(x, scores, 4, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = run(x, scores, 4, 8, stream=side)
    assert all((a == b).all() for a, b in zip(got, want))
    s = torch.tensor(scores, device="cuda")
    mk = lambda d: torch.empty(64, dtype=d, device="cuda")  # noqa: E731
    out = [mk(FP32), mk(torch.int32), mk(torch.int32)]
    ws = torch.empty(fp4idx.beam_select_workspace_bytes(32, 30000, 8), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp4idx.beam_select(x, s, 4, 8, ws, *out)
        fp4idx.beam_select(x, s, 4, 8, ws, *out)  # one workspace, one after another
    for _ in range(3):
        for o in out:
            o.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert all((o.cpu().numpy().reshape(8, 8) == w).all() for o, w in zip(out, want))
    x.copy_(x.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    ref.check_select([o.cpu().numpy().reshape(8, 8) for o in out] + [None], x.float().cpu().numpy(), np.float32(scores), 4, 8)


def test_workspace_filled_by_other_calls():
    """What another call left in the workspace does not matter."""
    from sparse_attention_fp4_gb300 import fp4idx
    a, sa = rows(18, 64, 30000, BF16)
    b, sb = rows(19, 4, 700, FP32)
    ws = torch.empty(fp4idx.beam_select_workspace_bytes(64, 30000, 8), dtype=torch.uint8, device="cuda")
    for x, scores, beams, k in ((a, sa, 4, 8), (b, sb, 2, 5), (a, sa, 64, 3)):
        n = x.shape[0] // beams * k
        out = [torch.empty(n, dtype=d, device="cuda") for d in (FP32, torch.int32, torch.int32)]
        fp4idx.beam_select(x, torch.tensor(scores, device="cuda"), beams, k, ws, *out)
        ref.check_select([o.cpu().numpy().reshape(-1, k) for o in out] + [None], x.float().cpu().numpy(), np.float32(scores), beams, k)


def test_refusals_of_the_binding():
    from sparse_attention_fp4_gb300 import fp4idx
    x, scores = rows(20, 4, 100, BF16)
    s = torch.tensor(scores, device="cuda")
    ws = torch.empty(fp4idx.beam_select_workspace_bytes(4, 100, 2), dtype=torch.uint8, device="cuda")
    o = [torch.empty(4, dtype=d, device="cuda") for d in (FP32, torch.int32, torch.int32)]
    f = lambda x=x, s=s, beams=2, k=2, ws=ws, o=o, **kw: fp4idx.beam_select(x, s, beams, k, ws, *o, **kw)  # noqa: E731
    f()
    for kw in (dict(x=x.t()), dict(x=x.double()), dict(x=x.cpu()), dict(x=x[0]), dict(s=s[:3]), dict(o=[o[0][:3], o[1], o[2]]),
               dict(x=x.as_strided((4, 100), (50, 1)))):
        with pytest.raises(ValueError):
            f(**kw)
    for kw in (dict(beams=3), dict(beams=0), dict(k=0), dict(end_token=100), dict(end_token=-2), dict(ws=ws[:-1].clone()),
               dict(done=torch.zeros(4, dtype=torch.int32, device="cuda"))):
        with pytest.raises(fp4idx.Fp4IdxError):
            f(**kw)
