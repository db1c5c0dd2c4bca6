"""Expanded causal latent attention against the formula in float64."""
import math

import pytest
import torch

from tests import latent_ref as ref

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def cu(v):
    return i32([sum(v[:i]) for i in range(len(v) + 1)])


class Prompts:
    def __init__(self, seed, nq, nk, heads, behind=0, qscale=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.nq, self.nk, self.H = nq, nk, heads
        Q, K = sum(nq) + behind, sum(nk) + behind
        mk = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        self.q, self.kv, self.kr = mk(Q, heads, 192) * qscale, mk(K, heads, 256), mk(K, 64)
        self.cu_q, self.cu_k = cu(nq), cu(nk)
        self.scale = 192 ** -0.5

    def run(self, status=None, lse=True, **kw):
        from sparse_attention_fp4_gb300 import fp4idx
        out = torch.full((self.q.shape[0], self.H, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        l = torch.full((self.q.shape[0], self.H), 3.0, dtype=torch.float32, device="cuda")
        a = dict(max_q=max(self.nq, default=0), max_kv=max(self.nk, default=0), cu_q=self.cu_q, cu_kv=self.cu_k)
        a.update(kw)
        fp4idx.latent_prefill(self.q, self.kv, self.kr, a["cu_q"], a["cu_kv"], a["max_q"], a["max_kv"], self.scale, out,
                              lse=l if lse else None, status=status)
        return out, l if lse else None

    def check(self, out, lse, every=1, seqs=None):
        q0 = k0 = 0
        for b, (n, m) in enumerate(zip(self.nq, self.nk)):
            if seqs is None or b in seqs:
                picks = sorted(set(list(range(0, n, every)) + ([n - 1] if n else [])))
                for h in range(self.H):
                    key = torch.cat([self.kv[k0:k0 + m, h, :128], self.kr[k0:k0 + m]], 1).double()
                    val = self.kv[k0:k0 + m, h, 128:].double()
                    for i in picks:
                        see = max(0, min(m, m - n + i + 1))
                        want = ref.attend(self.q[q0 + i, h].double()[None], key[:see], val[:see], self.scale)
                        ref.check(out[q0 + i, h][None], None if lse is None else lse[q0 + i, h][None], want, "seq %d row %d head %d" % (b, i, h))
            q0, k0 = q0 + n, k0 + m
        assert bool((out[q0:] == 3).all()) and (lse is None or bool((lse[q0:] == 3).all()))


@pytest.mark.parametrize("heads", [1, 3])
@pytest.mark.parametrize("nq,nk", [([1], [1]), ([1], [300]), ([127], [127]), ([128], [128]), ([129], [129]), ([257], [257]),
                                   ([5, 0, 64, 1], [5, 0, 200, 129]), ([130, 1, 255], [400, 2, 255]), ([3, 300], [1, 40]),
                                   ([20, 10], [0, 10]), ([513], [700])])
def test_prompts(heads, nq, nk):
    from sparse_attention_fp4_gb300 import fp4idx
    p = Prompts(heads + sum(nq), nq, nk, heads, behind=7)
    status = i32([0])
    out, lse = p.run(status)
    p.check(out, lse, every=5)
    out2, _ = p.run(status, lse=False)
    assert torch.equal(out, out2) and fp4idx.read_status(status) == 0


def test_long_prompt():
    p = Prompts(1, [2500, 100], [2500, 1700], 2)
    out, lse = p.run()
    p.check(out, lse, every=61)


def test_many_heads_and_sequences():
    nq = [1 + (i * 37) % 150 for i in range(40)]
    p = Prompts(2, nq, [n + (i % 3) * 50 for i, n in enumerate(nq)], 16)
    out, lse = p.run(max_q=400, max_kv=1000)
    p.check(out, lse, every=29, seqs=(0, 3, 11, 39))


def test_large_scores():
    p = Prompts(3, [300], [300], 2, qscale=20.0)
    out, lse = p.run()
    p.check(out, lse, every=3)


def test_nan_behind_the_end():
    """What stands behind a sequence's last key and value (another sequence, padding) does not matter."""
    p = Prompts(4, [70, 50, 40], [70, 90, 40], 2, behind=200)
    p.kv[70:160] = math.nan
    p.kr[70:160] = math.nan
    p.kv[200:] = math.inf
    p.kr[200:] = math.nan
    out, lse = p.run()
    p.check(out, lse, seqs=(0, 2))


def test_bad_offsets():
    """Offsets that decrease or leave the arrays: the sequence is skipped and reported."""
    from sparse_attention_fp4_gb300 import fp4idx
    p = Prompts(5, [30, 40], [30, 40], 2)
    for kw in (dict(cu_q=i32([0, 30, 71])), dict(cu_kv=i32([0, 30, 71])), dict(cu_q=i32([0, 30, 20])), dict(cu_kv=i32([0, 30, 29])),
               dict(max_q=39), dict(max_kv=39)):
        status = i32([0])
        out, lse = p.run(status, **kw)
        assert fp4idx.read_status(status) == 8
        half = Prompts(5, [30, 40], [30, 40], 2)
        half.nq, half.nk = [30], [30]
        half.check(out, lse, every=7)
    for kw in (dict(cu_q=i32([-1, 30, 70])), dict(cu_kv=i32([-1, 30, 70]))):
        status = i32([0])
        out, lse = p.run(status, **kw)
        assert fp4idx.read_status(status) == 8
        assert bool((out[:30] == 3).all()) and not bool((lse[30:] == 3).any())


def test_graph_and_stream():
    p = Prompts(6, [200, 33], [240, 33], 4)
    out, lse = p.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out2, lse2 = p.run()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    p.q.copy_(p.q.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    p.check(out2, lse2, every=17)


def test_nothing():
    from sparse_attention_fp4_gb300 import fp4idx
    p = Prompts(7, [0, 0], [0, 5], 2, behind=4)
    out, lse = p.run(max_q=4)
    assert bool((out == 3).all()) and bool((lse == 3).all())
    with pytest.raises(ValueError):
        fp4idx.latent_prefill(p.q[:, :, :100], p.kv, p.kr, p.cu_q, p.cu_k, 4, 5, 1.0, out)
    with pytest.raises(ValueError):
        fp4idx.latent_prefill(p.q, p.kv[:, :, :200], p.kr, p.cu_q, p.cu_k, 4, 5, 1.0, out)
    with pytest.raises(ValueError):
        fp4idx.latent_prefill(p.q, p.kv, p.kr[:2], p.cu_q, p.cu_k, 4, 5, 1.0, out)


def test_loose_bounds():
    """Bounds far above the lengths change nothing."""
    from sparse_attention_fp4_gb300 import fp4idx
    p = Prompts(15, [5, 130], [9, 300], 2, behind=3)
    status = i32([0])
    out, lse = p.run(status, max_q=2 ** 31 - 1, max_kv=2 ** 31 - 1)
    assert fp4idx.read_status(status) == 0
    p.check(out, lse, every=9)


@pytest.mark.parametrize("heads,nq,nk", [(1, [1], [2000]), (1, [300], [1900]), (2, [36, 1, 0, 257], [1100, 1000, 0, 300]),
                                         (1, [256, 5], [4, 2300]), (3, [129], [1000]), (4, [700, 20], [700, 30])])
def test_keys_of_a_block_split(heads, nq, nk):
    """Few blocks of queries: clusters of two to eight CTAs share a block's keys, with pieces that
    some rows or all see nothing of; the same bits every time."""
    from sparse_attention_fp4_gb300 import fp4idx
    p = Prompts(heads + sum(nk), nq, nk, heads, behind=5)
    status = i32([0])
    out, lse = p.run(status)
    p.check(out, lse, every=7)
    for _ in range(3):
        out2, lse2 = p.run(status)
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert fp4idx.read_status(status) == 0
    try:
        fp4idx.test_pipeline_waits(True, 30_000_000)
        p.run(status)
        assert fp4idx.read_status(status) == 6
    finally:
        fp4idx.test_pipeline_waits(False, 0)
    status.zero_()
    out2, lse2 = p.run(status)
    assert fp4idx.read_status(status) == 0 and torch.equal(out, out2) and torch.equal(lse, lse2)


def test_keys_split_nan():
    """A NaN row of values in one piece: NaN for the rows that see it and up to 255 before it."""
    p = Prompts(21, [200], [1500], 1)
    p.kv[1450, 0, 130:] = math.nan
    out, lse = p.run()
    first = 1450 - 1300  # the first query that sees it
    assert bool(out[first:, 0, 2:].isnan().all()) and not bool(lse.isnan().any())
    q = Prompts(21, [200], [1500], 1)
    want, _ = q.run()
    assert torch.equal(out[:, 0, :2], want[:, 0, :2])
    p.kv[1450, 0, 130:] = 0
    p.kv[3, 0, 0] = math.nan
    out, lse = p.run()
    assert bool(out.isnan().all()) and bool(lse.isnan().all())
