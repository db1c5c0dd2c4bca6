"""The largest calls that the latent entry points allow, and counts beyond one round of a kernel's loops."""
import math

import pytest
import torch

from tests import latent_ref as ref
from tests.test_gpu_plan_store import NAMES, cos_sin_table, run_plan

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


UNWRITTEN = -1e30


def empty_outputs(rows, heads, dims):
    return (torch.full((rows, heads, dims), 3.0, dtype=torch.bfloat16, device="cuda"),
            torch.full((rows, heads), UNWRITTEN, dtype=torch.float32, device="cuda"))


ROWS, SEQS = 1 << 20, 4096


def many_rows(width):
    """2^20 rows of one head, 256 of every sequence, of 0 to 150 tokens."""
    g = torch.Generator(device="cuda").manual_seed(3)
    lens = [(i * 89) % 151 for i in range(SEQS)]
    cache = torch.randn((3 * SEQS, 64, width), generator=g, device="cuda").to(torch.bfloat16)
    table = torch.randperm(3 * SEQS, generator=g, device="cuda").to(torch.int32).view(SEQS, 3).contiguous()
    q = torch.randn((ROWS, 1, width), generator=g, device="cuda").to(torch.bfloat16)
    seq = torch.arange(SEQS, dtype=torch.int32, device="cuda").repeat_interleave(ROWS // SEQS)
    return lens, cache, table, q, seq


def check_rows(out, lse, q, cache, table, positions, scale):
    """Whole sequences, spread over the call; a sequence's rows see the same tokens."""
    n = ROWS // SEQS
    for b in list(range(0, SEQS, 97)) + [SEQS - 1]:
        k = ref.tokens(cache, table[b], positions(b))
        at = slice(b * n, (b + 1) * n)
        ref.check(out[at, 0], lse[at, 0], ref.attend(q[at, 0].double(), k, k[:, :512], scale), "sequence %d" % b)
    assert not bool((lse == UNWRITTEN).any())


def test_rows_over_whole_contexts():
    from sparse_attention_fp4_gb300 import fp4idx
    lens, cache, table, q, seq = many_rows(512)
    out, lse = empty_outputs(ROWS, 1, 512)
    ws = torch.empty(fp4idx.latent_attn_workspace_bytes(ROWS, 1), dtype=torch.uint8, device="cuda")
    status = i32([0])
    fp4idx.latent_attn(q, cache, table, seq, i32(lens)[seq.long()], 192, 0.05, ws, out, lse=lse, status=status)
    assert fp4idx.read_status(status) == 0
    check_rows(out, lse, q, cache, table, lambda b: list(range(lens[b])), 0.05)


def test_rows_over_selections():
    from sparse_attention_fp4_gb300 import fp4idx
    lens, cache, table, q, seq = many_rows(576)
    out, lse = empty_outputs(ROWS, 1, 512)
    ws = torch.empty(fp4idx.latent_attn_workspace_bytes(ROWS, 1), dtype=torch.uint8, device="cuda")
    status = i32([0])
    picks = [sorted(set((7 * j * j + b) % lens[b] for j in range(20))) if lens[b] else [] for b in range(SEQS)]
    idx = i32([p + [-1] * (20 - len(p)) for p in picks])[seq.long()]
    fp4idx.latent_attn_topk(q, cache, table, seq, idx, 0.05, ws, out, lse=lse, status=status)
    assert fp4idx.read_status(status) == 0
    check_rows(out, lse, q, cache, table, lambda b: picks[b], 0.05)


def test_sequences_of_expanded_attention():
    """65,535 sequences of no to three queries."""
    from sparse_attention_fp4_gb300 import fp4idx
    B, H = 65535, 2
    b = torch.arange(B, device="cuda")
    nq, nk = b * 7 % 4, b * 7 % 4 + b % 3
    cu = lambda v: torch.cat([v.new_zeros(1), v.cumsum(0)]).to(torch.int32)  # noqa: E731
    cq, ck = cu(nq), cu(nk)
    g = torch.Generator(device="cuda").manual_seed(4)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    Q, K = int(cq[-1]), int(ck[-1])
    q, kv, kr, scale = mk(Q + 5, H, 192), mk(K + 5, H, 256), mk(K + 5, 64), 192 ** -0.5
    out, lse = empty_outputs(Q + 5, H, 128)
    status = i32([0])
    fp4idx.latent_prefill(q, kv, kr, cq, ck, 3, 5, scale, out, lse=lse, status=status)
    assert fp4idx.read_status(status) == 0
    assert bool((out[Q:] == 3).all()) and bool((lse[Q:] == UNWRITTEN).all()) and not bool((lse[:Q] == UNWRITTEN).any())
    cq, ck = cq.tolist(), ck.tolist()
    for s in list(range(0, B, 1301)) + list(range(B - 4, B)):
        n, m = cq[s + 1] - cq[s], ck[s + 1] - ck[s]
        for i in range(n):
            for h in range(H):
                rows = slice(ck[s], ck[s] + m - n + i + 1)
                key = torch.cat([kv[rows, h, :128], kr[rows]], 1).double()
                want = ref.attend(q[cq[s] + i, h].double()[None], key, kv[rows, h, 128:].double(), scale)
                ref.check(out[cq[s] + i, h][None], lse[cq[s] + i, h][None], want, "sequence %d row %d" % (s, i))


@pytest.mark.parametrize("width", [512, 576])
def test_store_of_many_rows(width):
    """More rows than a kernel's warps take in their first round, a third of them padding or bad."""
    from sparse_attention_fp4_gb300 import fp4idx
    n, pages = 200001, 3200
    g = torch.Generator(device="cuda").manual_seed(width)
    kv = (2 * torch.randn((n, width), generator=g, device="cuda")).to(torch.bfloat16)
    w = (1 + 0.1 * torch.randn(512, generator=g, device="cuda")).to(torch.bfloat16)
    pos = torch.randint(0, 5000, (n,), generator=g, device="cuda", dtype=torch.int32)
    slots = torch.randperm(pages * 64, generator=g, device="cuda")[:n].to(torch.int32)
    drop = torch.rand(n, generator=g, device="cuda")
    slots = torch.where(drop < 0.2, -1, slots).to(torch.int32)
    pos = torch.where((drop > 0.2) & (drop < 0.33), 5000, pos).to(torch.int32)
    cs = cos_sin_table(5000)
    cache = torch.full((pages, 64, width), 7.5, dtype=torch.bfloat16, device="cuda")
    status = i32([0])
    fp4idx.store_latent(kv, pos, slots, w, 1e-6, cs, cache, status=status)
    assert fp4idx.read_status(status) == 7
    keep = (slots >= 0) & (pos < 5000)
    flat = cache.view(-1, width)
    at = slots[keep].long()
    for part in torch.arange(int(keep.sum()), device="cuda").split(40000):
        want, tol = ref.store(kv[keep][part], pos[keep][part], w, 1e-6, cs)
        assert bool(((flat[at[part]].double() - want).abs() <= tol).all())
    rest = torch.ones(pages * 64, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert bool((flat[rest] == 7.5).all())


def test_plan_of_most_sequences():
    B = 65536
    cached, new = [(i * 37) % 200 for i in range(B)], [(i * 11) % 3 for i in range(B)]
    free = list(range(B * 5, B * 6))
    table = [[b * 4 + j if j < -(-cached[b] // 64) else -5 for j in range(4)] for b in range(B)]
    rows, stores = sum(new) + 9, sum(new) + 2
    want = ref.plan(cached, new, 1, free, 0, [list(t) for t in table], rows, stores)
    got, status = run_plan(cached, new, 1, free, table, rows, stores)
    assert status == 0 and not want["full"]
    for n in NAMES + ("table",):
        assert got[n] == want[n], n


def test_plan_context_sum():
    """Entries after the step that 32-bit offsets cannot count: the sequences from there on get nothing."""
    from sparse_attention_fp4_gb300 import fp4idx
    each = 900_000_000
    cols = math.ceil(each / 64) + 1
    table = torch.full((4, cols), 3, dtype=torch.int32, device="cuda")
    new = lambda n: torch.full((n,), -77, dtype=torch.int32, device="cuda")  # noqa: E731
    pos, seq, ctx, spos, slots, cu, cu_ctx, counts = new(5), new(5), new(5), new(5), new(5), new(5), new(5), new(4)
    status = i32([0])
    fp4idx.plan_step(i32([each, each, each, 10]), i32([1, 2, 1, 1]), 1, i32([7, 8, 9, 10]), table, pos, seq, ctx, spos, slots, cu, cu_ctx, counts,
                     status=status)
    assert fp4idx.read_status(status) == 11
    assert counts.tolist() == [3, 3, 2, 2] and cu.tolist() == [0, 1, 3, 3, 3]
    assert cu_ctx.tolist() == [0, each + 1, 2 * each + 3, 2 * each + 3, 2 * each + 3]
    assert pos.tolist() == [each, each, each + 1, 0, 0] and seq.tolist() == [0, 1, 1, 0, 0] and ctx.tolist() == [each + 1, each + 1, each + 2, 0, 0]
    assert slots.tolist() == [7 * 64, 8 * 64, 8 * 64 + 1, -1, -1] and spos.tolist() == [each, each, each + 1, 0, 0]
    assert (900_000_000 % 64, table[0, -1].item(), table[2, -1].item()) == (0, 7, 3)
