"""Requests decoded as several hypotheses, as a program runs them: plan, stores, attention, selection, fork, page
copies, and a compaction on the way; against hypotheses that each keep a full record of their own."""
import math

import pytest
import torch

from tests import beam_ref
from tests import latent_ref as ref
from tests.test_gpu_plan_store import cos_sin_table, i32

pytestmark = pytest.mark.gpu

W, H, V, WIDTH, MAX_PAGES = 3, 8, 700, 576, 6


def bf16(g, *shape, scale=1.0):
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(torch.bfloat16)


class Step:
    """The buffers of a step of up to `rows` new tokens, and the calls on them."""

    def __init__(self, pages, g):
        from sparse_attention_fp4_gb300 import fp4idx
        self.f, self.pages, self.g = fp4idx, pages, g
        self.cs = cos_sin_table(2048)
        self.norm_k, self.norm_kv = bf16(g, 128) + 1, bf16(g, 512, scale=0.1) + 1
        self.payload, self.scale = fp4idx.alloc_cache(pages)
        self.latents = fp4idx.alloc_latent_cache(pages, WIDTH)
        self.free = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        self.head, self.status = i32([0]), i32([0])
        self.embed, self.w_q = bf16(g, V, WIDTH), bf16(g, WIDTH, H * WIDTH, scale=WIDTH ** -0.5)
        self.w_out = bf16(g, H * 512, V, scale=3 * (H * 512) ** -0.5)

    def run(self, table, cached, tokens, new):
        """tokens: the new tokens of the rows, packed; returns logits of every new row."""
        f, B, n = self.f, len(new), sum(new)
        mk = lambda m: torch.empty(m, dtype=torch.int32, device="cuda")  # noqa: E731
        pos, seq, ctx, spos, slots, cu, cu_ctx, counts = (mk(m) for m in (n,) * 5 + (B + 1, B + 1, 4))
        f.plan_step(cached, i32(new), 1, self.free, table, pos, seq, ctx, spos, slots, cu, cu_ctx, counts, free_head=self.head, status=self.status)
        x = self.embed[tokens.long()]
        f.store_latent(x, spos, slots, self.norm_kv, 1e-6, self.cs, self.latents, status=self.status)
        f.store_k(x[:, :128].contiguous(), spos, slots, self.norm_k, 1e-6, self.cs, self.payload, self.scale, status=self.status)
        q = (x.float() @ self.w_q.float()).to(torch.bfloat16).view(n, H, WIDTH)
        out = torch.empty((n, H, 512), dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(f.latent_attn_workspace_bytes(n, H), dtype=torch.uint8, device="cuda")
        f.latent_attn(q, self.latents, table, seq, ctx, MAX_PAGES * 64, 0.05, ws, out, status=self.status)
        self.head += counts[2:3]
        cached += i32(new)
        return out.view(n, -1).float() @ self.w_out.float()


def test_beams_over_a_paged_cache():
    g = torch.Generator(device="cuda").manual_seed(4)
    pages, G, end = 80, 4, 5
    st = Step(pages, g)
    f = st.f
    prompts = [64, 70, 1, 130]
    table = torch.full((G, MAX_PAGES), -1, dtype=torch.int32, device="cuda")
    cached = i32([0] * G)
    told = torch.randint(0, V, (sum(prompts),), generator=g, device="cuda")
    logits = st.run(table, cached, told, prompts)
    last = torch.tensor(prompts, device="cuda").cumsum(0) - 1
    logits = logits[last].to(torch.bfloat16)
    # the record: per row the tokens of its hypothesis
    at = 0
    record = []
    for n in prompts:
        record.append(told[at:at + n].tolist())
        at += n
    scores, done, beams = torch.zeros(G, device="cuda"), None, 1
    for step in range(70):
        n = G * W
        out_s, out_r, out_t, out_d = (torch.empty(n, dtype=d, device="cuda") for d in (torch.float32, torch.int32, torch.int32, torch.int32))
        ws = torch.empty(f.beam_select_workspace_bytes(G * beams, V, W), dtype=torch.uint8, device="cuda")
        f.beam_select(logits, scores, beams, W, ws, out_s, out_r, out_t, done=done, end_token=end, done_out=out_d, status=st.status)
        # a hypothesis that has ended is as good as its score says, and goes on; against float64
        beam_ref.check_select([v.cpu().numpy().reshape(G, W) for v in (out_s, out_r, out_t, out_d)], logits.float().cpu().numpy(), scores.cpu().numpy(),
                              beams, W, None if done is None else done.tolist(), end)
        if step == 40:  # one request is cancelled
            out_r[:W] = -1
            out_s[:W] = -math.inf
        rows = out_r.tolist()
        new_table, new_cached = torch.empty((n, MAX_PAGES), dtype=torch.int32, device="cuda"), i32([0] * n)
        src, dst, counts = i32([0] * n), i32([0] * n), i32([0] * 4)
        f.fork_pages(table, cached, 1, out_r, pages, st.free, new_table, new_cached, src, dst, counts, free_head=st.head, status=st.status)
        f.copy_pages(src, dst, [st.payload, st.scale, st.latents], count=counts[:1], status=st.status)
        st.head += counts[2:3]
        table, cached = new_table, new_cached
        record = [list(record[r]) if r >= 0 else [] for r in rows]
        if step in (25, 55):  # the pool shrinks to what is in use
            packed, m = torch.empty_like(table), pages
            msrc, mdst, counts = i32([0] * m), i32([0] * m), i32([0] * 4)
            cws = torch.empty(f.compact_pages_workspace_bytes(pages), dtype=torch.uint8, device="cuda")
            f.compact_pages(table, cached, 1, pages, cws, st.free, packed, msrc, mdst, counts, status=st.status)
            f.copy_pages(msrc, mdst, [st.payload, st.scale, st.latents], count=counts[:1], status=st.status)
            table = packed
            st.head.copy_(counts[3:4])
            moves, used, top, _ = counts.tolist()
            assert top == used and moves > 0
        # the next tokens: rows that are empty get none; finished rows get theirs again and again (and a place in the cache)
        new = [1 if r >= 0 else 0 for r in rows]
        tokens = torch.tensor([t for t, r in zip(out_t.tolist(), rows) if r >= 0], device="cuda")
        got = st.run(table, cached, tokens, new).to(torch.bfloat16)
        logits = torch.zeros((n, V), dtype=torch.bfloat16, device="cuda")
        logits[torch.tensor(new, device="cuda") == 1] = got
        for r, t in zip([i for i in range(n) if new[i]], tokens.tolist()):
            record[r].append(t)
        scores, done, beams = out_s, out_d, W
        assert f.read_status(st.status) == 0
        assert cached.tolist() == [len(t) for t in record]
        # no page lost, none held that is free
        held = {p for t, c in zip(table.tolist(), cached.tolist()) for p in t[:-(-c // 64)]}
        spare = st.free[int(st.head):].tolist()
        assert sorted(spare + list(held)) == list(range(pages))
    # every hypothesis' cache is that of its own tokens, at its own positions
    for r in range(n):
        if not record[r]:
            continue
        x = st.embed[torch.tensor(record[r], device="cuda")]
        want, tol = ref.store(x, i32(list(range(len(record[r])))), st.norm_kv, 1e-6, st.cs)
        at = torch.arange(len(record[r]), device="cuda")
        stored = st.latents[table[r].long()[at // 64], at % 64].double()
        assert bool(((stored - want).abs() <= tol).all()), r
        fresh_p, fresh_s = f.alloc_cache(MAX_PAGES)
        f.store_k(x[:, :128].contiguous(), at.to(torch.int32), at.to(torch.int32), st.norm_k, 1e-6, st.cs, fresh_p, fresh_s)
        for p in range(-(-len(record[r]) // 64)):
            m = min(64, len(record[r]) - 64 * p)
            assert bool((st.payload[table[r, p].long()][:, :m] == fresh_p[p][:, :m]).all()), (r, p)
            assert bool((st.scale[table[r, p].long()][:, :m] == fresh_s[p][:, :m]).all()), (r, p)


def test_a_beam_step_in_one_graph():
    """Selection, fork and copies captured together; replays on other inputs."""
    from sparse_attention_fp4_gb300 import fp4idx as f
    g = torch.Generator(device="cuda").manual_seed(6)
    G, pages, n = 5, 300, 5 * W
    logits, scores = bf16(g, n, V, scale=3), -5 * torch.rand(n, generator=g, device="cuda")
    lens = torch.tensor([100, 64, 65, 300, 1], device="cuda").repeat_interleave(W).to(torch.int32)
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = ids[:n * MAX_PAGES].view(n, MAX_PAGES).contiguous()
    free, head = ids[n * MAX_PAGES - 40:].clone(), i32([40])
    latents = bf16(g, pages, 64, WIDTH)
    ws = torch.empty(f.beam_select_workspace_bytes(n, V, W), dtype=torch.uint8, device="cuda")
    out = [torch.empty(n, dtype=d, device="cuda") for d in (torch.float32, torch.int32, torch.int32)]
    new_table, new_cached, src, dst, counts = torch.empty_like(table), i32([0] * n), i32([0] * n), i32([0] * n), i32([0] * 4)

    def step():
        f.beam_select(logits, scores, W, W, ws, *out)
        f.fork_pages(table, lens, 1, out[1], pages, free, new_table, new_cached, src, dst, counts, free_head=head)
        f.copy_pages(src, dst, [latents], count=counts[:1])

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    first = free.clone()
    for seed in range(3):
        logits.copy_(bf16(g, n, V, scale=3))
        free.copy_(first)
        before = latents.clone()
        graph.replay()
        torch.cuda.synchronize()
        beam_ref.check_select([v.cpu().numpy().reshape(G, W) for v in out] + [None], logits.float().cpu().numpy(), scores.cpu().numpy(), W, W)
        want = beam_ref.fork(table.tolist(), lens.tolist(), 1, out[1].tolist(), pages, first.tolist(), 40)
        assert new_table.tolist() == want["table"] and src.tolist() == want["src"] and dst.tolist() == want["dst"]
        assert counts.tolist() == want["counts"] and free.tolist() == want["free"]
        for s, d in zip(want["src"], want["dst"]):
            if s >= 0:
                before[d] = before[s]
        assert bool((before == latents).all())
