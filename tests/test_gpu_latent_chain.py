"""A decode step as a program runs it: plan, both stores, queries, selection, attention."""
import pytest
import torch

from tests import latent_ref as ref
from tests.test_gpu_plan_store import cos_sin_table, i32

pytestmark = pytest.mark.gpu


def bf16(g, *shape, scale=1.0):
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(torch.bfloat16)


def test_prompt_then_decode_steps():
    from sparse_attention_fp4_gb300 import fp4idx
    g = torch.Generator(device="cuda").manual_seed(0)
    B, width, H, k, max_pages, pages = 5, 576, 16, 48, 8, 48
    cs = cos_sin_table(1024)
    norm_k, norm_kv = bf16(g, 128) + 1, bf16(g, 512, scale=0.1) + 1
    payload, scale = fp4idx.alloc_cache(pages)
    latents = fp4idx.alloc_latent_cache(pages, width)
    truth = torch.zeros((B, max_pages * 64, width), dtype=torch.float64, device="cuda")
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    head, status = i32([0]), i32([0])
    cached = [0] * B
    cached_dev = i32(cached)
    for new in ([70, 1, 128, 0, 200], [1] * 5, [3, 1, 0, 2, 1]):
        rows, pad = sum(new), 3
        new_dev = i32(new)
        mk = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        pos, seq, ctx, spos, slots, cu, cu_ctx, counts = (mk(n) for n in (rows + pad,) * 5 + (B + 1, B + 1, 4))
        fp4idx.plan_step(cached_dev, new_dev, 1, free, table, pos, seq, ctx, spos, slots, cu, cu_ctx, counts, free_head=head, status=status)
        T = rows + pad
        kv, kidx, qidx = bf16(g, T, width), bf16(g, T, 128), bf16(g, T, 64, 128)
        q, w = bf16(g, T, H, width), torch.randn((T, 64), generator=g, device="cuda")
        fp4idx.store_latent(kv, spos, slots, norm_kv, 1e-6, cs, latents, status=status)
        fp4idx.store_k(kidx, spos, slots, norm_k, 1e-6, cs, payload, scale, status=status)
        qp, qs = fp4idx.alloc_query(T)
        fp4idx.quant_q(qidx, pos, cs, qp, qs, status=status)
        sched = torch.empty(fp4idx.schedule_workspace_bytes(T), dtype=torch.uint8, device="cuda")
        fp4idx.build_schedule(ctx, seq, sched)
        most = max(c + n for c, n in zip(cached, new))
        lws = torch.empty(fp4idx.logits_workspace_bytes(T, most, k), dtype=torch.uint8, device="cuda")
        topk = torch.empty((T, k), dtype=torch.int32, device="cuda")
        fp4idx.logits_topk(qp, qs, w, payload, scale, table, seq, ctx, most, k, sched, lws, topk, status=status)
        aws = torch.empty(fp4idx.latent_attn_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
        out, whole = torch.empty((2, T, H, 512), dtype=torch.bfloat16, device="cuda").unbind(0)
        lse, wlse = torch.empty((2, T, H), dtype=torch.float32, device="cuda").unbind(0)
        sc = 192 ** -0.5
        fp4idx.latent_attn_topk(q, latents, table, seq, topk, sc, aws, out, lse=lse, context_lens=ctx, status=status)
        fp4idx.latent_attn(q, latents, table, seq, ctx, most, sc, aws, whole, lse=wlse, status=status)
        assert fp4idx.read_status(status) == 0
        assert counts.tolist()[0] == rows and cu.tolist()[-1] == rows
        # the reference keeps its own, unpaged record of the rows (as stored: bf16)
        want_rows, tol = ref.store(kv[:rows], spos[:rows], norm_kv, 1e-6, cs)
        at = 0
        for b in range(B):
            for i in range(new[b]):
                s = cached[b] + i
                stored = latents[int(table[b, s // 64]), s % 64].double()
                assert bool(((stored - want_rows[at]).abs() <= tol[at]).all())
                truth[b, s] = stored
                at += 1
        at = 0
        for b in range(B):
            for i in range(new[b]):
                L = cached[b] + i + 1
                assert int(ctx[at]) == L and int(seq[at]) == b and int(pos[at]) == L - 1
                picked = [p for p in topk[at].tolist() if p >= 0]
                assert len(picked) == min(k, L) and max(picked) < L
                if i % 23 == 0 or i == new[b] - 1:
                    x = truth[b, picked]
                    ref.check(out[at], lse[at], ref.attend(q[at].double(), x, x[:, :512], sc), "selected")
                    x = truth[b, :L]
                    ref.check(whole[at], wlse[at], ref.attend(q[at].double(), x, x[:, :512], sc), "whole")
                at += 1
        assert bool((out[rows:] == 0).all()) and bool((whole[rows:] == 0).all())
        head += counts[2:3]
        cached_dev += new_dev
        cached = [c + n for c, n in zip(cached, new)]


def test_expanded_and_absorbed_agree():
    """A prompt's attention in both forms: queries and values carried through the expansion
    matrices give the same result as attention over the latents, up to the bf16 roundings of
    the expanded keys and values."""
    from sparse_attention_fp4_gb300 import fp4idx
    g = torch.Generator(device="cuda").manual_seed(2)
    n, H = 150, 4
    latent = bf16(g, n, 512)
    rope = bf16(g, n, 64)
    w_k, w_v = bf16(g, H, 128, 512, scale=512 ** -0.5), bf16(g, H, 128, 512, scale=512 ** -0.5)
    q = bf16(g, n, H, 192)
    key = torch.einsum("hdc,nc->nhd", w_k.float(), latent.float())
    val = torch.einsum("hdc,nc->nhd", w_v.float(), latent.float())
    kv = torch.cat([key, val], 2).to(torch.bfloat16)
    sc = 192 ** -0.5
    out = torch.empty((n, H, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((n, H), dtype=torch.float32, device="cuda")
    fp4idx.latent_prefill(q, kv, rope, i32([0, n]), i32([0, n]), n, n, sc, out, lse=lse)
    q_lat = torch.cat([torch.einsum("nhd,hdc->nhc", q[:, :, :128].float(), w_k.float()), q[:, :, 128:].float()], 2).to(torch.bfloat16)
    cache = fp4idx.alloc_latent_cache(3, 576)
    cache.view(-1, 576)[:n] = torch.cat([latent, rope], 1)
    o_lat = torch.empty((n, H, 512), dtype=torch.bfloat16, device="cuda")
    lse2 = torch.empty((n, H), dtype=torch.float32, device="cuda")
    ws = torch.empty(fp4idx.latent_attn_workspace_bytes(n, H), dtype=torch.uint8, device="cuda")
    fp4idx.latent_attn(q_lat, cache, i32([[0, 1, 2]]), i32([0] * n), i32(list(range(1, n + 1))), n, sc, ws, o_lat, lse=lse2)
    back = torch.einsum("nhc,hdc->nhd", o_lat.float(), w_v.float())
    # scores differ by the roundings of keys (expanded) and of absorbed queries: each 2^-8 of
    # a term, 192 or 576 terms of unit variance times scale; five standard deviations
    ds = 5 * 2.0 ** -8 * 2
    assert float((lse - lse2).abs().max()) <= ds
    # outputs: a weight changes by up to 2 ds; values and outputs have a few bf16 roundings
    bound = (2 * ds + 4 * 2.0 ** -8) * float(val.abs().max())
    assert float((back - out.float()).abs().max()) <= bound
