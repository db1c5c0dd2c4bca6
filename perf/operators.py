"""Cases for the latent-attention operators: what is computed, on which sizes.

Five operators, as a sparse-attention serving step uses them one after another:

  plan     request lengths -> page table, slots, positions, context lengths of the step's rows
  store    new latent rows -> RMSNorm, RoPE -> the paged latent cache
  topk     absorbed latent attention over the tokens that the indexer selected for each row
  dense    absorbed latent attention over the whole context, with or without a tree of drafted tokens
  prefill  expanded latent attention: causal, ragged prompts, per-head keys and values

A latent row has `width` values: all of them are the key, the first 512 are the value.  `run` computes the operators
from elementary torch operations in 32 bits, or, where `own` is true, calls the package.
"""
import math

import torch

own = False

PAGE = 64      # tokens a cache page
VALUE = 512    # value dims of a latent row
ROPE = 64      # rotated dims at the end of a latent row
EPS = 1e-6


# ---------------------------------------------------------------- cases
def listed():
    return [
        # decode step of 64 sequences, one new token each; one cache entry for every 4 tokens
        dict(name="plan decode", op="plan", seqs=64, lo=32768, hi=131072, new_lo=1, new_hi=1, ratio=4, pad=0),
        # chunked prompts beside running sequences: about 64 k rows
        dict(name="plan prompts", op="plan", seqs=256, lo=0, hi=8192, new_lo=1, new_hi=512, ratio=1, pad=77),
        # the new rows of a decode step
        dict(name="store decode", op="store", rows=64, width=512, pages=2048, pad=0),
        # the rows of a prefill batch, with padding rows behind the last sequence
        dict(name="store prefill", op="store", rows=65536, width=576, pages=2048, pad=100),
        # one row over a short selection: latency
        dict(name="topk one row", op="topk", seqs=1, rows=1, heads=64, width=512, lo=4096, hi=4096, k=512, empty=0),
        # a decode batch: long contexts, 2,048 selected tokens a row
        dict(name="topk decode", op="topk", seqs=64, rows=1, heads=64, width=512, lo=8192, hi=32768, k=2048, empty=0),
        # drafted rows, six a sequence; some contexts shorter than the selection, some sequences empty padding
        dict(name="topk drafts", op="topk", seqs=256, rows=6, heads=64, width=576, lo=1024, hi=17408, k=2048, empty=8),
        # a decode batch over the whole context, heads split over several cards
        dict(name="dense decode", op="dense", seqs=64, rows=1, heads=16, width=576, lo=2000, hi=16384, tree=0, empty=1),
        # one long sequence alone: the length is what there is to split
        dict(name="dense long", op="dense", seqs=1, rows=1, heads=128, width=576, lo=60001, hi=60001, tree=0, empty=0),
        # trees of 13 drafted tokens over a cache
        dict(name="tree drafts", op="dense", seqs=32, rows=13, heads=16, width=512, lo=900, hi=9000, tree=1, empty=0),
        # short ragged prompts, some with a cached prefix
        dict(name="prefill short", op="prefill", seqs=9, q_lo=1, q_hi=700, prefix=300, heads=16),
        # long prompts
        dict(name="prefill long", op="prefill", seqs=2, q_lo=4000, q_hi=6000, prefix=0, heads=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "store", "topk", "topk", "dense", "dense", "dense", "prefill"])
    heads = rng.choice([8, 12, 16, 32, 40, 64, 128])
    width = rng.choice([512, 576])
    if op == "plan":
        new_hi = _log(rng, 1, 1024)
        return dict(op=op, seqs=_log(rng, 1, min(4096, 65536 // (new_hi + 1))), lo=rng.randrange(0, 3000), hi=rng.randrange(3000, 60000),
                    new_lo=rng.randrange(0, 2), new_hi=new_hi, ratio=rng.choice([1, 2, 4]), pad=rng.randrange(0, 200))
    if op == "store":
        rows = _log(rng, 1, 60000)
        return dict(op=op, rows=rows, width=width, pages=2048, pad=rng.randrange(0, min(rows, 300)))
    if op == "topk":
        rows, k = rng.randrange(1, 7), _log(rng, 33, 2048)
        seqs = _log(rng, 1, min(128, (1 << 20) // (rows * k)))
        lo = _log(rng, 1, 4000)
        return dict(op=op, seqs=seqs, rows=rows, heads=heads, width=width, lo=lo, hi=lo + _log(rng, 1, 12000), k=k,
                    empty=rng.randrange(0, 2) if seqs > 1 else 0)
    if op == "dense":
        tree = rng.randrange(0, 2)
        rows = rng.randrange(2, 49) if tree else 1
        seqs = _log(rng, 1, 48 if rows == 1 else 400 // rows)
        lo = _log(rng, 1, 5000)
        return dict(op=op, seqs=seqs, rows=rows, heads=heads if not tree else min(heads, 32), width=width, lo=lo,
                    hi=lo + _log(rng, 1, 10000), tree=tree, empty=rng.randrange(0, 2) if seqs > 1 else 0)
    seqs, q_hi = _log(rng, 1, 12), _log(rng, 33, 1500)
    return dict(op=op, seqs=seqs, q_lo=rng.randrange(1, 33), q_hi=q_hi, prefix=rng.choice([0, 1, 77, 1000]),
                heads=rng.choice([1, 3, 8, 16]))


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _lengths(case, n, lo, hi, salt):
    """Whole numbers of [lo, hi], spread evenly and in a fixed order: the sizes are the case's, not the seed's."""
    if n == 1:
        return [hi]
    order = sorted(range(n), key=lambda i: (i * 7919 + salt) % n * n + i)
    got = [0] * n
    for at, i in enumerate(order):
        got[i] = lo + (hi - lo) * at // (n - 1)
    return got


def _row_lengths(case):
    """Context length of each sequence before its rows' own tokens; the last `empty` sequences are padding."""
    L = _lengths(case, case["seqs"], case["lo"], case["hi"], 3)
    for i in range(case["empty"]):
        L[case["seqs"] - 1 - i] = 0
    return L


def _tree_parents(n):
    """A tree of n drafted tokens: node i hangs below a node before it (node 0 is the root)."""
    return [-1] + [(i - 1) // 2 if i % 3 else i - 1 for i in range(1, n)]


def _tree_masks(n):
    """Bit j of mask i: drafted token j is i itself or above it."""
    up, masks = _tree_parents(n), []
    for i in range(n):
        masks.append((1 << i) | (masks[up[i]] if up[i] >= 0 else 0))
    return masks


def _table(lens, g):
    """Pages of each sequence in a random order of one pool: (page_table, pages in the pool)."""
    need = [max(1, -(-n // PAGE)) for n in lens]
    pool = sum(need) + 3
    ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    most = max(need)
    start = torch.tensor([sum(need[:i]) for i in range(len(need))], device="cuda")
    at = start[:, None] + torch.arange(most, device="cuda")[None, :]
    inside = torch.arange(most, device="cuda")[None, :] < torch.tensor(need, device="cuda")[:, None]
    return torch.where(inside, ids[at.clamp(max=pool - 1)], -1).to(torch.int32).contiguous(), pool


def _latents(n, width, g):
    """Latent rows as a cache holds them: unit RMS, a few strong channels."""
    x = torch.randn((n, width), generator=g, device="cuda", dtype=torch.bfloat16)
    x[:, ::97] *= 3
    return x


def _cos_sin(n):
    f = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f[None, :]
    return torch.cat([a.cos(), a.sin()], 1).to(torch.bfloat16)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "plan":
        B, r = case["seqs"], case["ratio"]
        c = torch.randint(case["lo"], case["hi"] + 1, (B,), generator=g, device="cuda")
        n = torch.tensor(_lengths(case, B, case["new_lo"], case["new_hi"], 5), device="cuda")
        held = (c // r + PAGE - 1) // PAGE
        most = (case["hi"] + case["new_hi"]) // r // PAGE + 1
        grown = int(n.sum()) // r // PAGE + 2 * B + 1
        pool = B * most + grown
        ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
        cols = torch.arange(most, device="cuda")[None, :]
        table = torch.where(cols < held[:, None], ids[: B * most].view(B, most), -1).to(torch.int32)
        rows = int(n.sum()) + case["pad"]
        stores = int(n.sum()) // r + B + case["pad"]
        new = lambda m: torch.empty(m, dtype=torch.int32, device="cuda")  # noqa: E731
        return dict(op=op, ratio=r, cached=c.to(torch.int32), new=n.to(torch.int32), table=table.contiguous(),
                    free=ids[B * most:].contiguous(), head=torch.randint(0, 3, (1,), generator=g, device="cuda", dtype=torch.int32),
                    out=[new(rows), new(rows), new(rows), new(stores), new(stores), new(B + 1), new(B + 1), new(4)])
    if op == "store":
        n, w, slots = case["rows"], case["width"], case["pages"] * PAGE
        s = torch.randperm(slots, generator=g, device="cuda")[:n].to(torch.int32)
        s[n - case["pad"]:] = -1
        return dict(op=op, kv=_latents(n, w, g) * 2, slots=s, cos_sin=_cos_sin(65536), cache=torch.zeros((case["pages"], PAGE, w), dtype=torch.bfloat16, device="cuda"),
                    positions=torch.randint(0, 65536, (n,), generator=g, device="cuda", dtype=torch.int32),
                    norm_w=(1 + 0.1 * torch.randn(VALUE, generator=g, device="cuda")).to(torch.bfloat16))
    if op == "prefill":
        nq = _lengths(case, case["seqs"], case["q_lo"], case["q_hi"], 1)
        nk = [a + (case["prefix"] if i % 2 else 0) for i, a in enumerate(nq)]
        cu = lambda v: torch.tensor([sum(v[:i]) for i in range(len(v) + 1)], dtype=torch.int32, device="cuda")  # noqa: E731
        H, Q, K = case["heads"], sum(nq), sum(nk)
        mk = lambda *m: torch.randn(m, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
        return dict(op=op, q=mk(Q, H, 192), kv=mk(K, H, 256), k_rope=mk(K, 64), cu_q=cu(nq), cu_k=cu(nk), max_q=max(nq), max_k=max(nk), scale=192 ** -0.5,
                    out=torch.empty((Q, H, 128), dtype=torch.bfloat16, device="cuda"), lse=torch.empty((Q, H), dtype=torch.float32, device="cuda"))
    B, n, H, w = case["seqs"], case["rows"], case["heads"], case["width"]
    L = _row_lengths(case)
    seq = torch.arange(B, device="cuda", dtype=torch.int32).repeat_interleave(n)
    base = torch.tensor(L, device="cuda", dtype=torch.int32).repeat_interleave(n)
    live = (base > 0).to(torch.int32)
    at = torch.arange(n, device="cuda", dtype=torch.int32).repeat(B)
    drafted = n if op == "dense" and case["tree"] else 0
    table, pool = _table([v + (n if op == "topk" else drafted) if v else 0 for v in L], g)
    T = B * n
    s = dict(op=op, rows=n, q=torch.randn((T, H, w), generator=g, device="cuda", dtype=torch.bfloat16), cache=_latents(pool * PAGE, w, g).view(pool, PAGE, w),
             table=table, row_seq=seq, scale=192 ** -0.5, out=torch.empty((T, H, VALUE), dtype=torch.bfloat16, device="cuda"),
             lse=torch.empty((T, H), dtype=torch.float32, device="cuda"))
    if op == "topk":
        lens = (base + at) * live  # row i of a sequence sees i tokens more
        k = case["k"]
        most = max(int(lens.max()), k)
        order = torch.rand((T, most), generator=g, device="cuda")
        order.masked_fill_(torch.arange(most, device="cuda")[None, :] >= lens[:, None], 2.0)
        pos = order.topk(k, largest=False).indices.to(torch.int32)
        pos = torch.where(torch.arange(k, device="cuda")[None, :] < lens[:, None], pos, 1 << 30).sort(1).values
        s.update(lens=lens, idx=torch.where(pos == 1 << 30, -1, pos).to(torch.int32).contiguous())
    else:
        s.update(lens=base, longest=max(L) + drafted, mask=None)
        if case["tree"]:
            s["mask"] = _words(torch.tensor(_tree_masks(n), device="cuda").repeat(B) * live, (n + 31) // 32)
    return s


def _words(masks, n):
    """Whole-number masks as n 32-bit words each, lowest first."""
    w = (masks.long()[:, None] >> (32 * torch.arange(n, device="cuda"))) & 0xFFFFFFFF
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32).contiguous()


# ---------------------------------------------------------------- plain forms
def _plan(s):
    """Sequence b has c tokens cached and gets n more; an entry of the cache stands for `ratio` tokens."""
    c, n, r, table, free = s["cached"].long(), s["new"].long(), s["ratio"], s["table"], s["free"]
    B, most = table.shape
    rows, stores = s["out"][0].numel(), s["out"][3].numel()
    e0, e1 = c // r, (c + n) // r
    p0, p1 = (e0 + PAGE - 1) // PAGE, (e1 + PAGE - 1) // PAGE
    zero = torch.zeros(1, dtype=torch.long, device=c.device)
    cu = torch.cat([zero, n.cumsum(0)])
    cu_ctx = torch.cat([zero, e1.cumsum(0)])
    cu_e = torch.cat([zero, (e1 - e0).cumsum(0)])
    cu_p = torch.cat([zero, (p1 - p0).cumsum(0)])
    col = torch.arange(most, device=c.device)[None, :]
    take = (s["head"].long() + cu_p[:-1])[:, None] + col - p0[:, None]
    grows = (col >= p0[:, None]) & (col < p1[:, None])
    table.copy_(torch.where(grows, free[take.clamp(0, free.numel() - 1)], table))
    i = torch.arange(rows, device=c.device)
    b = torch.searchsorted(cu[1:], i, right=True)
    ok = b < B
    b = b.clamp(max=B - 1)
    p = torch.where(ok, c[b] + i - cu[b], 0)
    j = torch.arange(stores, device=c.device)
    d = torch.searchsorted(cu_e[1:], j, right=True)
    fine = d < B
    d = d.clamp(max=B - 1)
    e = torch.where(fine, e0[d] + j - cu_e[d], 0)
    slot = torch.where(fine, table[d, e // PAGE].long() * PAGE + e % PAGE, -1)
    counts = torch.stack([cu[-1], cu_e[-1], cu_p[-1], torch.full_like(cu[-1], B)])
    got = [p, torch.where(ok, b, 0), torch.where(ok, (p + 1) // r, 0), e, slot, cu, cu_ctx, counts]
    return [v.to(torch.int32) for v in got] + [table]


def _store(s):
    x = s["kv"].float()
    v = x[:, :VALUE]
    y = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * s["norm_w"].float()
    y = torch.cat([y, x[:, VALUE:]], 1)
    cs = s["cos_sin"][s["positions"].long()].float()
    cos, sin = cs[:, :32], cs[:, 32:]
    a, b = y[:, -ROPE:-ROPE // 2], y[:, -ROPE // 2:]
    y = torch.cat([y[:, :-ROPE], a * cos - b * sin, b * cos + a * sin], 1).to(torch.bfloat16)
    kept = s["slots"] >= 0
    s["cache"].view(-1, y.shape[1])[s["slots"][kept].long()] = y[kept]
    return s["cache"]


def _softmax_sum(scores, seen, values):
    """Over the seen tokens: the softmax-weighted sum of the values, and log(sum(exp(scores))); nothing seen: 0 and -inf."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    out = (p @ values) / torch.where(total == 0, 1.0, total)
    return out, (top + torch.log(total)).squeeze(-1)


def _topk(s):
    idx, q = s["idx"].long(), s["q"].float()
    seen = idx >= 0
    at = idx.clamp(min=0)
    slot = s["table"].long().gather(1, (at // PAGE).view(s["table"].shape[0], -1)).view_as(at) * PAGE + at % PAGE
    rows = s["cache"].view(-1, q.shape[2])[torch.where(seen, slot, 0)].float()
    out, lse = _softmax_sum(s["scale"] * (q @ rows.transpose(1, 2)), seen[:, None, :], rows[:, :, :VALUE])
    return out.to(torch.bfloat16), lse


def _dense(s):
    B, n = s["table"].shape[0], s["rows"]
    T, H, w = s["q"].shape
    at = torch.arange(s["longest"], device=s["q"].device)
    page = s["table"].long()[:, at // PAGE]
    rows = s["cache"].view(-1, w)[page.clamp(min=0) * PAGE + at % PAGE].float()
    base = s["lens"].long()[:, None]
    seen = at < base
    if s["mask"] is not None:
        bit = at - base
        word = s["mask"].long().gather(1, (bit // 32).clamp(0, s["mask"].shape[1] - 1))
        inside = (bit >= 0) & (bit < 32 * s["mask"].shape[1])
        seen = seen | (inside & ((word >> (bit % 32)) & 1 == 1))
    seen = seen[:, None, :].expand(T, H, -1).reshape(B, n * H, -1)
    scores = s["scale"] * (s["q"].float().view(B, n * H, w) @ rows.transpose(1, 2))
    out, lse = _softmax_sum(scores, seen, rows[:, :, :VALUE])
    return out.view(T, H, VALUE).to(torch.bfloat16), lse.view(T, H)


def _prefill(s):
    cq, ck = s["cu_q"].long(), s["cu_k"].long()
    Q, K, dev = s["q"].shape[0], s["kv"].shape[0], s["q"].device
    i, j = torch.arange(s["max_q"], device=dev), torch.arange(s["max_k"], device=dev)
    nq, nk = (cq[1:] - cq[:-1])[:, None], (ck[1:] - ck[:-1])[:, None]
    qi, kj = (cq[:-1, None] + i).clamp(max=Q - 1), (ck[:-1, None] + j).clamp(max=K - 1)
    q = s["q"][qi].float().transpose(1, 2)
    kv = s["kv"][kj].float().transpose(1, 2)
    scores = q[..., :128] @ kv[..., :128].transpose(2, 3) + q[..., 128:] @ s["k_rope"][kj].float().transpose(1, 2)[:, None]
    seen = (j[None, None, :] < nk[:, :, None]) & (j[None, None, :] <= (nk - nq)[:, :, None] + i[None, :, None])
    out, lse = _softmax_sum(scores.mul_(s["scale"]), seen[:, None], kv[..., 128:])
    b = torch.searchsorted(cq[1:], torch.arange(Q, device=dev), right=True)
    at = torch.arange(Q, device=dev) - cq[b]
    return out[b, :, at].to(torch.bfloat16), lse[b, :, at]


# ---------------------------------------------------------------- the framework's calls
def _workspace(s, need):
    """A workspace is kept with the buffers of a program."""
    if "ws" not in s:
        s["ws"] = torch.empty(need(), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _own(s):
    from sparse_attention_fp4_gb300 import fp4idx
    op = s["op"]
    if op == "plan":
        pos, seq, ctx, spos, slots, cu, cu_ctx, counts = s["out"]
        fp4idx.plan_step(s["cached"], s["new"], s["ratio"], s["free"], s["table"], pos, seq, ctx, spos, slots, cu, cu_ctx, counts, free_head=s["head"])
        return s["out"] + [s["table"]]
    if op == "store":
        fp4idx.store_latent(s["kv"], s["positions"], s["slots"], s["norm_w"], EPS, s["cos_sin"], s["cache"])
        return s["cache"]
    if op == "topk":
        T, H, w = s["q"].shape
        ws = _workspace(s, lambda: fp4idx.latent_attn_workspace_bytes(T, H))
        fp4idx.latent_attn_topk(s["q"], s["cache"], s["table"], s["row_seq"], s["idx"], s["scale"], ws, s["out"], lse=s["lse"], context_lens=s["lens"])
    elif op == "dense":
        T, H, w = s["q"].shape
        ws = _workspace(s, lambda: fp4idx.latent_attn_workspace_bytes(T, H))
        fp4idx.latent_attn(s["q"], s["cache"], s["table"], s["row_seq"], s["lens"], s["longest"], s["scale"], ws, s["out"], lse=s["lse"], tree_mask=s["mask"])
    else:
        fp4idx.latent_prefill(s["q"], s["kv"], s["k_rope"], s["cu_q"], s["cu_k"], s["max_q"], s["max_k"], s["scale"], s["out"], lse=s["lse"])
    return s["out"], s["lse"]


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    return _plan(state) if op == "plan" else _store(state) if op == "store" else _topk(state) if op == "topk" else _dense(state) if op == "dense" else _prefill(state)


# ---------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "plan":
        B, r = case["seqs"], case["ratio"]
        n = sum(_lengths(case, B, case["new_lo"], case["new_hi"], 5))
        # lengths in; three arrays a row, two a stored entry, the new pages' ids in and out, two offsets a sequence
        return dict(bytes=4 * (2 * B + 3 * (n + case["pad"]) + 2 * (n // r + B + case["pad"]) + 2 * (n // r // PAGE) + 2 * B + 6), flops=n)
    if op == "store":
        n, w = case["rows"] - case["pad"], case["width"]
        return dict(bytes=n * (4 * w + 2 * ROPE + 8) + 4 * case["pad"] + 2 * VALUE, flops=n * (4 * VALUE + 3 * ROPE))
    H = case["heads"]
    if op == "prefill":
        nq = _lengths(case, case["seqs"], case["q_lo"], case["q_hi"], 1)
        nk = [a + (case["prefix"] if i % 2 else 0) for i, a in enumerate(nq)]
        pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(nq, nk))
        Q, K = sum(nq), sum(nk)
        return dict(bytes=2 * (Q * H * (192 + 128) + K * H * 256 + K * 64) + 4 * Q * H, flops=2 * 320 * H * pairs)
    n, w = case["rows"], case["width"]
    L = _row_lengths(case)
    T = n * len(L)
    io = T * H * (2 * w + 2 * VALUE + 4)
    if op == "topk":
        k = case["k"]
        pairs = sum(min(k, v + i) for v in L if v for i in range(n))
        # tokens of a sequence that one of its rows selects at least once, each read once: the selections are drawn independently
        read = sum(v * (1 - (1 - min(1.0, k / v)) ** n) for v in L if v)
        return dict(bytes=2 * w * int(read) + 4 * pairs + io, flops=2 * (w + VALUE) * H * pairs)
    drafted = n if case["tree"] else 0
    above = sum(bin(m).count("1") for m in _tree_masks(n)) if case["tree"] else 0
    live = [v for v in L if v]
    pairs = sum(v * n + above for v in live)
    return dict(bytes=2 * w * sum(v + drafted for v in live) + io, flops=2 * (w + VALUE) * H * pairs)


# ---------------------------------------------------------------- from the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "plan":
        return None
    d = torch.float64
    if op == "store":
        out = s["cache"].to(d)
        flat = out.view(-1, case["width"])
        live = [i for i, v in enumerate(s["slots"].tolist()) if v >= 0]
        x = s["kv"][live].to(d)
        ms = (x[:, :VALUE] ** 2).sum(1) / VALUE + EPS
        x[:, :VALUE] *= s["norm_w"].to(d)[None, :] / ms.sqrt()[:, None]
        t = s["cos_sin"][s["positions"][live].long()].to(d)
        lo, hi = case["width"] - ROPE, case["width"] - ROPE // 2
        z = torch.complex(x[:, lo:hi].clone(), x[:, hi:].clone()) * torch.complex(t[:, :32].clone(), t[:, 32:].clone())
        x[:, lo:hi], x[:, hi:] = z.real, z.imag
        flat[s["slots"][live].long()] = x
        return out
    if op == "prefill":
        out, lse = torch.zeros(s["out"].shape, dtype=d, device="cuda"), torch.full(s["lse"].shape, -math.inf, dtype=d, device="cuda")
        cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
        for b in range(case["seqs"]):
            nq, nk = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
            for h in range(case["heads"]):
                kv = s["kv"][ck[b]:ck[b + 1], h].to(d)
                key = torch.cat([kv[:, :128], s["k_rope"][ck[b]:ck[b + 1]].to(d)], 1)
                z = (s["q"][cq[b]:cq[b + 1], h].to(d) @ key.T) * s["scale"]
                hidden = torch.ones((nq, nk), dtype=torch.bool, device="cuda").triu(nk - nq + 1)
                z[hidden] = -math.inf
                lse[cq[b]:cq[b + 1], h] = torch.logsumexp(z, 1)
                out[cq[b]:cq[b + 1], h] = torch.softmax(z, 1) @ kv[:, 128:]
        return out, lse
    n = case["rows"]
    out, lse = torch.zeros(s["out"].shape, dtype=d, device="cuda"), torch.full(s["lse"].shape, -math.inf, dtype=d, device="cuda")
    flat = s["cache"].view(-1, case["width"])
    lens = s["lens"].tolist()
    masks = _tree_masks(n) if op == "dense" and case["tree"] else [0] * n
    everything = torch.arange(case["hi"] + n, device="cuda")
    for t in range(len(lens)):
        b, i = divmod(t, n)
        if lens[t] == 0:
            continue
        if op == "topk":
            tokens = s["idx"][t].long()[: min(case["k"], lens[t])]
        else:
            own_path = [lens[t] + j for j in range(n) if masks[i] >> j & 1]
            tokens = torch.cat([everything[: lens[t]], everything.new_tensor(own_path)])
        x = flat[s["table"][b].long()[tokens // PAGE] * PAGE + tokens % PAGE].to(d)
        z = (s["q"][t].to(d) @ x.T) * s["scale"]
        lse[t] = torch.logsumexp(z, 1)
        out[t] = torch.softmax(z, 1) @ x[:, :VALUE]
    return out, lse
