"""Cases for the operators around beam search and the page pool: what is computed, on which sizes.

Four operators, as a serving step that decodes several hypotheses a request uses them one after another:

  select   logits and running scores of the beams -> the best continuations of each request
  fork     page tables -> page tables of the chosen continuations: whole pages shared, half-filled ones listed for
           copying, pages that nobody holds any more back on the free list
  copy     the listed pages copied in every cache
  compact  the pages in use get the lowest ids: new tables, a list of moves, the free list rebuilt

`run` computes the operators from elementary torch operations, or, where `own` is true, calls the package.  The
totals of `select` are compared with one another, so the plain form takes them in 64 bits.
"""
import math

import torch

own = False

PAGE = 64   # entries a cache page
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one request with four beams: latency
        dict(name="select one", op="select", groups=1, beams=4, vocab=32000, k=4, type="bf16", pad=0, first=0, done=0.0, kept=1.0),
        # a decode step of 64 requests, twice as many continuations as beams, so that ended ones can be set aside
        dict(name="select step", op="select", groups=64, beams=4, vocab=131072, k=8, type="bf16", pad=0, first=0, done=0.0, kept=1.0),
        # rows of an odd length, finished beams that stay, a grammar that leaves one token in fifty
        dict(name="select masked", op="select", groups=16, beams=5, vocab=50001, k=5, type="fp16", pad=2, first=0, done=0.2, kept=0.02),
        # wide beams over fp32 logits
        dict(name="select wide", op="select", groups=8, beams=32, vocab=131072, k=64, type="fp32", pad=0, first=0, done=0.05, kept=1.0),
        # 16 requests with four beams, index keys (an entry for every 4 tokens)
        dict(name="fork step", op="fork", groups=16, beams=4, lo=8192, hi=32768, ratio=4, shared=0.97, spare=310, ended=0, pinned=0, grow=0),
        # the step behind the prompts: one row a request becomes six
        dict(name="fork first", op="fork", groups=60, beams=6, lo=100, hi=9000, ratio=1, shared=0.0, spare=400, ended=0, pinned=0, grow=1),
        # 64 requests with four beams, an entry a token, long shared prompts held by a prefix cache, some requests at their end
        dict(name="fork long", op="fork", groups=64, beams=4, lo=5000, hi=60001, ratio=1, shared=0.9, spare=999, ended=7, pinned=20, grow=0),
        # the half-filled pages of a fork, in the index keys and the latent rows of four layers: latency
        dict(name="copy tails", op="copy", pages=48, pool=2048, layers=4, width=576, pad=16),
        # index keys alone: many small pages
        dict(name="copy index", op="copy", pages=20000, pool=40960, layers=1, width=0, pad=0),
        # moves of a compaction, latent rows
        dict(name="copy moves", op="copy", pages=4001, pool=9000, layers=1, width=512, pad=95),
        # a small pool
        dict(name="compact small", op="compact", groups=16, beams=4, lo=1024, hi=17408, ratio=4, shared=0.9, spare=100, ended=0, pinned=0, moves=4096),
        # a large one, with a bound on the moves of one step
        dict(name="compact pool", op="compact", groups=64, beams=4, lo=5000, hi=60001, ratio=1, shared=0.8, spare=4999, ended=7, pinned=20, moves=20000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["select", "select", "select", "fork", "fork", "copy", "copy", "compact", "compact"])
    if op == "select":
        kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        beams, vocab = _log(rng, 1, 32), _log(rng, 200, 262144)
        groups = _log(rng, 1, max(1, min(256, (1 << 25) // (beams * (vocab + 8) * (2 if kind == "fp32" else 1)))))
        return dict(op=op, groups=groups, beams=beams, vocab=vocab, k=min(64, rng.choice([1, beams, beams, 2 * beams, _log(rng, 1, 64)])),
                    type=kind, pad=rng.choice([0, 0, 1, 3, 8]), first=int(rng.random() < 0.15), done=rng.choice([0.0, 0.0, 0.1, 0.5]),
                    kept=rng.choice([1.0, 1.0, 1.0, 0.5, 0.01, 0.0005]))
    if op == "copy":
        layers, width = rng.choice([1, 1, 2, 4, 8]), rng.choice([0, 512, 576])
        page = layers * (4352 + 128 * width)
        pages = _log(rng, 1, min(8000, 260_000_000 // page))
        return dict(op=op, pages=pages, pool=2 * pages + rng.randrange(1, 500), layers=layers, width=width, pad=rng.randrange(0, 40))
    lo, ratio = _log(rng, 700, 20000), rng.choice([1, 1, 2, 4])
    case = dict(op=op, groups=_log(rng, 1, 60), beams=rng.choice([1, 2, 3, 4, 5]), lo=lo, hi=lo + _log(rng, 1, 30000), ratio=ratio,
                shared=rng.choice([0.0, 0.5, 0.9, 0.99]), spare=rng.randrange(310, 1000), ended=rng.randrange(0, 2), pinned=rng.choice([0, 0, 3, 40]))
    if op == "compact":
        case["moves"] = _log(rng, 1, 20000)
    else:
        case["grow"] = int(rng.random() < 0.25)
    return case


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _lengths(n, lo, hi):
    """Whole numbers of [lo, hi], spread evenly and in a fixed order: the sizes are the case's, not the seed's."""
    if n == 1:
        return [hi]
    order = sorted(range(n), key=lambda i: (i * 7919 + 3) % n * n + i)
    got = [0] * n
    for at, i in enumerate(order):
        got[i] = lo + (hi - lo) * at // (n - 1)
    return got


def _empty(*m, dtype=torch.int32):
    return torch.empty(m, dtype=dtype, device="cuda")


def _tables(case, g):
    """Beams of a request share its prompt's pages; each parts from the beam before it somewhere behind the prompt."""
    G, W, r = case["groups"], case["beams"], case["ratio"]
    tokens = torch.tensor(_lengths(G, case["lo"], case["hi"]), device="cuda")
    entries = tokens // r
    pages = (entries + PAGE - 1) // PAGE
    most = (case["hi"] // r + PAGE - 1) // PAGE + 2
    pool = G * W * most + case["spare"]
    ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    fresh = ids[: G * W * most].view(G, W, most)
    col = torch.arange(most, device="cuda")
    prompt = (entries * case["shared"]).long() // PAGE
    table = torch.empty_like(fresh)
    for b in range(W):
        part = prompt + ((entries // PAGE - prompt + 1) * torch.rand(G, generator=g, device="cuda")).long()
        part = torch.minimum(part, entries // PAGE)
        table[:, b] = fresh[:, b] if b == 0 else torch.where(col < part[:, None], table[:, b - 1], fresh[:, b])
    table = torch.where(col < pages[:, None, None], table, -1)
    pins = torch.zeros((pool + 31) // 32 * 32, dtype=torch.bool, device="cuda")
    if case["pinned"]:  # a prefix cache holds the first pages of each prompt
        held = table[:, 0, : case["pinned"]][(col[: case["pinned"]] < prompt[:, None])]
        pins[held.long()] = True
    return dict(ratio=r, num_pages=pool, table=table.reshape(G * W, most).contiguous(), cached=tokens.repeat_interleave(W).to(torch.int32),
                free=ids[G * W * most:].contiguous(), table_out=_empty(G * W, most), counts=_empty(4), pinned=_words(pins) if case["pinned"] else None)


def _words(bits):
    w = (bits.view(-1, 32).long() << torch.arange(32, device="cuda")).sum(1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "select":
        G, W, V, k = case["groups"], case["beams"], case["vocab"], case["k"]
        R = G * W
        x = 2 * torch.randn((R, V + case["pad"]), generator=g, device="cuda")
        peaks = torch.randint(0, V, (R, 24), generator=g, device="cuda")
        x.scatter_add_(1, peaks, 6 + 2 * torch.randn(R, 24, generator=g, device="cuda"))
        if case["kept"] < 1:
            x.masked_fill_(torch.rand(x.shape, generator=g, device="cuda") >= case["kept"], -math.inf)
        scores = -20 * torch.rand(R, generator=g, device="cuda") ** 2 - 1
        if case["first"]:
            scores.view(G, W)[:, 1:] = -math.inf
        done = (torch.rand(R, generator=g, device="cuda") < case["done"]).to(torch.int32)
        return dict(op=op, beams=W, k=k, logits=x.to(TYPES[case["type"]])[:, :V], scores=scores, done=done, end=V // 3,
                    out=[_empty(G * k, dtype=torch.float32), _empty(G * k), _empty(G * k), _empty(G * k)])
    if op == "copy":
        n, pool = case["pages"], case["pool"]
        ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
        pad = torch.full((case["pad"],), -1, dtype=torch.int32, device="cuda")
        caches = []
        for _ in range(case["layers"]):
            caches.append(torch.randint(0, 256, (pool, 4, PAGE, 16), generator=g, device="cuda", dtype=torch.uint8))
            caches.append(torch.randint(110, 140, (pool, 4, PAGE), generator=g, device="cuda", dtype=torch.uint8))
            if case["width"]:
                caches.append(torch.randn((pool, PAGE, case["width"]), generator=g, device="cuda", dtype=torch.bfloat16))
        return dict(op=op, src=torch.cat([ids[:n], pad]), dst=torch.cat([ids[n:2 * n], pad]), caches=caches,
                    count=torch.tensor([n], dtype=torch.int32, device="cuda"))
    s = _tables(case, g)
    G, W = case["groups"], case["beams"]
    R = G * W
    s["op"] = op
    if op == "fork":
        # each beam goes on from a beam of its request (behind the prompts: from its one row); the last requests have ended
        if case["grow"]:
            s["table"], s["cached"] = s["table"][::W].contiguous(), s["cached"][::W].contiguous()
            up = torch.arange(G, device="cuda")[:, None].repeat(1, W)
        else:
            up = torch.randint(0, W, (G, W), generator=g, device="cuda") + W * torch.arange(G, device="cuda")[:, None]
        if G > case["ended"] > 0:
            up[G - case["ended"]:] = -1
        # pages that come back go below the list's head: there is room for all of the pool
        s["free"] = torch.cat([torch.full((s["num_pages"],), -1, dtype=torch.int32, device="cuda"), s["free"]])
        s.update(parents=up.reshape(-1).to(torch.int32), head=torch.tensor([s["num_pages"] + 5], dtype=torch.int32, device="cuda"),
                 cached_out=_empty(R), src=_empty(R), dst=_empty(R))
    else:
        s.update(src=_empty(case["moves"]), dst=_empty(case["moves"]), free=torch.full((s["num_pages"],), -1, dtype=torch.int32, device="cuda"))
    return s


# ---------------------------------------------------------------- plain forms
def _select(s):
    x, W, k = s["logits"].double(), s["beams"], s["k"]
    R, V = x.shape
    top = x.amax(1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    lse = top + torch.log(torch.exp(x - top).sum(1, keepdim=True))
    score = s["scores"].double()[:, None]
    total = torch.where(torch.isfinite(lse) & torch.isfinite(score), score + (x - lse), -math.inf)
    done = s["done"][:, None] != 0
    at_end = torch.arange(V, device=x.device)[None, :] == s["end"]
    total = torch.where(done, torch.where(at_end, score, -math.inf), total)
    best, at = torch.sort(total.view(R // W, W * V), dim=1, descending=True, stable=True)
    if best.shape[1] < k:
        best = torch.nn.functional.pad(best, (0, k - best.shape[1]), value=-math.inf)
        at = torch.nn.functional.pad(at, (0, k - at.shape[1]))
    best, at = best[:, :k], at[:, :k]
    live = best > -math.inf
    row = torch.where(live, at // V + W * torch.arange(R // W, device=x.device)[:, None], -1)
    token = torch.where(live, at % V, -1)
    ended = live & ((s["done"][row.clamp(min=0)] != 0) | (token == s["end"]))
    return [best.float().reshape(-1), row.reshape(-1).to(torch.int32), token.reshape(-1).to(torch.int32), ended.reshape(-1).to(torch.int32)]


def _held(s, rows, pool):
    """Which pages the marked rows hold."""
    table = s["table"].long()
    n = ((s["cached"].long() // s["ratio"] + PAGE - 1) // PAGE)[:, None]
    valid = (torch.arange(table.shape[1], device=table.device)[None, :] < n) & rows[:, None]
    hit = torch.zeros(pool + 1, dtype=torch.bool, device=table.device)
    hit[torch.where(valid, table, pool)] = True
    return hit[:pool]


def _bits(words, pool):
    if words is None:
        return torch.zeros(pool, dtype=torch.bool, device="cuda")
    return ((words.long()[:, None] >> torch.arange(32, device="cuda")) & 1).reshape(-1)[:pool] == 1


def _ranks(mask):
    return mask.long().cumsum(0) - 1


def _packed(mask, n):
    """The first n positions of a mask, -1 behind the last one."""
    got = torch.full((n + 1,), -1, dtype=torch.long, device=mask.device)
    rank = _ranks(mask)
    got[torch.where(mask & (rank < n), rank, n)] = torch.arange(mask.numel(), device=mask.device)
    return got[:n]


def _fork(s):
    table, up, pool = s["table"].long(), s["parents"].long(), s["num_pages"]
    dev, (old, most), new = table.device, table.shape, up.numel()
    entries = s["cached"].long() // s["ratio"]
    goes = up >= 0
    par = up.clamp(min=0)
    kept = torch.zeros(old + 1, dtype=torch.bool, device=dev)
    kept[torch.where(goes, up, old)] = True
    kept = kept[:old]
    pins = _bits(s["pinned"], pool)
    back = _held(s, ~kept, pool) & ~_held(s, kept, pool) & ~pins
    freed = back.sum()
    ids = _packed(back, pool)
    # half-filled pages: the first row that goes on from a parent keeps it, unless it is pinned
    i = torch.arange(new, device=dev)
    first = torch.full((old + 1,), new, dtype=torch.long, device=dev).scatter_reduce(0, torch.where(goes, up, old), i, "amin")
    tail = entries[par] // PAGE
    half = goes & (entries[par] % PAGE != 0)
    page = table[par, tail.clamp(max=most - 1)]
    copied = half & ((first[par] != i) | pins[page.clamp(min=0)])
    c = _ranks(copied)
    n = copied.sum()
    head = s["head"].long()[0]
    fresh = torch.where(c < freed, ids[c.clamp(0, pool - 1)], s["free"][(head + c - freed).clamp(0, s["free"].numel() - 1)].long())
    pages = torch.where(goes, (entries[par] + PAGE - 1) // PAGE, 0)
    col = torch.arange(most, device=dev)[None, :]
    out = torch.where(col < pages[:, None], table[par], -1)
    out = torch.where(copied[:, None] & (col == tail[:, None]), fresh[:, None], out)
    at = _packed(copied, new)
    src = torch.where(at >= 0, page[at.clamp(min=0)], -1)
    dst = torch.where(at >= 0, fresh[at.clamp(min=0)], -1)
    # what is left of the pages that came back lies below the head of the list
    slot = torch.arange(s["free"].numel(), device=dev) - (head - (freed - n))
    s["free"].copy_(torch.where((slot >= 0) & (slot < freed - n), ids[(n + slot).clamp(0, pool - 1)], s["free"].long()))
    counts = torch.stack([n, freed, n - freed, goes.sum()])
    return [v.to(torch.int32) for v in (out, torch.where(goes, s["cached"][par], 0), src, dst, counts)] + [s["free"]]


def _copy(s):
    live = s["src"] >= 0
    src, dst = s["src"][live].long(), s["dst"][live].long()
    for c in s["caches"]:
        c[dst] = c[src]
    return s["caches"]


def _compact(s):
    pool, moves = s["num_pages"], s["src"].numel()
    dev = s["table"].device
    ids = torch.arange(pool, device=dev)
    pins = _bits(s["pinned"], pool)
    used = _held(s, s["cached"] >= 0, pool) | pins
    n = used.sum()
    hole, mover = ~used & (ids < n), used & ~pins & (ids >= n)
    rank = _ranks(mover)
    goes = mover & (rank < moves)
    src = _packed(goes, moves)
    dst = torch.where(src >= 0, _packed(hole, moves), -1)
    to = torch.where(goes, dst[rank.clamp(0, moves - 1)], ids)
    table = s["table"].long()
    held = ((s["cached"].long() // s["ratio"] + PAGE - 1) // PAGE)[:, None]
    valid = torch.arange(table.shape[1], device=dev)[None, :] < held
    out = torch.where(valid, to[torch.where(valid, table, 0)], -1)
    after = torch.zeros(pool + 1, dtype=torch.bool, device=dev)
    after[torch.where(used, to, pool)] = True
    after = after[:pool]
    free = _packed(~after, pool)
    # the lowest ids are taken first; the list ends where its buffer ends
    head = s["free"].numel() - (pool - n)
    at = torch.arange(s["free"].numel(), device=dev) - head
    s["free"].copy_(torch.where(at >= 0, free[at.clamp(0, pool - 1)], s["free"].long()))
    end = torch.where(after, ids + 1, 0).amax()
    counts = torch.stack([goes.sum(), n, end, head])
    return [v.to(torch.int32) for v in (out, src, dst, counts)] + [s["free"]]


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    from sparse_attention_fp4_gb300 import fp4idx
    op = s["op"]
    if op == "select":
        if "ws" not in s:  # a workspace is kept with the buffers of a program
            s["ws"] = torch.empty(fp4idx.beam_select_workspace_bytes(s["logits"].shape[0], s["logits"].shape[1], s["k"]), dtype=torch.uint8, device="cuda")
        scores, rows, tokens, ended = s["out"]
        fp4idx.beam_select(s["logits"], s["scores"], s["beams"], s["k"], s["ws"], scores, rows, tokens, done=s["done"], end_token=s["end"], done_out=ended)
        return s["out"]
    if op == "copy":
        fp4idx.copy_pages(s["src"], s["dst"], s["caches"], count=s["count"])
        return s["caches"]
    if op == "fork":
        fp4idx.fork_pages(s["table"], s["cached"], s["ratio"], s["parents"], s["num_pages"], s["free"], s["table_out"], s["cached_out"], s["src"],
                          s["dst"], s["counts"], free_head=s["head"], pinned=s["pinned"])
        return [s["table_out"], s["cached_out"], s["src"], s["dst"], s["counts"], s["free"]]
    if "ws" not in s:
        s["ws"] = torch.empty(fp4idx.compact_pages_workspace_bytes(s["num_pages"]), dtype=torch.uint8, device="cuda")
    fp4idx.compact_pages(s["table"], s["cached"], s["ratio"], s["num_pages"], s["ws"], s["free"], s["table_out"], s["src"], s["dst"], s["counts"],
                         pinned=s["pinned"])
    return [s["table_out"], s["src"], s["dst"], s["counts"], s["free"]]


def run(state):
    if own:
        return _own(state)
    return {"select": _select, "fork": _fork, "copy": _copy, "compact": _compact}[state["op"]](state)


# ---------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "select":
        rows = case["groups"] * (1 if case["first"] else case["beams"])
        n = int(rows * (1 - case["done"])) * case["vocab"]
        # a subtraction, an exponential, a sum and a comparison an element
        return dict(bytes=n * (4 if case["type"] == "fp32" else 2) + 8 * rows + 16 * case["groups"] * case["k"], flops=4 * n)
    if op == "copy":
        return dict(bytes=2 * case["pages"] * case["layers"] * (4352 + 128 * case["width"]) + 8 * case["pages"], flops=case["pages"])
    G, W, r = case["groups"], case["beams"], case["ratio"]
    most = (case["hi"] // r + PAGE - 1) // PAGE + 2
    old = 1 if op == "fork" and case["grow"] else W
    pages = old * sum((v // r + PAGE - 1) // PAGE for v in _lengths(G, case["lo"], case["hi"]))
    pool = G * W * most + case["spare"]
    pins = pool // 8 if case["pinned"] else 0
    # the entries in use in, the whole new table out, lengths and parents in and out; the pages that come back are few
    io = 4 * pages + 4 * G * W * most + pins + 16 * G * W + 16
    if op == "fork":
        return dict(bytes=io + 8 * G * W, flops=pages)
    # moves out, the free list out (what the requests' pages leave of the pool, at the least)
    return dict(bytes=io + 8 * case["moves"] + 4 * (pool - pages), flops=pages + pool // 32)


# ---------------------------------------------------------------- from the definitions, in 64 bits
def exact(case, seed):
    if case["op"] != "select":
        return None
    s = prepare(case, seed)
    W, k, d = case["beams"], case["k"], torch.float64
    got = []
    for g in range(case["groups"]):
        totals = []
        for r in range(g * W, (g + 1) * W):
            score = s["scores"][r].to(d)
            if int(s["done"][r]):
                totals.append(score.view(1))
            elif float(score) > -math.inf:
                x = s["logits"][r].to(d)
                x = x[x > -math.inf]
                if x.numel():
                    totals.append(score + torch.topk(torch.log_softmax(x, 0), min(k, x.numel())).values)
        t = torch.cat(totals) if totals else torch.empty(0, dtype=d, device="cuda")
        t = t[t > -math.inf].sort(descending=True).values[:k]
        got.append(torch.nn.functional.pad(t, (0, k - t.numel()), value=-math.inf))
    return [torch.cat(got), None, None, None]
