"""Plain references of the beam selection (float64) and of the page pool's operators (whole numbers)."""
import math

import numpy as np

PAGE = 64


# ---------------------------------------------------------------- beam selection
def totals(logits, scores, beams, done=None, end=-1):
    """Per group the candidates (total, row, logit, token) in order, from float64 arrays."""
    R, V = logits.shape
    out = []
    for g in range(R // beams):
        got = []
        for r in range(g * beams, (g + 1) * beams):
            s = float(scores[r])
            if s == -math.inf or math.isnan(s) or s == math.inf:
                continue
            if done is not None and done[r]:
                got.append((s, r, 0.0, end))
                continue
            x = logits[r].astype(np.float64)
            if np.isnan(x).any() or (x == np.inf).any() or (x == -np.inf).all():
                continue
            m = x.max()
            rest = math.log(np.exp(x - m).sum())  # lse = m + rest
            at = np.nonzero(x > -np.inf)[0]
            t = s + ((x[at] - m) - rest)
            keep = np.lexsort((at, -x[at]))[:256]
            got += [(float(t[i]), r, float(x[at[i]]), int(at[i])) for i in keep]
        got.sort(key=lambda c: (-c[0], c[1], -c[2], c[3]))
        out.append(got)
    return out


def check_select(got, logits, scores, beams, k, done=None, end=-1):
    """got: scores, rows, tokens (and done_out) as [groups, k] arrays.  A total is off by one rounding to fp32 and by lse's
    error, in units of 2^-24 of the sum of exponentials: 4 of an exponential (2^-22), 4 of its argument (two
    roundings of a number t that weighs 2^-t), 10 additions within a tile; per tile of its thread (of 2,048 logits of a
    row at the least, 64 at the most) one addition and, where its largest rises, a factor within 5; 2 for joining
    threads and chunks, the logarithm and the totals (some 36 bits or more).  Candidates whose totals are closer
    than twice that may change places (within a row the order is exact)."""
    out_s, out_r, out_t, out_d = got
    want = totals(logits, scores, beams, done, end)
    eps = (20 + 6 * min(64, -(-logits.shape[1] // 2048))) * 2.0 ** -24
    for g, w in enumerate(want):
        n = min(k, len(w))
        assert (out_r[g, n:] == -1).all() and (out_t[g, n:] == -1).all() and (out_s[g, n:] == -np.inf).all(), g
        assert (out_r[g, :n] >= 0).all(), g
        by = {(c[1], c[3]): c for c in w}
        seen = set()
        for i in range(n):
            key = (int(out_r[g, i]), int(out_t[g, i]))
            assert key in by and key not in seen, (g, i, key)
            seen.add(key)
            c = by[key]
            assert abs(out_s[g, i] - c[0]) <= eps + abs(c[0]) * 2.0 ** -24, (g, i, out_s[g, i], c)
            assert abs(c[0] - w[i][0]) <= 2 * eps, (g, i, c, w[i])
            near = any(0 <= j < len(w) and w[j][1] != w[i][1] and abs(w[j][0] - w[i][0]) <= 2 * eps for j in (i - 1, i + 1))
            if not near and not (i and key != (w[i][1], w[i][3]) and abs(w[i - 1][0] - w[i][0]) <= 2 * eps):
                assert key == (w[i][1], w[i][3]), (g, i, key, w[i])
        for r in set(c[1] for c in w):  # within a row: in order, none left out
            mine = [int(out_t[g, i]) for i in range(n) if int(out_r[g, i]) == r]
            assert mine == [c[3] for c in w if c[1] == r][:len(mine)], (g, r)
        if out_d is not None:
            for i in range(k):
                ended = i < n and (bool(done is not None and done[int(out_r[g, i])]) or int(out_t[g, i]) == end)
                assert bool(out_d[g, i]) == ended, (g, i)


# ---------------------------------------------------------------- page tables
def held(length, ratio, most):
    n = -(-(length // ratio) // PAGE)
    return -1 if length < 0 or n > most else n


def fork(table, cached, ratio, parents, pool, free, head, pinned=()):
    """Lists in, dict out; what the library writes, and the status codes that may be recorded."""
    table = [list(t) for t in table]
    most = len(table[0]) if table else 1
    free, bad = list(free), set()
    n_pages = [held(c, ratio, most) for c in cached]
    kept, first = set(), {}
    for i, p in enumerate(parents):
        if 0 <= p < len(table):
            kept.add(p)
            first.setdefault(p, i)
        elif p != -1:
            bad.add(5)
    gone, stay = set(), set()
    for r in range(len(table)):
        if n_pages[r] < 0:
            bad.add(8)
            continue
        for page in table[r][:n_pages[r]]:
            if 0 <= page < pool:
                (stay if r in kept else gone).add(page)
            else:
                bad.add(5)
    back = sorted(p for p in gone - stay if p not in pinned)
    good_head = 0 <= head <= len(free)
    if not good_head:
        head_used, avail = 0, []
    else:
        head_used, avail = head, free[head:]
    fresh = back + avail
    out, cached_out, src, dst, rows = [], [], [], [], 0
    n_copies = 0
    for i, p in enumerate(parents):
        if not 0 <= p < len(table) or n_pages[p] < 0:
            out.append([-1] * most)
            cached_out.append(0)
            continue
        row = table[p][:n_pages[p]] + [-1] * (most - n_pages[p])
        e = cached[p] // ratio
        own = False
        if e % PAGE:
            page = row[e // PAGE]
            own = 0 <= page < pool and (first[p] != i or page in pinned)
        if own:
            n_copies += 1
            if len(src) == len(fresh):
                bad.add(11)
                out.append([-1] * most)
                cached_out.append(0)
                continue
            src.append(page)
            dst.append(fresh[len(dst)])
            row[e // PAGE] = dst[-1]
        out.append(row)
        cached_out.append(cached[p])
        rows += 1
    left = back[n_copies:]
    listed = left[max(0, len(left) - head_used):]
    if len(listed) < len(left) or not good_head:
        bad.add(11)
    if listed:
        free[head_used - len(listed):head_used] = listed
    change = -len(listed) if len(back) > n_copies else len(src) - len(back)
    pad = [-1] * (len(parents) - len(src))
    return dict(table=out, cached=cached_out, src=src + pad, dst=dst + pad, counts=[len(src), len(back), change, rows], free=free, bad=bad)


def compact(table, cached, ratio, pool, free, max_moves, pinned=()):
    most = len(table[0]) if table else 1
    bad, used = set(), set(pinned)
    n_pages = [held(c, ratio, most) for c in cached]
    for r, t in enumerate(table):
        if n_pages[r] < 0:
            bad.add(8)
        for page in t[:max(0, n_pages[r])]:
            if 0 <= page < pool:
                used.add(page)
            else:
                bad.add(5)
    n = len(used)
    movers = [p for p in sorted(used) if p >= n and p not in pinned][:max_moves]
    holes = [p for p in range(n) if p not in used][:len(movers)]
    to = dict(zip(movers, holes))
    after = {to.get(p, p) for p in used}
    out = [[to.get(p, p) for p in t[:max(0, n_pages[r])]] + [-1] * (most - max(0, n_pages[r])) for r, t in enumerate(table)]
    spare = [p for p in range(pool) if p not in after]
    if len(spare) > len(free):
        bad.add(11)
        spare = spare[len(spare) - len(free):]
    free = list(free)
    head = len(free) - len(spare)
    free[head:] = spare
    pad = [-1] * (max_moves - len(movers))
    return dict(table=out, src=movers + pad, dst=holes + pad, counts=[len(movers), n, max(after) + 1 if after else 0, head], free=free, bad=bad)


def words(pinned, pool):
    w = [0] * ((pool + 31) // 32)
    for p in pinned:
        w[p >> 5] |= 1 << (p & 31)
    return [v - (1 << 32) if v >> 31 else v for v in w]
