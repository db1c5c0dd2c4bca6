"""Plain 64-bit references of the latent-attention entry points, and the bounds their
results are held to (derived from the roundings the kernels make)."""
import math

import torch

BF16 = torch.finfo(torch.bfloat16).eps / 2   # one rounding to bf16, relative
# One fp32 addition of a tensor-core or SIMT sum: 2^-24 if rounded; the tensor cores may
# truncate and align to fewer bits, so four times that is counted.
F32 = 4 * torch.finfo(torch.float32).eps / 2


def attend(q, keys, values, scale):
    """q [H, D] and the row's tokens [n, D], [n, V] (float64): out [H, V], lse [H] and the bounds of both.

    Scores: D products are summed in fp32, each addition off by F32 of a partial sum, so a
    score is off by ds <= (D + 2) F32 scale sum|q k|, which changes a weight by ds and the
    normaliser by ds (relative).  The exponential adds 2^-21 (two ulps and its argument's
    rounding, |s - max| 2^-24 <= 88 2^-24), the rounding of a weight to bf16 BF16, the n
    additions of either sum n F32; the output's own rounding BF16."""
    n, D = keys.shape
    if n == 0:
        z = torch.zeros((q.shape[0], values.shape[1]), dtype=torch.float64, device=q.device)
        lse = torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device)
        return z, lse, z.clone(), torch.zeros_like(lse)
    s = scale * (q @ keys.T)
    p = torch.softmax(s, 1)
    out, lse = p @ values, torch.logsumexp(s, 1)
    ds = ((D + 2) * F32 * abs(scale) * (q.abs() @ keys.abs().T)).amax(1)
    rel = BF16 + 2 * ds + 2 * (n + 8) * F32 + 2 * (88 * 2.0 ** -24 + 2.0 ** -21)
    tol = 1.01 * (BF16 * out.abs() + rel[:, None] * (p @ values.abs())) + 1e-30
    tol_lse = ds + (n + 8) * F32 + 88 * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -22 * lse.abs()
    return out, lse, tol, tol_lse


def check(got, got_lse, want, what):
    out, lse, tol, tol_lse = want
    err = (got.double() - out).abs()
    assert bool((err <= tol).all()), "%s: out off by %.3g where %.3g is allowed" % (
        what, float(err[~(err <= tol)].max()), float(tol[~(err <= tol)].max()))
    if got_lse is not None:
        empty = lse == -math.inf
        assert bool((got_lse[empty] == -math.inf).all()), what
        e = (got_lse.double() - lse).abs()[~empty]
        assert bool((e <= tol_lse[~empty]).all()), "%s: lse off by %.3g" % (what, float(e.max()))


def tokens(cache, table_row, positions):
    """Latent rows of a sequence's token positions, float64 [n, width]."""
    pos = torch.as_tensor(positions, dtype=torch.long, device=cache.device)
    pages = table_row.long()[pos // 64]
    return cache[pages, pos % 64].double()


def store(kv, positions, norm_w, eps, cos_sin):
    """The stored row in float64, before its rounding, and the fp32 chain's bound."""
    x = kv.double()
    y = x.clone()
    r = 1 / torch.sqrt((x[:, :512] ** 2).mean(1, keepdim=True) + eps)
    y[:, :512] = x[:, :512] * r * norm_w.double()
    a = y.abs()
    t = cos_sin.double()[positions.long()]
    c, s = t[:, :32], t[:, 32:]
    lo, hi = y[:, -64:-32].clone(), y[:, -32:].clone()
    y[:, -64:-32], y[:, -32:] = lo * c - hi * s, hi * c + lo * s
    a[:, -64:-32], a[:, -32:] = a[:, -64:-32] * c.abs() + a[:, -32:] * s.abs(), a[:, -32:] * c.abs() + a[:, -64:-32] * s.abs()
    # the sum of 512 squares (half of its relative error in the root), root, divide, two
    # products, and two products and a sum of the rotation: well under 600 fp32 roundings
    return y, BF16 * y.abs() + 600 * 2.0 ** -24 * a


def plan(cached, new, ratio, free, head, table, max_rows, max_stores):
    """fp4idx_plan_step in Python integers; table: list of lists, changed in place."""
    q_pos, seq, ctx, s_pos, slots, cu, cu_ctx = [], [], [], [], [], [0], [0]
    taken, planned, full, bad = 0, 0, False, False
    width = len(table[0]) if table else 0
    for b, (c, n) in enumerate(zip(cached, new)):
        wrong = c < 0 or n < 0 or c + n > 2 ** 31 - 1 or (c + n) // ratio > 64 * width
        if wrong and not full:
            bad = True
            planned += 1
        elif not full:
            e0, e1 = c // ratio, (c + n) // ratio
            p0, p1 = -(-e0 // 64), -(-e1 // 64)
            if len(q_pos) + n > max_rows or len(s_pos) + e1 - e0 > max_stores or taken + p1 - p0 > len(free) - head:
                full = True
            else:
                planned += 1
                for j in range(p0, p1):
                    table[b][j] = free[head + taken]
                    taken += 1
                for i in range(n):
                    q_pos.append(c + i)
                    seq.append(b)
                    ctx.append((c + i + 1) // ratio)
                for e in range(e0, e1):
                    s_pos.append(e)
                    slots.append(table[b][e // 64] * 64 + e % 64 if table[b][e // 64] >= 0 else -1)
                cu_ctx.append(cu_ctx[-1] + e1)
                cu.append(len(q_pos))
                continue
        cu_ctx.append(cu_ctx[-1])
        cu.append(len(q_pos))
    counts = [len(q_pos), len(s_pos), taken, planned]
    pad = max_rows - len(q_pos)
    pads = max_stores - len(s_pos)
    return dict(q_positions=q_pos + [0] * pad, row_seq=seq + [0] * pad, context_lens=ctx + [0] * pad,
                store_positions=s_pos + [0] * pads, store_slots=slots + [-1] * pads, cu_rows=cu, cu_context=cu_ctx,
                counts=counts, table=table, full=full, bad=bad)
