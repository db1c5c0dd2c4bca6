"""Beam selection: equal totals of a row whose tokens several CTAs read, and whose end is no vector boundary."""
import math

import numpy as np
import pytest
import torch

from tests import beam_ref as ref
from tests.test_gpu_beam_select import BF16, FP16, FP32, run

pytestmark = pytest.mark.gpu
INF = math.inf


def tied(seed, R, V, kind, pad=0, offset=0):
    """Whole numbers below zero, and equal largest values: at the row's ends, one by one, and at places in between."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    stride = V + pad
    buf = torch.randint(-9, 0, (offset + R * stride,), generator=g, device="cuda").to(kind)
    x = buf.as_strided((R, V), (stride, 1), offset)
    between = (torch.rand((R, 6), generator=g, device="cuda") * V).long()
    ends = V - 1 - torch.randint(0, 7, (R, 3), generator=g, device="cuda")
    begins = torch.randint(0, 7, (R, 1), generator=g, device="cuda")
    at = torch.cat([between, ends, begins], 1)
    x.scatter_(1, at, torch.full_like(at, 10).to(kind))
    return x


def order(row):
    """A row's tokens, the largest first, of equal ones the lowest."""
    v = row.float().cpu().numpy()
    return np.lexsort((np.arange(v.size), -v))


@pytest.mark.parametrize("kind", [BF16, FP16, FP32])
@pytest.mark.parametrize("beams", [1, 4, 9])  # (a group of nine takes two launches)
@pytest.mark.parametrize("V,pad", [(50257, 0), (50256, 1), (4103, 0), (131075, 2), (32001, 0)])
def test_ties_between_a_rows_ends_and_its_middle(kind, beams, V, pad):
    """Rows at every offset from a vector boundary; lists that end among the equal tokens, and behind them."""
    for groups, offset in ((1, 0), (1, 3), (2, 0)):
        R = groups * beams
        x = tied(V + R + offset, R, V, kind, pad, offset)
        scores = [-3.0 * (r % beams) for r in range(R)]
        s32 = np.array(scores, dtype=np.float32)
        for k in (1, 3, 24):
            got, status = run(x, scores, beams, k)
            assert status == 0
            ref.check_select(got, x.float().cpu().numpy(), s32, beams, k)
            for g in range(groups):  # a row's own tokens, in order
                for r in set(got[1][g].tolist()):
                    mine = got[2][g][got[1][g] == r]
                    assert mine.tolist() == order(x[r])[:mine.size].tolist(), (k, g, r)


@pytest.mark.parametrize("kind", [BF16, FP32])
def test_the_last_token_equals_one_before_it(kind):
    """The end token of a vocabulary that ends with it, as good as one token before: the latter is chosen."""
    V = 50257
    for first in (0, 1, 7, 12000, 25200, 30000, 50000, 50255):
        x = torch.zeros((1, V), dtype=kind, device="cuda")
        x[0, first] = x[0, V - 1] = 10
        got, status = run(x, [-1.0], 1, 2, end=V - 1)
        assert status == 0 and got[2][0].tolist() == [first, V - 1] and got[3][0].tolist() == [0, 1]
        got, _ = run(x, [-1.0], 1, 1, end=V - 1)
        assert got[2][0].tolist() == [first]


@pytest.mark.parametrize("kind", [BF16, FP16, FP32])
def test_a_tied_row_is_the_same_in_any_batch(kind):
    one = tied(5, 1, 50257, kind)
    want = order(one[0])[:8].tolist()
    for R in (1, 2, 4, 16, 60, 256, 300, 400):
        x = one.repeat(R, 1)
        for beams in (1, 4):
            if R % beams == 0:
                got, _ = run(x, [0.0 if r % beams == 0 else -40.0 for r in range(R)], beams, 8)
                assert (got[2] == want).all(), (R, beams)


@pytest.mark.parametrize("kind,V", [(BF16, 4104), (FP16, 4104), (FP32, 4100), (FP32, 2052), (BF16, 8200)])
@pytest.mark.parametrize("beams", [1, 3, 9])
def test_a_last_part_without_a_vector(kind, V, beams):
    """Rows off a vector boundary have a vector less, and what is left of their last part are single tokens."""
    R = 9 * (8 if beams == 1 else 1)
    x = tied(V + beams, R, V, kind, pad=1)
    for k in (1, 5, 20):
        got, status = run(x, [-3.0 * (r % beams) for r in range(R)], beams, k)
        assert status == 0
        for g in range(R // beams):
            for r in set(got[1][g].tolist()):
                mine = got[2][g][got[1][g] == r]
                assert mine.tolist() == order(x[r])[:mine.size].tolist(), (k, g, r)


@pytest.mark.parametrize("kind", [BF16, FP16, FP32])
@pytest.mark.parametrize("V", [4100, 4104, 50257])
@pytest.mark.parametrize("beams", [1, 9])
def test_rows_of_which_only_the_ends_are_left(kind, V, beams):
    """Nothing but a row's first or last token is allowed; and what is no number there takes the row away."""
    R = 9
    stride = V + 1
    x = torch.full((R * stride,), -INF, dtype=kind, device="cuda").as_strided((R, V), (stride, 1))
    for r in range(R):
        x[r, V - 1 if r % 3 else 0] = -2.0
    scores = [-1.0 - r for r in range(R)]
    want = [V - 1 if r % 3 else 0 for r in range(R)]
    got, status = run(x, scores, beams, 2)
    assert status == 0
    if beams == 1:
        assert got[2][:, 0].tolist() == want and got[0][:, 0].tolist() == scores and (got[1][:, 1] == -1).all()
    else:
        assert got[1][0].tolist() == [0, 1] and got[2][0].tolist() == want[:2] and got[0][0].tolist() == scores[:2]
    for bad in (float("nan"), INF):
        for at in (0, V - 1):
            y = x.clone()
            y[4, at] = bad
            got, status = run(y, scores, 1, 1)
            assert status == 12 and got[1][:, 0].tolist() == [r if r != 4 else -1 for r in range(R)]
