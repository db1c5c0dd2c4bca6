"""Beam selection: how far the logarithm of a row's sum may be off, as the header states it.

In units of 2^-24, of the sum of exponentials and so of its logarithm: an exponential 4 (2^-22), the sums within a tile 10,
an edge of the row 6; for each of a thread's tiles (512 16-byte vectors of a row at the least, 64 tiles at the most) one
addition, and a factor (5: exponential and product) where its largest rises; the factors to the largest of the CTA and of
the row, 5 each.  The arguments of an element's exponentials add up to its distance below the row's largest; two
roundings and that of log2 e, 2.3 of the distance, whose mean over the row's probabilities is no more than their entropy,
and so than ln vocab.  A total has one rounding to fp32, and some 36 bits before that."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
FP32, BF16, FP16 = torch.float32, torch.bfloat16, torch.float16
INF = math.inf


def bound(V, kind):
    tiles = min(64, -(-V * (4 if kind == FP32 else 2) // 16 // 512))
    return (30 + 6 * tiles + 2.3 * math.log(V)) * 2.0 ** -24


def best(x, scores):
    """The total of each row's best token."""
    from sparse_attention_fp4_gb300 import fp4idx
    R, V = x.shape
    out = [torch.empty(R, dtype=d, device="cuda") for d in (FP32, torch.int32, torch.int32)]
    ws = torch.empty(fp4idx.beam_select_workspace_bytes(R, V, 1), dtype=torch.uint8, device="cuda")
    fp4idx.beam_select(x, scores, 1, 1, ws, *out)
    assert bool((out[1] == torch.arange(R, device="cuda")).all())
    return out[0].double()


def check(x, tol):
    """Scores that bring the best total next to zero, where its own rounding is small."""
    xd = x.double()
    top = xd.amax(1)
    rest = torch.log(torch.exp(xd - top[:, None]).sum(1))
    scores = rest.float()
    want = scores.double() - rest
    off = (best(x, scores) - want).abs()
    assert bool((off <= tol + (want.abs() + rest) * 2.0 ** -36 + want.abs() * 2.0 ** -24).all()), float(off.max())


def test_logarithm_of_whole_sums():
    """n equal logits: the sum is n exactly, and what is left is the logarithm's own error.  Its series without the first
    term is 0.0028 at the most, with 7 roundings, and doubled (2.3e-9); four sums of numbers below 2^-7 round by 2^-32 each."""
    n = torch.cat([torch.arange(1, 3000), torch.randint(3000, 1 << 16, (1000,), generator=torch.Generator().manual_seed(1))]).cuda()
    x = torch.where(torch.arange(1 << 16, device="cuda")[None] < n[:, None], 0.0, -INF)
    check(x.to(BF16), 3.3e-9)
    n = torch.tensor([1 << 19, (1 << 19) - 1, 392843, 400000, 65537], device="cuda")
    x = torch.where(torch.arange(1 << 19, device="cuda")[None] < n[:, None], 7.5, -INF)
    check(x.to(FP16), 3.3e-9)
    check(x, 3.3e-9)


@pytest.mark.parametrize("V", [700, 4096, 50257, 1 << 19])
@pytest.mark.parametrize("R", [1, 8, 400])
def test_many_equal_logits_below_the_largest(V, R):
    """All exponentials round alike, and carry much of the sum."""
    g = torch.Generator(device="cuda").manual_seed(V + R)
    below = 4 + 10 * torch.rand((R, 1), generator=g, device="cuda")
    x = (-below).repeat(1, V)
    x[:, V // 3] = 0.0
    check(x, bound(V, FP32))
    x += 100 * torch.randn((R, 1), generator=g, device="cuda")
    for kind in (FP32, BF16, FP16):
        check(x.to(kind), bound(V, kind))


@pytest.mark.parametrize("kind", [FP32, BF16, FP16])
@pytest.mark.parametrize("V", [3001, 131072])
def test_rows_whose_largest_rises(kind, V):
    for span in (0.5, 3, 20, 80):
        x = torch.linspace(-span, 0, V, device="cuda")
        check(torch.stack([x, x.flip(0), x.roll(V // 2)]).to(kind), bound(V, kind))
        check(x.repeat(310, 1).to(kind), bound(V, kind))


@pytest.mark.parametrize("kind", [FP32, BF16, FP16])
def test_rows_as_models_give_them(kind):
    g = torch.Generator(device="cuda").manual_seed(3)
    for R, V in ((1, 32000), (64, 50257), (300, 20000)):
        x = 3 * torch.randn((R, V), generator=g, device="cuda")
        check(x.to(kind), bound(V, kind))
        check(torch.log_softmax(x, 1).to(kind), bound(V, kind))  # (sums next to one: an error relative to their logarithm would be none)


def test_totals_below_the_range_of_fp32():
    """Candidates all the same, in order; their totals are written as -inf."""
    from sparse_attention_fp4_gb300 import fp4idx
    most = torch.finfo(FP32).max
    x = torch.tensor([[-most, most, 0.0], [-INF, -INF, -INF]], device="cuda")
    out = [torch.empty(4, dtype=d, device="cuda") for d in (FP32, torch.int32, torch.int32)]
    ws = torch.empty(fp4idx.beam_select_workspace_bytes(2, 3, 4), dtype=torch.uint8, device="cuda")
    fp4idx.beam_select(x, torch.tensor([-most, 0.0], device="cuda"), 2, 4, ws, *out)
    assert out[0].tolist() == [-most, -INF, -INF, -INF] and out[1].tolist() == [0, 0, 0, -1] and out[2].tolist() == [1, 2, 0, -1]
