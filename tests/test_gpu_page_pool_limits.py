"""The page pool's operators at the ends of their documented ranges."""
import pytest
import torch

pytestmark = pytest.mark.gpu
GUARD = 8192


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def all_are(v, value):
    return all(bool((part == value).all()) for part in v.split(1 << 28))


@pytest.mark.parametrize("moves", [2 ** 31 - 1, 2 ** 31 - 1024, 2 ** 31 - 1025])
def test_compact_with_the_longest_move_lists(moves):
    """Every place behind the last move is -1, and nothing before or behind the lists is written."""
    from sparse_attention_fp4_gb300 import fp4idx
    src, dst = (torch.full((GUARD + moves + GUARD,), -77, dtype=torch.int32, device="cuda") for _ in range(2))
    table, cached, pool = i32([[90, 3], [90, 70]]), i32([128, 65]), 100
    out, counts, free, status = torch.empty_like(table), i32([0] * 4), i32([-3] * pool), i32([0])
    ws = torch.empty(fp4idx.compact_pages_workspace_bytes(pool), dtype=torch.uint8, device="cuda")
    fp4idx.compact_pages(table, cached, 1, pool, ws, free, out, src[GUARD:GUARD + moves], dst[GUARD:GUARD + moves], counts, status=status)
    assert fp4idx.read_status(status) == 0
    assert counts.tolist() == [3, 3, 3, 3] and out.tolist() == [[2, 0], [2, 1]] and free.tolist() == [-3] * 3 + list(range(3, 100))
    for v, want in ((src, [3, 70, 90]), (dst, [0, 1, 2])):
        assert v[GUARD:GUARD + 3].tolist() == want
        assert all_are(v[GUARD + 3:GUARD + moves], -1)
        assert all_are(v[:GUARD], -77) and all_are(v[GUARD + moves:], -77)
