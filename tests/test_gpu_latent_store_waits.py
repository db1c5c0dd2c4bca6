"""The latent store's bounded wait: with copies that never come it ends with a status and
writes nothing, and the next call is right."""
import pytest
import torch

from tests import latent_ref as ref
from tests.test_gpu_plan_store import cos_sin_table, i32, store_inputs

pytestmark = pytest.mark.gpu

TIMEOUT = 6
LIMIT_NS = 5_000_000


@pytest.mark.parametrize("n,width", [(1, 576), (5, 512), (600, 512), (20000, 576)])
def test_store_wait_runs_out_then_recovers(n, width):
    from sparse_attention_fp4_gb300 import fp4idx
    pages = -(-n // 64) + 1
    kv, w, pos, slots = store_inputs(n, width, pages, n)
    cs = cos_sin_table(5000)
    cache = torch.full((pages, 64, width), 7.5, dtype=torch.bfloat16, device="cuda")
    status = i32([0])

    def call():
        fp4idx.store_latent(kv, pos, slots, w, 1e-6, cs, cache, status=status)
        return fp4idx.read_status(status)

    try:
        fp4idx.test_pipeline_waits(True, LIMIT_NS)
        assert call() == TIMEOUT
    finally:
        fp4idx.test_pipeline_waits(False, 0)
    assert bool((cache == 7.5).all())
    status.zero_()
    assert call() == 0
    want, tol = ref.store(kv, pos, w, 1e-6, cs)
    got = cache.view(-1, width)[slots.long()].double()
    assert bool(((got - want).abs() <= tol).all())
