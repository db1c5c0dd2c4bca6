"""The expanded and the absorbed form of one attention, each against the same float64 result.

Every head's expansion picks 128 of the 512 latent dims as key and 128 as value, so the expanded
keys, values and absorbed queries hold the latents' own bf16 numbers and both forms compute
the same attention without a rounding between them."""
import pytest
import torch

from tests import latent_ref as ref

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("n,heads", [(1, 2), (150, 4), (700, 3), (330, 16)])
def test_both_forms(n, heads):
    from sparse_attention_fp4_gb300 import fp4idx
    g = torch.Generator(device="cuda").manual_seed(n)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    latent, rope, q, scale = mk(n, 512), mk(n, 64), mk(n, heads, 192), 192 ** -0.5
    pick_k = torch.stack([torch.randperm(512, generator=g, device="cuda")[:128] for _ in range(heads)])
    pick_v = torch.stack([torch.randperm(512, generator=g, device="cuda")[:128] for _ in range(heads)])
    kv = torch.cat([latent[:, pick_k], latent[:, pick_v]], 2).contiguous()
    out = torch.empty((n, heads, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((n, heads), dtype=torch.float32, device="cuda")
    status = i32([0])
    fp4idx.latent_prefill(q, kv, rope, i32([0, n]), i32([0, n]), n, n, scale, out, lse=lse, status=status)

    absorbed = torch.zeros((n, heads, 576), dtype=torch.bfloat16, device="cuda")
    absorbed.scatter_(2, pick_k.expand(n, heads, 128), q[:, :, :128].contiguous())
    absorbed[:, :, 512:] = q[:, :, 128:]
    pages = -(-n // 64)
    cache = fp4idx.alloc_latent_cache(pages, 576)
    rows = torch.cat([latent, rope], 1)
    cache.view(-1, 576)[:n] = rows
    table = i32([list(range(pages))])
    whole = torch.empty((n, heads, 512), dtype=torch.bfloat16, device="cuda")
    lse2 = torch.empty((n, heads), dtype=torch.float32, device="cuda")
    ws = torch.empty(fp4idx.latent_attn_workspace_bytes(n, heads), dtype=torch.uint8, device="cuda")
    fp4idx.latent_attn(absorbed, cache, table, i32([0] * n), i32(list(range(1, n + 1))), n, scale, ws, whole, lse=lse2, status=status)
    assert fp4idx.read_status(status) == 0

    keys = rows.double()
    for i in sorted(set(list(range(0, n, 1 + n // 60)) + [n - 1])):
        ref.check(whole[i], lse2[i], ref.attend(absorbed[i].double(), keys[:i + 1], keys[:i + 1, :512], scale), "absorbed, row %d" % i)
        for h in range(heads):
            key = torch.cat([latent[:i + 1, pick_k[h]], rope[:i + 1]], 1).double()
            want = ref.attend(q[i, h].double()[None], key, latent[:i + 1, pick_v[h]].double(), scale)
            ref.check(out[i, h][None], lse[i, h][None], want, "expanded, row %d, head %d" % (i, h))
            # ... and each within its bound of the same number: the absorbed output in the head's value dims
            ref.check(whole[i, h, pick_v[h]][None], None, (want[0], want[1], 2 * want[2], want[3]), "row %d, head %d" % (i, h))
