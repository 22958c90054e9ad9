"""The workspace of kv_tree_attn and kv_cross_attn: no more than two partials a
CTA, nothing written behind it, nothing read that the call did not write."""
import numpy as np
import pytest

from tests import test_gpu_multi_attn as M
from tests.parity import torch_act

pytestmark = pytest.mark.gpu


def partial_bytes(rows, D):
    tile = 16 if rows <= 16 else 32 if rows <= 32 else 128  # (64 rows are held twice)
    return tile * (D + 2) * 4


@pytest.mark.parametrize("B,H,gqa,D", [(1, 1, 1, 64), (1, 8, 4, 128), (64, 8, 4, 128), (300, 2, 1, 64)])
def test_two_partials_a_cta(B, H, gqa, D):
    import torch
    from bit_kv_cache_append_gb300.binding import KVCache
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    gc = KVCache(n_layers=1, batch=B, n_kv_heads=H, n_q_heads=H * gqa, head_dim=D, max_tokens=64)
    for n in (1, 4, 8, 9, 16, 33, 61, 256, 1000, 4097):
        tiles = -(-gqa * n // 128) if gqa * n > 64 else 1
        slots = sms + min(B * H * tiles, sms)
        assert gc.workspace_bytes(n) <= slots * partial_bytes(gqa * n, D) + 512, n


# few units cut by many shares, more units than CTAs, ragged ones, and a CTA for each
@pytest.mark.parametrize("T", [3, 14, 20, 70, 200])
@pytest.mark.parametrize("B,H,gqa,D,ctx,ragged", [(1, 1, 2, 64, 3000, False), (5, 4, 2, 128, 700, True), (90, 2, 2, 64, 150, False),
                                                  (90, 2, 2, 64, 150, True), (30, 4, 1, 64, 100, False)])
def test_nothing_behind_the_workspace(B, H, gqa, D, ctx, ragged, T):
    import torch
    gc, oc, k, v, f = M.make_caches(B, H, gqa, D, ctx, "f16", 4, 4)
    M.fill(gc, oc, k, v, "f16")
    q = torch_act(M.drafts(B, H, gqa, D, T, f, "f16", 3)[0], "f16")
    lens = None
    if ragged:
        lens = torch.from_numpy(np.random.default_rng(T).integers(0, ctx + 1, B).astype(np.int32)).cuda()
    want = gc.cross_attn(0, q, lens)
    need = gc.workspace_bytes(T)
    room = torch.full((need + (32 << 20),), 255, dtype=torch.uint8, device="cuda")  # (NaN as floats)
    got = gc.cross_attn(0, q, lens, workspace=room[:need])
    torch.cuda.synchronize()
    gc.check_device_error()
    assert bool((room[need:] == 255).all())
    assert bool(torch.isfinite(got).all()) and torch.equal(got, want)
