"""Values that f16 does not hold, in kv_tree_attn: what is hidden stays
hidden, what is seen shows.
Tolerances are those of test_gpu_multi_attn.py."""
import numpy as np
import pytest

from tests import test_gpu_multi_attn as M

pytestmark = pytest.mark.gpu


# 12, 28, 40 and 80 rows a KV head are tiles of 16, 32, 64 (twice over) and 128 rows
@pytest.mark.parametrize("T", [6, 14, 20, 40])
@pytest.mark.parametrize("D,kb,vb,ctx,window", [(64, 4, 4, 70, 0), (128, 2, 2, 70, 33), (64, 8, 3, 2500, 64), (128, 4, 8, 2500, 0)])
@pytest.mark.parametrize("huge", [1e5, -3e38])
def test_bf16_values_above_the_range_of_f16(huge, D, kb, vb, ctx, window, T):
    """A finite bf16 draft value of 2^16 and more (times 2 and 8 with 2- and
    3-bit V codes, which are held in halves and eighths) is an infinity where
    it is seen, and nothing where it is not."""
    import torch
    gc, oc, k, v, f = M.make_caches(1, 2, 2, D, ctx, "bf16", kb, vb, window=window)
    M.fill(gc, oc, k, v, "bf16")
    q, kd, vd = M.drafts(1, 2, 2, D, T, f, "bf16", 2)
    see = M.tree(1, T, 1)
    see[0, T - 2] = see[0, T - 1] = False          # padding: nobody sees the last two
    see[0, :, T - 2:] = False
    clean = M.reference(oc, q, "bf16", see, kd, vd)
    plain, _ = M.run_tree(gc, q, kd, vd, see, "bf16")
    vd[:, :, T - 2:] = M._act(np.full_like(vd[:, :, T - 2:], huge), "bf16")
    out, lse = M.run_tree(gc, q, kd, vd, see, "bf16")
    M.compare(out, lse, clean)
    assert torch.equal(out, plain)
    vd[:, :, 1, 5] = M._act(np.full_like(vd[:, :, 1, 5], huge), "bf16")  # a value that some see
    out2, lse2 = M.run_tree(gc, q, kd, vd, see, "bf16")
    hit = see[0, :, 1]
    assert hit.any() and not hit.all()
    assert torch.equal(lse2, lse)
    o1, o2 = out.float().cpu().numpy(), out2.float().cpu().numpy()
    assert np.array_equal(o1[:, :, ~hit], o2[:, :, ~hit])
    rest = np.ones(D, bool)
    rest[5] = False
    assert np.array_equal(o1[..., rest], o2[..., rest])
    if abs(huge) < {2: 2.0 ** 17, 3: 2.0 ** 19}.get(vb, 2.0 ** 16):
        M.compare(out2, lse2, M.reference(oc, q, "bf16", see, kd, vd))
    else:
        assert (o2[:, :, hit, 5] == np.copysign(np.inf, huge)).all()
