"""Values that f16 does not hold and queries and keys that are not numbers, in
kv_tree_attn and kv_cross_attn: what is hidden stays hidden, what is seen
shows. Tolerances are those of test_gpu_multi_attn.py."""
import numpy as np
import pytest

from tests import test_gpu_multi_attn as M
from tests.parity import torch_act

pytestmark = pytest.mark.gpu


def rows_that_count(got, lse, ref, count):
    """compare() over the rows of `count` [B, T]; the others are taken out on both sides."""
    import torch
    keep = torch.from_numpy(np.broadcast_to(count[:, None], lse.shape).copy()).cuda()
    want, l64 = (torch.from_numpy(x).cuda() for x in ref[:2])
    got = torch.where(keep[..., None], got.double(), want)
    M.compare(got, torch.where(keep, lse.double(), l64), ref)


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


# 2 x 70 tokens: a unit to a CTA, no merge; 2500: units cut by many shares, their partials shared by a block's warps;
# 40 x 70: several units a CTA, some cut
@pytest.mark.parametrize("T", [5, 14, 20, 40])
@pytest.mark.parametrize("B,H,D,ctx", [(2, 2, 64, 70), (1, 1, 128, 2500), (1, 2, 64, 6007), (40, 4, 64, 70)])
def test_a_query_that_is_not_a_number(B, H, D, ctx, T):
    """It gives NaN in its own row, sums and output, however the columns were shared out."""
    gc, oc, k, v, f = M.make_caches(B, H, 2, D, ctx, "f16", 4, 4)
    M.fill(gc, oc, k, v, "f16")
    q, kd, vd = M.drafts(B, H, 2, D, T, f, "f16", 2)
    see = M.tree(B, T, 1)
    ref = M.reference(oc, q, "f16", see, kd, vd)
    q[:, :, T - 2, 3] = np.nan
    out, lse = M.run_tree(gc, q, kd, vd, see, "f16")
    assert bool(out[:, :, T - 2].isnan().all()) and bool(lse[:, :, T - 2].isnan().all())
    count = np.ones((B, T), bool)
    count[:, T - 2] = False
    rows_that_count(out, lse, ref, count)


@pytest.mark.parametrize("T", [5, 14, 20, 40])
@pytest.mark.parametrize("B,H,D,ctx", [(2, 2, 64, 70), (1, 1, 128, 2500), (40, 4, 64, 70)])
def test_a_drafted_key_that_is_not_a_number(B, H, D, ctx, T):
    """It gives NaN in the rows that see it, also where it is outweighed by far: the scores of the cached keys are
    some 2^8 above those of the drafts."""
    gc, oc, k, v, f = M.make_caches(B, H, 2, D, ctx, "f16", 4, 4)
    q, kd, vd = M.drafts(B, H, 2, D, T, f, "f16", 2)
    q, kd = np.abs(q), -np.abs(kd)
    k = np.abs(k)
    k[:, :, : ctx // 32 * 32] = M._act(k[:, :, : ctx // 32 * 32] * 8, "f16")
    M.fill(gc, oc, k, v, "f16")
    see = M.tree(B, T, 1)
    ref = M.reference(oc, q, "f16", see, kd, vd)
    kd[:, :, 1, 3] = np.nan
    out, lse = M.run_tree(gc, q, kd, vd, see, "f16")
    hit = see[:, :, 1]
    assert hit.any() and not hit.all()
    for b in range(B):
        assert bool(out[b][:, hit[b]].isnan().all()) and bool(lse[b][:, hit[b]].isnan().all())
    rows_that_count(out, lse, ref, ~hit)


def test_cross_queries_that_are_not_numbers():
    """One query a sequence, ragged: NaN where there is a position to see, zeros where there is none."""
    import torch
    gc, oc, k, v, f = M.make_caches(4, 2, 2, 64, 3000, "f16", 4, 4)
    M.fill(gc, oc, k, v, "f16")
    q = M.drafts(4, 2, 2, 64, 1, f, "f16", 2)[0]
    lens = [3000, 0, 7, 1500]
    ref = M.reference(oc, q, "f16", lens=lens)
    q[0], q[1], q[2, 1] = np.nan, np.nan, np.nan
    lse = torch.full(q.shape[:3], float("nan"), dtype=torch.float32, device="cuda")
    out = gc.cross_attn(0, torch_act(q, "f16"), torch.tensor(lens, dtype=torch.int32, device="cuda"), lse=lse)
    torch.cuda.synchronize()
    gc.check_device_error()
    assert bool(out[0].isnan().all()) and bool(lse[0].isnan().all())
    assert bool((out[1] == 0).all()) and bool(torch.isneginf(lse[1]).all())
    assert bool(out[2, 1].isnan().all()) and bool(lse[2, 1].isnan().all())
    for b, heads in ((2, [0, 2, 3]), (3, [0, 1, 2, 3])):
        M.compare(out[b:b + 1, heads], lse[b:b + 1, heads], tuple(r[b:b + 1, heads] for r in ref[:4]) + (ref[4],))
