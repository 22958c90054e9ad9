"""The failure path of the waits of kv_tree_attn and kv_cross_attn, made to run
out on purpose: on barriers that nothing arrives at and no copy completes on,
with a short budget. No fault and no hang is involved."""
import pytest

from tests import test_gpu_multi_attn as M

pytestmark = pytest.mark.gpu


def test_bounded_waits_give_up_and_the_cache_stays_usable():
    import torch
    from bit_kv_cache_append_gb300.binding import KV_ERR_TIMEOUT, KVError
    gc, oc, k, v, f = M.make_caches(1, 2, 2, 64, 200, "f16", 4, 4)
    M.fill(gc, oc, k, v, "f16")
    args = {T: M.drafts(1, 2, 2, 64, T, f, "f16", 2) + (M.tree(1, T, 1),) for T in (6, 40)}  # both kernels
    before = {T: M.run_tree(gc, *a, "f16") for T, a in args.items()}
    budget = 2_000_000  # SM clock cycles, about a millisecond
    res = gc.test_attn_bounded_wait(budget)
    assert res[:4] == [0, 0, 0, 0], res
    own, through_flag, own_short, through_flag_short = res[4:]
    # the first warp looks at the clock after every round of polls
    assert budget <= own < 4 * budget, res
    # 8 rounds; the kernels' bound of 8192 has to be about a second, at 0.5 to 2.1 GHz
    assert 2 ** 29 <= own_short * (8192 // 8) <= 2 ** 32, res
    # the other two, whose bounds are 2^31 cycles and 8192 rounds, left soon after the flag was raised
    assert budget // 2 < through_flag < 4 * budget, res
    assert own_short // 2 < through_flag_short < 4 * own_short, res
    with pytest.raises(KVError) as e:
        gc.check_device_error()
    assert e.value.status == KV_ERR_TIMEOUT
    gc.check_device_error()                     # reading the flag cleared it
    for T, a in args.items():
        for x, y in zip(before[T], M.run_tree(gc, *a, "f16")):
            assert torch.equal(x, y)


def test_budgets_out_of_range():
    from bit_kv_cache_append_gb300.binding import KV_ERR_INVALID_ARG, KVError
    gc = M.make_caches(1, 1, 1, 64, 32, "f16", 4, 4)[0]
    for bad in (0, 999, (1 << 31) + 1):
        with pytest.raises(KVError) as e:
            gc.test_attn_bounded_wait(bad)
        assert e.value.status == KV_ERR_INVALID_ARG
