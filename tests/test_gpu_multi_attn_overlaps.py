"""Outputs and workspaces of kv_tree_attn and kv_cross_attn that lie on
something else are refused before anything is launched; ones that only touch it
are not."""
import pytest

from tests import test_gpu_multi_attn as M

pytestmark = pytest.mark.gpu

B, H, GQA, D, T = 4, 2, 2, 64, 8


@pytest.fixture(scope="module")
def setup():
    import torch
    gc, oc, k, v, f = M.make_caches(B, H, GQA, D, 70, "f16", 4, 4)
    M.fill(gc, oc, k, v, "f16")
    sizes = {"q": B * H * GQA * T * D * 2, "k": B * H * T * D * 2, "v": B * H * T * D * 2, "mask": B * T * 8,
             "lengths": B * 4, "out": B * H * GQA * T * D * 2, "lse": B * H * GQA * T * 4, "workspace": gc.workspace_bytes(T)}
    step = max(sizes.values()) + 1024 & ~255
    room = torch.zeros(step * (2 * len(sizes) + 1), dtype=torch.uint8, device="cuda")
    return gc, sizes, room, {n: step * (2 * i + 1) for i, n in enumerate(sizes)}  # (the allocator aligns to 512 bytes)


def call(setup, op, **moved):
    """The call with every tensor a view of one room, at its own place or where `moved` says."""
    import torch
    gc, sizes, room, place = setup
    place = {**place, **moved}

    def view(name, dtype, *shape):
        return room[place[name]:place[name] + sizes[name]].view(dtype).view(shape)

    q = view("q", torch.float16, B, H * GQA, T, D)
    more = dict(out=view("out", torch.float16, B, H * GQA, T, D), lse=view("lse", torch.float32, B, H * GQA, T),
                workspace=view("workspace", torch.uint8, sizes["workspace"]))
    if op == "tree":
        k, v = (view(n, torch.float16, B, H, T, D) for n in "kv")
        mask = view("mask", torch.int64, B, T, 1)
        return gc.tree_attn(0, q, k, v, mask, **more)
    return gc.cross_attn(0, q, view("lengths", torch.int32, B), **more)


PAIRS = [(op, w, r) for op, reads in (("tree", ("q", "k", "v", "mask")), ("cross", ("q", "lengths")))
         for w in ("out", "lse", "workspace") for r in reads + ("out", "lse", "workspace") if r != w]


@pytest.mark.parametrize("op,written,other", PAIRS)
def test_memory_that_is_written_lies_apart(setup, op, written, other):
    import torch
    from bit_kv_cache_append_gb300 import binding as Bd
    gc, sizes, room, place = setup
    align = {"out": 16, "lse": 4, "workspace": 256}[written]
    low = place[other] - sizes[written]            # its end touches the other's begin
    for at in (low + align, place[other]):
        with pytest.raises(Bd.KVError) as e:
            call(setup, op, **{written: at})
        assert e.value.status == Bd.KV_ERR_INVALID_ARG
        assert "overlap" in str(e.value)
    room.zero_()
    if low % align == 0:
        call(setup, op, **{written: low})
    torch.cuda.synchronize()
    gc.check_device_error()


@pytest.mark.parametrize("written", ["out", "lse", "workspace"])
def test_memory_of_the_cache_is_not_written(setup, written):
    """(An empty cache, so that nothing could be launched.)"""
    import torch
    from bit_kv_cache_append_gb300 import binding as Bd
    gc, sizes, room, place = setup
    big = Bd.KVCache(**dict(gc.kwargs, max_tokens=65536))
    q = torch.zeros((B, H * GQA, T, D), dtype=torch.float16, device="cuda")
    dtype, shape = {"out": (torch.float16, q.shape), "lse": (torch.float32, q.shape[:3]),
                    "workspace": (torch.uint8, (sizes["workspace"],))}[written]
    for at in (0, big.arena.numel() - sizes[written] & ~255):
        with pytest.raises(Bd.KVError) as e:
            big.cross_attn(0, q, **{written: big.arena[at:at + sizes[written]].view(dtype).view(shape)})
        assert e.value.status == Bd.KV_ERR_INVALID_ARG and "the cache" in str(e.value)
