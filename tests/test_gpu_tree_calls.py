"""Calls of a tree-drafted step that its documentation allows or refuses, beside the operators' own tests."""
import gc

import pytest
import torch
from torch.multiprocessing.reductions import StorageWeakRef

import workloads
from test_gpu_tree import Tree, kvc  # noqa: F401  (kvc is a fixture)

pytestmark = pytest.mark.gpu


def test_a_workspace_among_the_tensors_of_its_call_is_refused(kvc):
    w = Tree(30, [30000], [4], 4, 4, 2, 64)
    w.run(kvc)
    d = w.d
    need = kvc.paged_decode_tree_plan(1, 4, 2, 64, w.max_ctx, 4)
    assert need > 0
    room = torch.zeros(need + 4096, dtype=torch.uint8, device="cuda")
    q = room[need - 512:need - 512 + d["q"].numel() * 2].view(torch.float16).view_as(d["q"])
    out = room[:w.out.numel() * 2].view(torch.float16).view_as(w.out)
    args = lambda q, out: (q, d["k"], d["v"], d["table"], d["ctx"], d["masks"], w.scale, out, room[:need], w.max_ctx)  # noqa: E731
    for a in (args(q, w.out), args(d["q"], out)):
        with pytest.raises(kvc.KvcError, match="overlaps") as e:
            kvc.paged_decode_tree_attention(*a)
        assert e.value.name == "KVC_ERR_INVALID"
    got = room[need:need + w.out.numel() * 2].view(torch.float16).view_as(w.out)  # behind it
    kvc.paged_decode_tree_attention(*args(d["q"], got))
    assert torch.equal(got, w.out)


def test_a_prepared_commit_and_its_cache(kvc):
    """It keeps the pools alive as long as it lives, and refuses once the cache is destroyed."""
    pools = [torch.zeros((1, 4, 2, 16, 64), dtype=torch.float16, device="cuda") for _ in range(2)]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pools[0].view(4, 2, 16, 64)[2, :, 5] = 1.0
    new = torch.zeros(1, dtype=torch.int32, device="cuda")
    h = kvc.kv_cache_create(kvc.KvcConfig(1, 4, 2, 64), *pools)
    alive = [StorageWeakRef(p.untyped_storage()) for p in pools]
    call = kvc.kv_tree_commit(h, i32(2, 3).view(1, 2), i32(6), i32(0, 3).view(1, 2), i32(2), new, tree_lens=i32(4),
                              prepare=True)
    rows = pools[0].view(4, 2, 16, 64)[2, :, 3].clone()
    del pools
    gc.collect()
    assert not any(p.expired() for p in alive)
    call()
    torch.cuda.synchronize()
    assert new.item() == 4 and (rows == 0).all()
    kept = torch.empty(0, dtype=torch.float16, device="cuda").set_(call._keep[-2], 0, (4, 2, 16, 64))
    assert (kept[2, :, 3] == 1).all()
    kvc.kv_cache_destroy(h)
    with pytest.raises(ValueError, match="destroyed"):
        call()
    del call, kept
    gc.collect()
    assert all(p.expired() for p in alive)


def test_a_commit_to_freed_pools_is_refused(kvc):
    pools = [torch.zeros((1, 4, 2, 16, 64), dtype=torch.float16, device="cuda") for _ in range(2)]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    args = (i32(2, 3).view(1, 2), i32(6), i32(0, 3).view(1, 2), i32(2), i32(0))
    h = kvc.kv_cache_create(kvc.KvcConfig(1, 4, 2, 64), *pools)
    try:
        pools.clear()
        gc.collect()
        for prepare in (False, True):
            with pytest.raises(ValueError, match="freed"):
                kvc.kv_tree_commit(h, *args, tree_lens=i32(4), prepare=prepare)
    finally:
        kvc.kv_cache_destroy(h)


def test_a_closed_session_does_not_step(kvc):
    from paged_kv_cache_27_gb300.harness import TreeSession
    s = TreeSession(workloads.tree_decode(3, [20], [4], 4, L=1))
    s.step()
    torch.cuda.synchronize()
    s.close()
    with pytest.raises(ValueError, match="destroyed"):
        s.step()
    torch.cuda.synchronize()


def test_an_ordinary_decode_behind_a_step_under_launch_overlap(kvc):
    """With another kernel between the commit and the decode call, as the header asks, the decode follows the lengths and
    rows that the commit wrote, launch overlap on or off."""
    from paged_kv_cache_27_gb300.harness import TreeSession
    wl = workloads.tree_decode(4, [700, 33, 300], [12, 7, 9], 12, L=2)
    s = TreeSession(wl)
    fresh = [p.clone() for p in (s.k_pool, s.v_pool)]
    q = torch.randn(3, wl.Hq, wl.D, device="cuda").half()
    _, _, need = kvc.paged_decode_plan(3, wl.Hq, wl.Hkv, wl.D, s.max_ctx)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    big = torch.zeros(32 << 20, device="cuda")
    outs = []
    try:
        for on in (False, True, True):
            kvc.kvc_set_launch_overlap(on)
            for p, x in zip((s.k_pool, s.v_pool), fresh):
                p.copy_(x)
            s.new_context_lens.fill_(1)
            out = torch.empty((2, 3, wl.Hq, wl.D), dtype=torch.float32, device="cuda")
            torch.cuda.synchronize()
            big.add_(1)  # long, so that its successors queue up
            s.step()
            big[:1].add_(1)
            for layer in range(2):
                kvc.paged_decode_attention(q, s.k_pool[layer], s.v_pool[layer], s.block_table, s.new_context_lens,
                                           wl.scale, out[layer], ws, s.max_ctx)
            torch.cuda.synchronize()
            outs.append(out)
    finally:
        kvc.kvc_set_launch_overlap(False)
    assert kvc.kvc_device_error_flags() == 0
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    s.close()
