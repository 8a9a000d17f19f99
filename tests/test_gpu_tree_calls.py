"""Calls of a tree-drafted step that its documentation allows or refuses, beside the operators' own tests."""
import dataclasses
import gc

import numpy as np
import pytest
import torch
from torch.multiprocessing.reductions import StorageWeakRef

import workloads
from oracle import tree
from test_gpu_tree import Tree, dev, host, kvc, reference_step  # noqa: F401  (kvc is a fixture)

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


def test_steps_in_a_row_from_the_lengths_on_the_device(kvc):
    """Three steps: positions, slots and lengths of each follow on the device from what the commit before it wrote, with
    nothing read on the host in between; every step is checked against its definition on the sequences so far."""
    hist, lens, T, L = [0, 15, 300, 77], [6, 6, 4, 1], 24, 2
    steps = [workloads.tree_decode(40 + i, hist, lens, T, L=L) for i in range(3)]
    wl = steps[0]
    B, Hq, Hkv, D = 4, wl.Hq, wl.Hkv, wl.D
    i32 = dict(dtype=torch.int32, device="cuda")
    k_pool, v_pool = dev(wl.k_pool), dev(wl.v_pool)
    h = kvc.kv_cache_create(kvc.KvcConfig(L, wl.NB, Hkv, D), k_pool, v_pool)
    table, tree_lens, turns = dev(wl.block_table), dev(wl.tree_lens), dev(kvc.kv_rope_turns(wl.inv_freq))
    most = table.shape[1] * 16
    ws = torch.empty(max(16, kvc.paged_decode_tree_plan(B, Hq, Hkv, D, most, T)), dtype=torch.uint8, device="cuda")
    node = torch.arange(T, **i32)
    now = torch.tensor(hist, **i32)  # the sequences' lengths
    done = []
    for x in steps:
        masks, depths = kvc.kv_tree_masks(x.parents, x.tree_lens)
        at = now[:, None] + node
        slots = table.gather(1, (at // 16).clamp(max=table.shape[1] - 1).long()).long() * 16 + at % 16
        slots = torch.where(node < tree_lens[:, None], slots, -1).flatten()
        positions, ctx = (now[:, None] + dev(depths)).flatten(), now + tree_lens
        q_rot, out = (torch.zeros((L, B, T, Hq, D), dtype=torch.float16, device="cuda") for _ in range(2))
        qkv, qw, kw, masks = dev(x.qkv), dev(x.q_weight), dev(x.k_weight), dev(masks)
        for layer in range(L):
            q, k, v = (r.unflatten(1, (-1, D)) for r in qkv[layer].split((Hq * D, Hkv * D, Hkv * D), 1))
            kvc.kv_append_rope(q, k, v, positions, turns, q_rot[layer].view(B * T, Hq, D), k_pool[layer], v_pool[layer],
                               slots, q_weight=qw[layer], k_weight=kw[layer], eps=x.eps)
            kvc.paged_decode_tree_attention(q_rot[layer], k_pool[layer], v_pool[layer], table, ctx, masks, x.scale,
                                            out[layer], ws, most, tree_lens=tree_lens)
        path = torch.zeros((B, T), **i32)
        n, token, new = (torch.zeros(B, **i32) for _ in range(3))
        kvc.draft_tree_verify(dev(x.p), dev(x.q), dev(x.tokens), dev(x.parents), dev(x.uniforms), path, n, token,
                              tree_lens=tree_lens)
        kvc.kv_tree_commit(h, table, ctx, path, n, new, tree_lens=tree_lens)
        done.append((out, path, n, token, new, k_pool.clone(), v_pool.clone()))
        now = new
    torch.cuda.synchronize()
    assert kvc.kvc_device_error_flags() == 0
    length, pools = np.array(hist, np.int32), [wl.k_pool, wl.v_pool]
    live = node.cpu().numpy()[None] < wl.tree_lens[:, None]
    for x, (out, path, n, token, new, k_dev, v_dev) in zip(steps, done):
        ref = dataclasses.replace(x, hist=length, k_pool=pools[0], v_pool=pools[1], block_table=wl.block_table)
        masks, qs, pools = reference_step(ref)
        for layer in range(L):
            want, spread = tree.tree_attention(qs[layer], pools[0][layer], pools[1][layer], wl.block_table,
                                               length + wl.tree_lens, masks, wl.tree_lens, x.scale)
            # the query's and the keys' own fp16 roundings, as in the single step's test
            qk = np.abs(qs[layer].astype(np.float64)).max() * np.abs(pools[0][layer].astype(np.float64)).max() * x.scale
            bound = 2 * (2.0 ** -10 * qk * np.sqrt(D) + 2.0 ** -11) * spread + 2.0 ** -11 * np.abs(want) + 2e-4
            assert (np.abs(host(out[layer]).astype(np.float64) - want)[live] <= bound[live]).all()
        walks = [tree.verify(x.p[b, :m], x.q[b, :m], x.tokens[b, :m], x.parents[b, :m],
                             x.uniforms[b, :m].astype(np.float64), False) for b, m in enumerate(lens)]
        paths = np.full((B, T), -1, np.int32)
        for b, (walk, _) in enumerate(walks):
            paths[b, :len(walk)] = walk
        assert (host(path) == paths).all() and host(token).tolist() == [w[1] for w in walks]
        length = tree.commit(pools, wl.block_table, length + wl.tree_lens, wl.tree_lens, paths, host(n))
        assert (host(new) == length).all()
        for pool, got in zip(pools, (k_dev, v_dev)):
            for b in range(B):
                for layer in range(L):
                    rows = tree.rows_of(pool[layer], wl.block_table[b], int(length[b])).astype(np.float64)
                    have = tree.rows_of(host(got[layer]), wl.block_table[b], int(length[b]))
                    assert np.abs(have - rows).max() <= 2.0 ** -10 * np.abs(rows).max()
    assert (length > np.array(hist) + 3).any()  # some path was longer than its root
    kvc.kv_cache_destroy(h)


def test_a_commit_to_pools_of_another_device_is_refused(kvc):
    pools = [torch.zeros((1, 4, 2, 16, 64), dtype=torch.float16, device="cuda") for _ in range(2)]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    h = kvc.kv_cache_create(kvc.KvcConfig(1, 4, 2, 64), *pools)
    try:
        assert kvc._caches[h].device == 0
        kvc._caches[h].device = 1
        with pytest.raises(ValueError, match="pools on cuda:1"):
            kvc.kv_tree_commit(h, i32(2, 3).view(1, 2), i32(6), i32(0, 3).view(1, 2), i32(2), i32(0), tree_lens=i32(4))
    finally:
        kvc.kv_cache_destroy(h)


@pytest.mark.parametrize("V", [2, 33, 5000])
def test_no_child_is_kept_of_a_residual_that_is_nothing(kvc, V):
    """Two refusals leave 3 * 2^-49 of the last child's token, which is nothing in the sums' units of 2^-45: the child is
    refused, although that difference by itself is positive, and the token comes from the target's own row."""
    p, q = np.zeros((2, 4, V), np.float32)
    x, y = 0, V - 1
    q[0, x], q[0, y] = 0.5, 0.5 - 2.0 ** -25
    p[0, x], p[0, y] = 0.5 - 2.0 ** -24, 0.5 + 2.0 ** -24
    i32 = lambda *a: torch.tensor([a], dtype=torch.int32, device="cuda")  # noqa: E731
    for u0, token in ((0.25, x), (0.75, y)):
        u = torch.tensor([[u0, 1 - 2.0 ** -24, 0.5, 0.5]], dtype=torch.float32, device="cuda")
        path, n, nxt = i32(9, 9, 9, 9), i32(9)[0], i32(9)[0]
        kvc.draft_tree_verify(dev(p[None]), dev(q[None]), i32(0, x, x, y), i32(-1, 0, 0, 0), u, path, n, nxt, distinct=True)
        assert path.tolist() == [[0, -1, -1, -1]] and n.item() == 1 and nxt.item() == token
    assert kvc.kvc_device_error_flags() == 0


def test_as_many_sequences_as_a_call_takes(kvc):
    """65,535 sequences of one block each: append, attention of two-node chains, verification, commit."""
    B, D, n = 65535, 64, 2
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float16)  # noqa: E731
    pools = [rows(1, B, 1, 16, D) for _ in range(2)]
    table = torch.randperm(B, generator=g, device="cuda").int()[:, None].contiguous()
    hist = torch.randint(0, 14, (B,), generator=g, device="cuda", dtype=torch.int32)
    ctx = hist + n
    node = torch.arange(n, dtype=torch.int32, device="cuda")
    at = hist[:, None] + node
    slots = (table.long() * 16 + at).flatten()
    q, k, v = rows(B * n, 1, D), rows(B * n, 1, D), rows(B * n, 1, D)
    q_out = torch.empty_like(q)
    kvc.kv_append_rope(q, k, v, None, None, q_out, pools[0][0], pools[1][0], slots)
    assert torch.equal(q_out, q)
    assert torch.equal(pools[0].view(-1, D)[slots], k[:, 0]) and torch.equal(pools[1].view(-1, D)[slots], v[:, 0])
    masks = torch.tensor([[1, 3]], dtype=torch.int64, device="cuda").expand(B, n).contiguous()
    out = torch.empty((B, n, 1, D), dtype=torch.float32, device="cuda")
    ws = torch.empty(max(16, kvc.paged_decode_tree_plan(B, 1, 1, D, 16, n)), dtype=torch.uint8, device="cuda")
    kvc.paged_decode_tree_attention(q_out.view(B, n, 1, D), pools[0][0], pools[1][0], table, ctx, masks, 0.125, out, ws, 16)
    K, V = (p.view(B, 16, D)[table[:, 0].long()].double() for p in pools)
    s = q.view(B, n, D).double() @ K.transpose(1, 2) * 0.125
    seen = torch.arange(16, device="cuda")[None, None] <= at[:, :, None]
    w = torch.softmax(s.masked_fill(~seen, -float("inf")), -1)
    # per weight 2^-20, D 2^-24 of its score's terms (below 64 * 25 * 0.125) and the sums'; values up to 6
    assert (out[:, :, 0] - w @ V).abs().max() < 2 * (2.0 ** -20 + 64 * 2.0 ** -24 * 200 + 2.0 ** -20) * 6
    p = torch.rand(B, n, 3, generator=g, device="cuda")
    p /= p.sum(-1, keepdim=True)
    tokens, parents = torch.full((B, n), 1, dtype=torch.int32, device="cuda"), (node - 1).expand(B, n).contiguous()
    u = torch.rand(B, n, generator=g, device="cuda")
    path = torch.zeros((B, n), dtype=torch.int32, device="cuda")
    length, token, new = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
    kvc.draft_tree_verify(p, p.flip(-1).contiguous(), tokens, parents, u, path, length, token)
    kept = u[:, 1] < 1  # token 1 has the same mass in both rows
    assert bool(kept.all()) and (length == 2).all() and torch.equal(path, node.expand(B, n))
    c = p[:, 1].double().cumsum(-1)
    near = ((c - u[:, :1].double() * c[:, -1:]).abs().amin(-1) < 2.0 ** -40)
    assert ((token == (c <= u[:, :1].double() * c[:, -1:]).sum(-1)) | near).all()
    # node 1 alone behind the root's place: a path of the root keeps one row, all others two
    length[::3] = 1
    h = kvc.kv_cache_create(kvc.KvcConfig(1, B, 1, D), *pools)
    before = [x.clone() for x in pools]
    kvc.kv_tree_commit(h, table, ctx, path, length, new)
    assert torch.equal(new, hist + length) and all(torch.equal(a, b) for a, b in zip(before, pools))
    kvc.kv_cache_destroy(h)
    assert kvc.kvc_device_error_flags() == 0


@pytest.mark.parametrize("graphs", [False, True])
def test_two_sessions_at_once(kvc, graphs):
    """Whole steps of two caches on two streams, over and over: each as if it were alone."""
    from paged_kv_cache_27_gb300.harness import TreeSession
    wls = [workloads.tree_decode(5, [3000, 40, 900], [12, 9, 12], 12, L=3),
           workloads.tree_decode(6, [100] * 30, [24] * 30, 24, L=3, Hq=8, Hkv=1)]
    sessions = [TreeSession(wl) for wl in wls]
    fresh = [[p.clone() for p in (s.k_pool, s.v_pool)] for s in sessions]
    results = lambda s: [x.clone() for x in (s.out, s.path, s.path_len, s.next_token, s.new_context_lens, s.k_pool, s.v_pool)]  # noqa: E731

    def run(s, first):
        for p, x in zip((s.k_pool, s.v_pool), first):
            p.copy_(x)
        s.step()
    alone = []
    for s, first in zip(sessions, fresh):
        run(s, first)
        torch.cuda.synchronize()
        alone.append(results(s))
    streams = [torch.cuda.Stream() for _ in sessions]
    captured = []
    if graphs:
        for s, first, st in zip(sessions, fresh, streams):
            captured.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(captured[-1], stream=st):
                run(s, first)
    torch.cuda.synchronize()
    for _ in range(20):
        for s in sessions:
            s.out.zero_()
            s.path.zero_()
        torch.cuda.synchronize()
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                if graphs:
                    captured[i].replay()
                else:
                    run(sessions[i], fresh[i])
        torch.cuda.synchronize()
        for s, want in zip(sessions, alone):
            # (bit patterns: cache rows that nobody owns may be NaN)
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(results(s), want))
    assert kvc.kvc_device_error_flags() == 0
    for s in sessions:
        s.close()


def test_offsets_beyond_32_bits(kvc):
    """Pools, projected rows and probabilities of more than 2^31 elements: what lies at their far end comes out as it does
    in small ones."""
    D, NB, T = 128, 1_200_000, 5
    g = torch.Generator(device="cuda").manual_seed(2)
    rows = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float16)  # noqa: E731
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    turns = dev(kvc.kv_rope_turns(1e4 ** (-np.arange(0, D, 2) / D)))
    # a sequence of 37 tokens, 5 of them nodes, at a pool's far end and in a pool of its own
    small = [rows(1, 4, 1, 16, D) for _ in range(2)]
    far = [torch.empty((1, NB, 1, 16, D), dtype=torch.float16, device="cuda") for _ in range(2)]
    assert far[0].numel() > 2 ** 31
    where = {0: NB - 1, 1: 3, 2: NB - 2}  # block of the small pool: block of the large one
    for s, f in zip(small, far):
        for a, b in where.items():
            f[0, b] = s[0, a]
    q, k, v = rows(T, 4, D), rows(T, 1, D), rows(T, 1, D)
    v[2, 0, 7] = float("inf")  # the way that looks values up again by their place in the pool
    pos = torch.arange(32, 37, dtype=torch.int32, device="cuda")
    masks = torch.tensor([[1, 3, 7, 11, 19]], dtype=torch.int64, device="cuda")
    done = []
    for pools, blocks in ((small, [0, 1, 2]), (far, [where[i] for i in range(3)])):
        table, slots = i32(*blocks).view(1, 3), blocks[2] * 16 + torch.arange(T, device="cuda")
        q_out, out = torch.empty_like(q), torch.empty((1, T, 4, D), dtype=torch.float16, device="cuda")
        kvc.kv_append_rope(q, k, v, pos, turns, q_out, pools[0][0], pools[1][0], slots)
        kvc.paged_decode_tree_attention(q_out[None], pools[0][0], pools[1][0], table, i32(37), masks, D ** -0.5, out, None, 48)
        h, new = kvc.kv_cache_create(kvc.KvcConfig(1, pools[0].shape[1], 1, D), *pools), i32(0)
        kvc.kv_tree_commit(h, table, i32(37), i32(0, 2, 4).view(1, 3), i32(3), new, tree_lens=i32(T))
        done.append((q_out, out, new, *(p[0, blocks[2], 0, :T].clone() for p in pools)))
        kvc.kv_cache_destroy(h)
    assert torch.isinf(done[0][1]).any()
    for a, b in zip(*done):
        assert torch.equal(a, b)
    del far
    # projected rows, in place
    n = 2 ** 20 + 3
    x = torch.empty((n, 17, D), dtype=torch.float16, device="cuda")
    assert x.numel() > 2 ** 31
    x[-9:] = rows(9, 17, D)
    k, v = rows(9, 1, D), rows(9, 1, D)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    ref, want = x[-9:].clone(), torch.empty((9, 17, D), dtype=torch.float16, device="cuda")
    kvc.kv_append_rope(ref, k, v, pos[-9:].clone(), turns, want)
    kv = torch.zeros((n, 1, D), dtype=torch.float16, device="cuda")
    kvc.kv_append_rope(x, kv, kv, pos, turns, x)
    assert torch.equal(x[-9:], want)
    del x, kv
    # probabilities: the last sequence's chain of nodes is kept to its end, and its last row drawn from
    B, T, V = 3, 64, 2 ** 24
    p = torch.zeros((B, T, V), dtype=torch.float16, device="cuda")
    assert p.numel() > 2 ** 31
    tokens = torch.randint(0, V, (B, T), generator=g, device="cuda", dtype=torch.int32)
    tokens[-1, -1] = V - 1
    for t in range(T - 1):
        p[torch.arange(B), t, tokens[:, t + 1].long()] = 1
    p[:, T - 1, V - 2] = 1
    parents = torch.arange(-1, T - 1, device="cuda", dtype=torch.int32).expand(B, T).contiguous()
    path = torch.zeros((B, T), dtype=torch.int32, device="cuda")
    length, token = i32(0, 0, 0), i32(0, 0, 0)
    kvc.draft_tree_verify(p, p, tokens, parents, torch.rand((B, T), generator=g, device="cuda"), path, length, token)
    assert length.tolist() == [T] * B and torch.equal(path, parents + 1) and token.tolist() == [V - 2] * B
    assert kvc.kvc_device_error_flags() == 0
